// Rows of a call on the 8-bit or the 4-bit cache: which tokens of a sequence they are, their pages and
// tail block, and the launch of one warp for each (page, KV head, keys or values).
#pragma once

#include <algorithm>

#include "common.cuh"
#include "kv8_layout.cuh"

namespace oscar {

constexpr int kCWarps = 4;

struct Kv8CacheParams {
  int hkv, max_pages, batch, pages_per_seq, max_rows;
  int room;                   // most tokens of a sequence: whole pages of its table row, a tail's, what int32 holds
  int64_t n_pages, n_tails, total_rows, k_stride, v_stride;
  uint8_t* pool;
  uint16_t* tail;
  const int32_t* page_table;
  const int32_t* tail_ids;
  int32_t* status;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* k_out;
  uint16_t* v_out;
  const int32_t* first;       // position of each sequence's first row
  const int32_t* row_starts;
  const int32_t* seq_lens;    // gather: tokens stored
};

// The rows of sequence b: positions [t0, t1), first row r0.  false when there are
// none or they are not acceptable (reported).
struct Span {
  int t0, t1;
  int64_t r0;
};

__device__ __forceinline__ void report(const Kv8CacheParams& p, int bits) {
  if (p.status && (threadIdx.x & 31) == 0) atomicOr(p.status, bits);
}

__device__ __forceinline__ bool span_of(const Kv8CacheParams& p, int b, Span& s) {
  const int r0 = p.row_starts[b], r1 = p.row_starts[b + 1], t0 = p.first[b];
  const int64_t n = static_cast<int64_t>(r1) - r0;
  if (n == 0) return false;
  if (n < 0 || n > p.max_rows || r0 < 0 || r1 > p.total_rows || t0 < 0 || t0 + n > p.room) {
    report(p, OSCAR_DEVERR_SEQ_LEN);
    return false;
  }
  s.t0 = t0;
  s.t1 = t0 + static_cast<int>(n);
  s.r0 = r0;
  return true;
}

__device__ __forceinline__ int64_t page_id(const Kv8CacheParams& p, int b, int pg) {
  const int id = p.page_table[static_cast<size_t>(b) * p.max_pages + pg];
  if (id < 0 || id >= p.n_pages) {
    report(p, OSCAR_DEVERR_PAGE_ID);
    return -1;
  }
  return id;
}

// The tail area (keys or values) of sequence b; null when its id is refused.
template <int D>
__device__ __forceinline__ uint16_t* tail_area(const Kv8CacheParams& p, int b, int h, int kv) {
  const int64_t id = p.tail_ids ? p.tail_ids[b] : b;
  if (id < 0 || id >= p.n_tails) {
    report(p, OSCAR_DEVERR_PAGE_ID);
    return nullptr;
  }
  return p.tail + ((id * p.hkv + h) * 2 + kv) * Kv8Fmt<D>::kTailHalf;
}

// A lane's part of one block: kUnits chunks of 16 values, as packed bf16 pairs in
// chunk order.  Keys: 16 channels of a token; values: 4 channels x 4 tokens.
template <int D>
struct Lane {
  static constexpr int kUnits = D / 32;
  // chunk u of this lane
  static __device__ __forceinline__ void key(int lane, int u, int& t, int& cc) {
    constexpr int kPer = D / 16;                 // chunks of a token: neighbouring lanes
    t = lane / kPer + u * (32 / kPer);
    cc = lane % kPer;
  }
  static __device__ __forceinline__ void value(int lane, int u, int& tg, int& cg) {
    constexpr int kPer = D / 4;                  // channel groups of a row
    tg = (lane + 32 * u) / kPer;
    cg = (lane + 32 * u) % kPer;
  }
};

// Four rows of 4 channels (row r in w[2r], w[2r + 1]) <-> chunk order (channel x:
// tokens 0..3 in w[2x], w[2x + 1]), as packed pairs of 16-bit values.
__device__ __forceinline__ void transpose4(uint32_t (&w)[8]) {
  uint32_t o[8];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t sel = (x & 1) ? 0x7632 : 0x5410;
    o[2 * x] = __byte_perm(w[x >> 1], w[2 + (x >> 1)], sel);
    o[2 * x + 1] = __byte_perm(w[4 + (x >> 1)], w[6 + (x >> 1)], sel);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = o[i];
}

// Rows of positions [lo, s.t1) into their tail slots.
template <int D>
__device__ __forceinline__ void store_tail(const Kv8CacheParams& p, const Span& s, int h, int kv,
                                           int lo, uint16_t* tail, int lane) {
  const uint16_t* src = kv ? p.v : p.k;
  const int64_t stride = kv ? p.v_stride : p.k_stride;
  constexpr int kPer = D / 4;   // 4 channels a lane
  const int n = (s.t1 - lo) * kPer;
  for (int i = lane; i < n; i += 32) {
    const int pos = lo + i / kPer, cg = i % kPer, t = pos % kPage;
    const uint2 w = *reinterpret_cast<const uint2*>(src + (s.r0 + pos - s.t0) * stride + h * D + 4 * cg);
    if (kv == 0) {
      *reinterpret_cast<uint2*>(tail + kv8_key_chunk(t, cg >> 2) * 16 + 4 * (cg & 3)) = w;
    } else {
      uint16_t* dst = tail + kv8_value_chunk(t >> 2, cg) * 16 + (t & 3);
      dst[0] = static_cast<uint16_t>(w.x);
      dst[4] = static_cast<uint16_t>(w.x >> 16);
      dst[8] = static_cast<uint16_t>(w.y);
      dst[12] = static_cast<uint16_t>(w.y >> 16);
    }
  }
}

template <typename Kern>
oscar_status launch_cache(Kern kernel, const Kv8CacheParams& p, cudaStream_t st, int units) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * static_cast<unsigned>(p.pages_per_seq),
                     static_cast<unsigned>((units + kCWarps - 1) / kCWarps));   // a warp each
  cfg.blockDim = dim3(32 * kCWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

// Checks and fields that placing and gathering share.
inline oscar_status cache_params(const oscar_kv8_desc* c, const int32_t* first, const int32_t* row_starts,
                          int32_t batch, int64_t total_rows, int32_t max_rows, Kv8CacheParams* p) {
  if (batch < 0 || total_rows < 0 || max_rows < 0) return OSCAR_ERR_INVALID_ARG;
  if (batch == 0 || total_rows == 0 || max_rows == 0) return OSCAR_OK;
  if (!first || !row_starts) return OSCAR_ERR_INVALID_ARG;
  if (total_rows > 0x7fffffff) return OSCAR_ERR_UNSUPPORTED;   // row_starts are int32
  // pages that so many consecutive positions can touch
  const auto pages = [](int64_t rows) { return (rows + kPage - 2) / kPage + 1; };
  if (pages(max_rows) * batch > 0x7fffffff || c->num_kv_heads > kCWarps * 65535 / 2) return OSCAR_ERR_UNSUPPORTED;
  p->hkv = c->num_kv_heads;
  p->max_pages = c->max_pages_per_seq;
  p->batch = batch;
  p->pages_per_seq = static_cast<int>(pages(std::min<int64_t>(max_rows, total_rows)));   // (no sequence has more)
  p->max_rows = max_rows;
  p->room = static_cast<int>(std::min<int64_t>(0x7fffffff, static_cast<int64_t>(c->max_pages_per_seq) * kPage + kPage - 1));
  p->n_pages = c->num_pages;
  p->n_tails = c->num_tails;
  p->total_rows = total_rows;
  p->pool = static_cast<uint8_t*>(c->pool);
  p->tail = static_cast<uint16_t*>(c->tail);
  p->page_table = c->page_table;
  p->tail_ids = c->tail_ids;
  p->status = c->status;
  p->first = first;
  p->row_starts = row_starts;
  return OSCAR_OK;
}

// Those of placing: the new rows of k and v.
inline oscar_status place_params(const oscar_kv8_desc* c, const void* k, const void* v, int64_t k_stride,
                                 int64_t v_stride, const int32_t* lens_before, const int32_t* row_starts,
                                 int32_t batch, int64_t total_rows, int32_t max_new, Kv8CacheParams* p) {
  const oscar_status s = cache_params(c, lens_before, row_starts, batch, total_rows, max_new, p);
  if (s != OSCAR_OK || p->batch == 0) return s;
  if (!k || !v || ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15))
    return OSCAR_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(c->num_kv_heads) * c->head_dim;
  if (k_stride < row || v_stride < row || ((k_stride | v_stride) & 7)) return OSCAR_ERR_INVALID_ARG;
  p->k = static_cast<const uint16_t*>(k);
  p->v = static_cast<const uint16_t*>(v);
  p->k_stride = k_stride;
  p->v_stride = v_stride;
  return OSCAR_OK;
}

// Those of reading back.
inline oscar_status gather_params(const oscar_kv8_desc* c, const int32_t* seq_lens, const int32_t* first,
                                  const int32_t* row_starts, int32_t batch, int64_t total_rows, int32_t max_rows,
                                  void* k_out, void* v_out, Kv8CacheParams* p) {
  const oscar_status s = cache_params(c, first, row_starts, batch, total_rows, max_rows, p);
  if (s != OSCAR_OK || p->batch == 0) return s;
  if (!seq_lens || !k_out || !v_out ||
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15))
    return OSCAR_ERR_INVALID_ARG;
  p->seq_lens = seq_lens;
  p->k_out = static_cast<uint16_t*>(k_out);
  p->v_out = static_cast<uint16_t*>(v_out);
  return OSCAR_OK;
}

}  // namespace oscar
