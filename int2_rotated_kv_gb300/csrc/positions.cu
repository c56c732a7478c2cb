// What a serving step derives from request lengths and positions: page tables and
// per-token lists, and the rotary embedding of queries and keys.
//
// oscar_extend_pages.  A table holds pages for the tokens t < n - hold_back of a
// sequence of n tokens: pages(n) = max(0, ceil((n - hold_back) / 16)).  One CTA forms
// both exclusive prefix sums over the batch (rows, new pages) and advances the
// lengths and the free-list cursor; the rows and the new table entries follow in
// the same CTA when they are few, else in a grid of their own that finds each row's
// sequence by bisection of the prefix sums.  Bound by latency (a chain of a scan and
// two dependent loads) for a decode step, by the 16 bytes written per row for a
// large prefill.
//
// oscar_rope.  For a rotated pair (a, b) at position m with frequency f turns per
// token: a' = A (a cos 2 pi m f - b sin 2 pi m f), b' = A (b cos + a sin).  f is held
// as a 64-bit fraction, so m f modulo one turn is the low 64 bits of an integer
// product: no rounding at all whatever the position; the upper 32 bits of it go to
// sincospif.  cos and sin are formed once per (token, pair) in shared memory and
// shared by all heads.  Bound by HBM: 2 bytes read and 2 written per value.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace oscar {

inline cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                     cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// ------------------------------------------------------------------ page tables

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int64_t kInlineRows = 2048;   // see oscar_extend_pages

struct PagesParams {
  int batch, max_pages, hold;
  int64_t n_free, max_rows;
  int32_t* table;
  const int32_t* lens;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* cursor;
  int32_t* lens_after;
  int32_t* page_starts;
  int32_t* row_starts;
  int32_t* seq_ids;
  int32_t* positions;
  int64_t* slots;
  int32_t* status;
  int fill;   // the scan's CTA also writes rows and table entries
};

__device__ __forceinline__ int pages_held(int n, int hold) {
  return n > hold ? (n - hold - 1) / kPage + 1 : 0;
}

// Index of the sequence whose [starts[b], starts[b + 1]) holds i (starts ascend).
__device__ __forceinline__ int sequence_of(const int32_t* starts, int batch, int i) {
  int lo = 0, hi = batch;   // starts[lo] <= i < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Page of logical index `pg` that the step gives to sequence b, from the free list.
__device__ __forceinline__ int fresh_page(const PagesParams& p, int first, int pg, int held_before) {
  const int64_t at = static_cast<int64_t>(first) + pg - held_before;
  return at < p.n_free ? p.free_pages[at] : -1;
}

// Rows and new table entries, `i` of `n` workers.
__device__ __forceinline__ void fill_rows(const PagesParams& p, int64_t i, int64_t n) {
  const int64_t rows = p.row_starts[p.batch];
  for (int64_t r = i; r < p.max_rows; r += n) {
    int b = -1, pos = -1;
    int64_t slot = -1;
    if (r < rows) {
      b = sequence_of(p.row_starts, p.batch, static_cast<int>(r));
      const int start = p.row_starts[b], after = p.lens_after[b];
      const int before = after - (p.row_starts[b + 1] - start);
      pos = before + static_cast<int>(r) - start;
      const int pg = pos / kPage;
      if (p.slots && pg < p.max_pages && pg < pages_held(after, p.hold)) {
        const int held = pages_held(before, p.hold);
        const int id = pg >= held ? fresh_page(p, p.page_starts[b], pg, held)
                                  : p.table[static_cast<size_t>(b) * p.max_pages + pg];
        if (id >= 0) slot = static_cast<int64_t>(id) * kPage + pos % kPage;
      }
    }
    p.seq_ids[r] = b;
    p.positions[r] = pos;
    if (p.slots) p.slots[r] = slot;
  }
  const int first = p.page_starts[0];
  const int64_t fresh = static_cast<int64_t>(p.page_starts[p.batch]) - first;
  for (int64_t j = i; j < fresh; j += n) {
    const int at = first + static_cast<int>(j);
    const int b = sequence_of(p.page_starts, p.batch, at);
    const int after = p.lens_after[b];
    const int held = pages_held(after - (p.row_starts[b + 1] - p.row_starts[b]), p.hold);
    const int pg = held + at - p.page_starts[b];
    if (pg < p.max_pages)
      p.table[static_cast<size_t>(b) * p.max_pages + pg] = at < p.n_free ? p.free_pages[at] : -1;
  }
}

__global__ void __launch_bounds__(kScanThreads) extend_scan_kernel(const __grid_constant__ PagesParams p) {
  __shared__ int64_t sums[2][kScanThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cursor = *p.cursor;   // read before page_starts, which may hold it, is written
  // totals before this round; a cursor that cannot be used, or has run past the list, gives no page
  int64_t rows = 0, pages = cursor < 0 ? p.n_free : min(cursor, p.n_free);
  bool refused = cursor < 0;
  for (int b0 = 0; b0 < p.batch; b0 += kScanThreads) {
    const int b = b0 + tid;
    int n = 0, need = 0, before = 0;
    if (b < p.batch) {
      before = p.lens[b];
      n = p.new_tokens[b];
      // a sequence with an impossible length or more tokens than its table holds gets nothing
      const int64_t after = static_cast<int64_t>(before) + n;
      if (before < 0 || n < 0 || after > 0x7fffffff ||
          after - p.hold > static_cast<int64_t>(p.max_pages) * kPage) {
        n = 0;
        refused = true;
      }
      need = pages_held(before + n, p.hold) - pages_held(before, p.hold);
    }
    int64_t r = n, g = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, r, o), w = __shfl_up_sync(0xffffffffu, g, o);
      if (lane >= o) { r += u; g += w; }
    }
    if (lane == 31) { sums[0][warp] = r; sums[1][warp] = g; }
    __syncthreads();
    if (warp == 0) {
      int64_t u = sums[0][lane], w = sums[1][lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, u, o), y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) { u += x; w += y; }
      }
      sums[0][lane] = u;
      sums[1][lane] = w;
    }
    __syncthreads();
    const int64_t r0 = rows + r - n + (warp ? sums[0][warp - 1] : 0);
    const int64_t g0 = pages + g - need + (warp ? sums[1][warp - 1] : 0);
    if (b < p.batch) {
      // totals beyond int32 are cut here and reported; rows stop at max_rows anyway
      p.row_starts[b] = static_cast<int>(min(r0, static_cast<int64_t>(0x7fffffff)));
      p.page_starts[b] = static_cast<int>(min(g0, static_cast<int64_t>(0x7fffffff)));
      p.lens_after[b] = before + n;
    }
    rows += sums[0][kScanThreads / 32 - 1];
    pages += sums[1][kScanThreads / 32 - 1];
    __syncthreads();
  }
  if (tid == 0) {
    p.row_starts[p.batch] = static_cast<int>(min(rows, static_cast<int64_t>(0x7fffffff)));
    p.page_starts[p.batch] = static_cast<int>(min(pages, static_cast<int64_t>(0x7fffffff)));
  }
  if (p.status) {
    int bits = 0;
    if (refused || (tid == 0 && rows > p.max_rows)) bits |= OSCAR_DEVERR_SEQ_LEN;
    if (tid == 0 && pages > p.n_free) bits |= OSCAR_DEVERR_NO_PAGES;
    if (bits) atomicOr(p.status, bits);
  }
  if (p.fill) {
    __syncthreads();   // this CTA's global writes above are read back
    fill_rows(p, tid, kScanThreads);
  }
}

__global__ void __launch_bounds__(kFillThreads) extend_fill_kernel(const __grid_constant__ PagesParams p) {
  pdl_wait();
  pdl_trigger();
  fill_rows(p, static_cast<int64_t>(blockIdx.x) * kFillThreads + threadIdx.x,
            static_cast<int64_t>(gridDim.x) * kFillThreads);
}

// ----------------------------------------------------------------------- rotary

constexpr int kRopeThreads = 256;

struct RopeParams {
  int hq, hkv, d, half, tokens;   // half: rotated pairs per head; tokens per CTA
  int64_t n, q_stride, k_stride, q_out_stride, k_out_stride;
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  const int32_t* positions;
  const uint64_t* phases;
  float amplitude, sign;
  int copy;   // the output is not the input: unrotated channels are copied
};

__device__ __forceinline__ void rotate2(uint32_t a, uint32_t b, float2 c0, float2 c1, uint32_t& x,
                                        uint32_t& y) {
  const float a0 = bf16_lo_value(a), a1 = bf16_hi_value(a);
  const float b0 = bf16_lo_value(b), b1 = bf16_hi_value(b);
  x = pack_bf162(a0 * c0.x - b0 * c0.y, a1 * c1.x - b1 * c1.y);
  y = pack_bf162(b0 * c0.x + a0 * c0.y, b1 * c1.x + a1 * c1.y);
}

// kInter: pairs (2i, 2i + 1), else (i, i + half).  kVec: 16-byte accesses (the
// rotated part in runs of 8 channels, pointers and strides 16-byte aligned), else
// one pair, or one unrotated channel, at a time.
template <bool kInter, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 cs[];   // [tokens][half]: A cos, A sin
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.n - t0));
  for (int i = threadIdx.x; i < nt * p.half; i += kRopeThreads) {
    const int t = i / p.half, j = i - t * p.half;
    const int m = p.positions[t0 + t];
    // m * phase modulo 2^64: the position in the turn; its upper half as a signed fraction
    const uint64_t turn = p.phases[j] * static_cast<uint64_t>(static_cast<uint32_t>(m));
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * (1.f / 2147483648.f), &s, &c);
    cs[i] = make_float2(p.amplitude * c, p.amplitude * p.sign * s);
  }
  __syncthreads();
  const int heads = p.hq + p.hkv;
  constexpr int kRun = kVec ? 8 : 1;
  // items of a head: rotated pairs in runs, then the unrotated channels in runs
  const int pairs = kVec ? (kInter ? p.half / 4 : p.half / 8) : p.half;
  const int items = pairs + (p.copy ? (p.d - 2 * p.half) / kRun : 0);
  const int total = nt * heads * items;
  for (int i = threadIdx.x; i < total; i += kRopeThreads) {
    const int th = i / items, it = i - th * items;
    const int t = th / heads, h = th - t * heads;
    if (p.positions[t0 + t] < 0) continue;   // a padded row: left as it was
    const uint16_t* src = h < p.hq ? p.q + (t0 + t) * p.q_stride + h * p.d
                                   : p.k + (t0 + t) * p.k_stride + (h - p.hq) * p.d;
    uint16_t* dst = h < p.hq ? p.q_out + (t0 + t) * p.q_out_stride + h * p.d
                             : p.k_out + (t0 + t) * p.k_out_stride + (h - p.hq) * p.d;
    const float2* c = cs + t * p.half;
    if (it >= pairs) {
      const int ch = 2 * p.half + (it - pairs) * kRun;
      if constexpr (kVec) *reinterpret_cast<uint4*>(dst + ch) = *reinterpret_cast<const uint4*>(src + ch);
      else dst[ch] = src[ch];
    } else if constexpr (!kVec) {
      const int a = kInter ? 2 * it : it, b = kInter ? 2 * it + 1 : it + p.half;
      const float x = bf16_to_float(src[a]), y = bf16_to_float(src[b]);
      const float2 w = c[it];
      dst[a] = __bfloat16_as_ushort(__float2bfloat16_rn(x * w.x - y * w.y));
      dst[b] = __bfloat16_as_ushort(__float2bfloat16_rn(y * w.x + x * w.y));
    } else if constexpr (kInter) {
      const uint4 v = *reinterpret_cast<const uint4*>(src + 8 * it);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t o[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 r = c[4 * it + x];
        const float a = bf16_lo_value(w[x]), b = bf16_hi_value(w[x]);
        o[x] = pack_bf162(a * r.x - b * r.y, b * r.x + a * r.y);
      }
      *reinterpret_cast<uint4*>(dst + 8 * it) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(src + 8 * it);
      const uint4 b = *reinterpret_cast<const uint4*>(src + p.half + 8 * it);
      uint4 x, y;
      const float2* r = c + 8 * it;
      rotate2(a.x, b.x, r[0], r[1], x.x, y.x);
      rotate2(a.y, b.y, r[2], r[3], x.y, y.y);
      rotate2(a.z, b.z, r[4], r[5], x.z, y.z);
      rotate2(a.w, b.w, r[6], r[7], x.w, y.w);
      *reinterpret_cast<uint4*>(dst + 8 * it) = x;
      *reinterpret_cast<uint4*>(dst + p.half + 8 * it) = y;
    }
  }
}

}  // namespace oscar

using namespace oscar;

extern "C" {

oscar_status oscar_extend_pages(int32_t* page_table, int32_t max_pages_per_seq, const int32_t* lens,
                                const int32_t* new_tokens, int32_t batch, int32_t hold_back,
                                const int32_t* free_pages, int64_t num_free, const int32_t* cursor,
                                int32_t* lens_after, int32_t* page_starts, int32_t* row_starts,
                                int32_t* seq_ids, int32_t* positions, int64_t* slots,
                                int64_t max_rows, int32_t* status, void* stream) {
  if (batch < 0 || max_pages_per_seq < 1 || hold_back < 0 || num_free < 0 || max_rows < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (batch == 0) return OSCAR_OK;
  if (!page_table || !lens || !new_tokens || !cursor || !lens_after || !page_starts || !row_starts ||
      (num_free > 0 && !free_pages) || (max_rows > 0 && (!seq_ids || !positions)))
    return OSCAR_ERR_INVALID_ARG;
  if (num_free > 0x7fffffff || max_rows > 0x7fffffff || batch == 0x7fffffff)
    return OSCAR_ERR_UNSUPPORTED;
  PagesParams p{};
  p.batch = batch;
  p.max_pages = max_pages_per_seq;
  p.hold = hold_back;
  p.n_free = num_free;
  p.max_rows = max_rows;
  p.table = page_table;
  p.lens = lens;
  p.new_tokens = new_tokens;
  p.free_pages = free_pages;
  p.cursor = cursor;
  p.lens_after = lens_after;
  p.page_starts = page_starts;
  p.row_starts = row_starts;
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.slots = slots;
  p.status = status;
  p.fill = max_rows <= kInlineRows ? 1 : 0;
  cudaLaunchAttribute attr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3(kScanThreads), 0, st, &attr);
  if (cudaLaunchKernelEx(&cfg, extend_scan_kernel, p) != cudaSuccess) return OSCAR_ERR_CUDA;
  if (!p.fill) {
    const int64_t want = (max_rows + kFillThreads - 1) / kFillThreads;
    const int64_t most = static_cast<int64_t>(oscar_host::sm_count()) * 8;
    cfg = pdl_config(dim3(static_cast<unsigned>(std::min(want, most))), dim3(kFillThreads), 0, st, &attr);
    if (cudaLaunchKernelEx(&cfg, extend_fill_kernel, p) != cudaSuccess) return OSCAR_ERR_CUDA;
  }
  return OSCAR_OK;
}

oscar_status oscar_rope_phases(double base, int32_t rotary_dim, double factor, int32_t original_len,
                               double low_turns, double high_turns, uint64_t* phases_out) {
  if (!(base > 1.0) || !std::isfinite(base) || rotary_dim < 2 || rotary_dim % 2 || !phases_out ||
      !(factor >= 1.0) || !std::isfinite(factor) || original_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (original_len > 0 && !(std::isfinite(low_turns) && std::isfinite(high_turns) && low_turns < high_turns))
    return OSCAR_ERR_INVALID_ARG;
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    // turns per token; every value is below 1 / (2 pi)
    double f = std::pow(base, -2.0 * i / rotary_dim) / 6.283185307179586;
    if (original_len > 0) {
      const double keep = std::min(1.0, std::max(0.0, (f * original_len - low_turns) /
                                                          (high_turns - low_turns)));
      f = (1.0 - keep) * f / factor + keep * f;
    } else {
      f /= factor;
    }
    phases_out[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f, 64)));
  }
  return OSCAR_OK;
}

oscar_status oscar_rope(const void* q, const void* k, const int32_t* positions,
                        const uint64_t* phases, int64_t n, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim,
                        int32_t interleaved, float amplitude, int32_t inverse, int64_t q_stride,
                        int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride, void* q_out,
                        void* k_out, void* stream) {
  if (n < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + static_cast<int64_t>(num_kv_heads) < 1 ||
      head_dim < 2 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim ||
      !std::isfinite(amplitude) || (interleaved & ~1) || (inverse & ~1))
    return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if (!positions || !phases || (num_q_heads && (!q || !q_out)) || (num_kv_heads && (!k || !k_out)))
    return OSCAR_ERR_INVALID_ARG;
  const int64_t heads = static_cast<int64_t>(num_q_heads) + num_kv_heads;
  if (head_dim > 1024 || heads > 65536) return OSCAR_ERR_UNSUPPORTED;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if ((num_q_heads && (q_stride < qw || q_out_stride < qw)) ||
      (num_kv_heads && (k_stride < kw || k_out_stride < kw)))
    return OSCAR_ERR_INVALID_ARG;
  if ((num_q_heads && q_out == q && q_out_stride != q_stride) ||
      (num_kv_heads && k_out == k && k_out_stride != k_stride))
    return OSCAR_ERR_INVALID_ARG;   // in place: row by row
  RopeParams p{};
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.d = head_dim;
  p.half = rotary_dim / 2;
  p.n = n;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.q_stride = num_q_heads ? q_stride : 0;
  p.k_stride = num_kv_heads ? k_stride : 0;
  p.q_out_stride = num_q_heads ? q_out_stride : 0;
  p.k_out_stride = num_kv_heads ? k_out_stride : 0;
  p.positions = positions;
  p.phases = phases;
  p.amplitude = amplitude;
  p.sign = inverse ? -1.f : 1.f;
  p.copy = (num_q_heads && q_out != q) || (num_kv_heads && k_out != k);
  const bool vec =
      p.half % (interleaved ? 4 : 8) == 0 && head_dim % 8 == 0 &&
      ((p.q_stride | p.k_stride | p.q_out_stride | p.k_out_stride) & 7) == 0 &&
      ((reinterpret_cast<uintptr_t>(num_q_heads ? q : nullptr) |
        reinterpret_cast<uintptr_t>(num_kv_heads ? k : nullptr) |
        reinterpret_cast<uintptr_t>(num_q_heads ? q_out : nullptr) |
        reinterpret_cast<uintptr_t>(num_kv_heads ? k_out : nullptr)) & 15) == 0;
  p.tokens = 4;
  const int64_t ctas = (n + p.tokens - 1) / p.tokens;
  if (ctas > 0x7fffffff) return OSCAR_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(p.tokens) * p.half * sizeof(float2);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(ctas)), dim3(kRopeThreads),
                                            smem, static_cast<cudaStream_t>(stream), &attr);
  const cudaError_t e =
      interleaved ? (vec ? cudaLaunchKernelEx(&cfg, rope_kernel<true, true>, p)
                         : cudaLaunchKernelEx(&cfg, rope_kernel<true, false>, p))
                  : (vec ? cudaLaunchKernelEx(&cfg, rope_kernel<false, true>, p)
                         : cudaLaunchKernelEx(&cfg, rope_kernel<false, false>, p));
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // extern "C"
