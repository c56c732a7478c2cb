// Units of attention over the 8-bit cache: what the kernels of kv8_attention.cu and
// kv8_rows.cu share of parameters, lengths and the division of pages among CTAs.
#pragma once

#include "common.cuh"
#include "kv8_layout.cuh"

namespace oscar {

constexpr int kMaxCtas = 1024;
constexpr float kLowest = -3.402823466e38f;   // running maximum before the first logit
constexpr float kLag = 8.f;                   // the maximum is raised when passed by 2^8

struct Kv8Params {
  int hkv, hq, G, max_pages;
  int64_t n_pages, n_tails;
  const uint8_t* pool;
  const uint8_t* tail;
  const int32_t* page_table;
  const int32_t* tail_ids;
  int32_t* status;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* seq_lens;
  const int32_t* q_pos;    // null: one row per sequence, at its last token
  int m_rows, cols, tiles, entries, max_len;   // cols = m_rows * G; entries = batch * tiles
  int cluster;             // CTAs per unit when clusters serve units
  int team;                // warps per unit when teams of warps do
  float scale_log2;
  int4* info;              // per CTA: unit entry, KV head, parts of the unit that starts in it
  float* part;             // [2 * CTAs][8 * NT * (D + 2)]
};

// Floats of one partial result of 8 * NT columns: outputs, then (maximum, sum) pairs.
template <int D, int NT>
__host__ __device__ constexpr int kv8_slot() {
  return 8 * NT * (D + 2);
}

// A sequence's tile of query columns: pages it has to visit (at least one, so that
// a tile that sees nothing still writes its zeros).
struct Entry {
  int b, tile, len, vis, n8, pages;
};

__device__ __forceinline__ int row_limit(const Kv8Params& p, int b, int row, int len) {
  const int pos = p.q_pos[static_cast<size_t>(b) * p.m_rows + row];
  return pos >= 0 && pos < len ? pos + 1 : 0;
}

template <int NT>
__device__ __forceinline__ Entry entry_of(const Kv8Params& p, int e) {
  Entry t;
  t.b = e / p.tiles;
  t.tile = e - t.b * p.tiles;
  const int len = p.seq_lens[t.b];
  t.len = len >= 0 && len <= p.max_len ? len : 0;
  if (p.q_pos) {
    const int r0 = t.tile * 8 * NT / p.G;
    const int r1 = min(p.cols - 1, t.tile * 8 * NT + 8 * NT - 1) / p.G;
    t.vis = 0;
    for (int r = r0; r <= r1; ++r) t.vis = max(t.vis, row_limit(p, t.b, r, t.len));
  } else {
    t.vis = t.len;
  }
  const int whole = t.len / kPage;
  t.n8 = min(whole, (t.vis + kPage - 1) / kPage);
  t.pages = max(1, t.n8 + (t.vis > whole * kPage ? 1 : 0));
  return t;
}

// First element of column `col` of the tile; null when the tile has fewer columns.
__device__ __forceinline__ const uint16_t* column(const Kv8Params& p, const Entry& t, int h,
                                                  int col, int D) {
  if (col >= p.cols) return nullptr;
  const int row = col / p.G, g = col - row * p.G;
  return p.q + ((static_cast<size_t>(t.b) * p.m_rows + row) * p.hq + h * p.G + g) * D;
}

// Sum over the CTA's kWarps warps; scratch: a word for each.
template <int kWarps>
__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* scratch) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += scratch[w];
  __syncthreads();
  return total;
}

// The entry that holds page `at` of the entries laid end to end (each weighed by
// the KV heads), and the pages before it.
template <int NT, int kWarps>
__device__ void find_entry(const Kv8Params& p, int64_t at, int64_t* scratch, int& entry,
                           int64_t& before) {
  __shared__ int found;
  __shared__ int64_t found_before;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t base = 0;
  if (tid == 0) found = -1;
  __syncthreads();
  for (int e0 = 0; e0 < p.entries; e0 += 32 * kWarps) {
    const int e = e0 + tid;
    const int64_t v = e < p.entries ? static_cast<int64_t>(entry_of<NT>(p, e).pages) * p.hkv : 0;
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    int64_t off = base, all = base;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) off += scratch[w];
      all += scratch[w];
    }
    incl += off;
    if (v > 0 && incl - v <= at && at < incl) {
      found = e;
      found_before = incl - v;
    }
    __syncthreads();
    if (found >= 0) break;
    base = all;
  }
  entry = found;
  before = found_before;
}

// This CTA's equal share [at, end) of the pages of all units laid end to end, the unit
// that holds its first page, and that unit's own first page.  false: no pages.
struct Share {
  int64_t at, end, share, unit0;
  int e, h;
  Entry t;
};

template <int NT, int kWarps>
__device__ bool find_share(const Kv8Params& p, int min_share, int64_t* scratch, Share& s) {
  int64_t sum = 0, before = 0;
  if (p.entries == 1) {
    s.t = entry_of<NT>(p, 0);
    sum = s.t.pages;
  } else {
    for (int i = threadIdx.x; i < p.entries; i += 32 * kWarps) sum += entry_of<NT>(p, i).pages;
    sum = block_sum<kWarps>(sum, scratch);
  }
  const int64_t total = sum * p.hkv;
  // at least, and in multiples of, min_share
  s.share = max(static_cast<int64_t>(1), (total + static_cast<int64_t>(gridDim.x) * min_share - 1) /
                                             (static_cast<int64_t>(gridDim.x) * min_share)) * min_share;
  s.at = blockIdx.x * s.share;
  s.end = min(total, s.at + s.share);
  if (s.at >= s.end) return false;
  s.e = 0;
  if (p.entries > 1) {
    find_entry<NT, kWarps>(p, s.at, scratch, s.e, before);
    s.t = entry_of<NT>(p, s.e);
  }
  s.h = static_cast<int>((s.at - before) / s.t.pages);
  s.unit0 = before + static_cast<int64_t>(s.h) * s.t.pages;
  return true;
}

// Many query columns (tiles of 128) on the tensor-memory MMAs: kv8_rows.cu.
constexpr int kRowsNT = 16;
oscar_status run_kv8_rows(const Kv8Params& p, int head_dim, bool e4m3, int64_t ctas, int min_share,
                          cudaStream_t st);

}  // namespace oscar
