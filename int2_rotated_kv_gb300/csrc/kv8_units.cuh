// Units of attention over the 8-bit cache: what the kernels of kv8_attention.cu and
// kv8_rows.cu share of parameters, lengths and the division of pages among CTAs.
#pragma once

#include "common.cuh"
#include "kv8_layout.cuh"

namespace oscar {

constexpr int kMaxCtas = 1024;
constexpr float kLowest = -3.402823466e38f;   // running maximum before the first logit
constexpr float kLag = 8.f;                   // the maximum is raised when passed by 2^8

// Weights w = p s_V relative to the largest of a column: outputs are sums of w code in units of
// 2^(m + k), so that a page of huge values that nothing attends to takes no bits from the others.  m is a
// logit (log2 domain) and may be large, k an offset of about log2 s_V: differences of two m are exact
// where they matter, and k is added to them, never to m.
struct Unit {
  float m, k;
};
constexpr Unit kNoUnit = {kLowest, -300.f};   // of a column that has seen nothing
// How far (m, k) lies above u, or below.
__device__ __forceinline__ float above(Unit u, float m, float k) { return (m - u.m) + (k - u.k); }
// The higher of the two.
__device__ __forceinline__ Unit higher(Unit u, float m, float k) { return above(u, m, k) > 0.f ? Unit{m, k} : u; }

// Value scales go from 2^-109 to 2^121.  Tiles of 8 columns have m the largest logit, l the sum of p in
// units of 2^m, and a factor beside p for w.  In tiles of 128 a product more for each weight is left out: the
// scale rides in the exponent, (m, k) is the unit of both, and l is the sum of w / s_V.  Therefore, there:
//   - up to kSteep m is logit + log2 s_V as one number, and k is 0;
//   - a page of zeros counts as one of scale 2^-110, below every other (kZeroLog2);
//   - l is carried times 2^-12, so that 2^25 tokens of the least scale stay below 2^128;
//   - w / s_V is lost with w where a scale lies 2^100 below another's, which takes one outside
//     [2^-64, 2^32] (is_odd): from then on 2^(logit - m - k) takes the place of a w that is 0;
//   - a change of unit by 2^x takes l times 2^(x/2) twice, as 2^x alone may underflow;
//   - 1 / l is two factors.
constexpr float kZeroLog2 = -110.f;
constexpr int kSumLog2 = -12;
constexpr float kSumUnit = 1.f / 4096.f;   // 2^kSumLog2
constexpr float kZeroScale = 7.703719777548943e-34f;   // 2^kZeroLog2
constexpr float kSteep = 1024.f;   // beyond it that one number is off by 2^-14 and more
__device__ __forceinline__ bool is_odd(float log2_scale) { return fabsf(log2_scale + 16.f) > 48.f; }

__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// Power of two that brings a bf16 magnitude (bits) to [2^7, 2^8), as its exponent.  (From 2^120 on
// it comes higher, to 65280 at most, which fp16 holds; below 2^-113 lower.  The power, its
// inverse and the factors made of it stay normal.)
__device__ __forceinline__ int scale_up(uint32_t amax) {
  return amax ? max(-112, min(120, 134 - static_cast<int>(amax >> 7))) : 0;
}
// A logit per unit of a column's q.K: the key scale times the column's factor, whose product may
// overflow where q.K is 0 all the same.
__device__ __forceinline__ float logit_factor(float scale, float fac) {
  return fminf(scale * fac, 3.402823466e38f);
}

__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// 2^x, subnormal results kept.
__device__ __forceinline__ float whole_exp2(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// 1 / l of a sum l (carried times 2^kSumLog2, perhaps subnormal), 0 for 0: the product of two.
struct Inverse {
  float a, b;
};
__device__ __forceinline__ Inverse inverse_of(float l) {
  const float up = l < 7.888609052210118e-31f ? 1.2676506002282294e30f     // 2^-100, 2^100
                   : l > 1.2676506002282294e30f ? 7.888609052210118e-31f
                                                : 1.f;
  return {l == 0.f ? 0.f : 1.f / (l * up), up * kSumUnit};
}
// Two outputs x / l, y / l.
__device__ __forceinline__ uint32_t over_sum(float x, float y, Inverse inv) {
  return pack_bf162(x * inv.a * inv.b, y * inv.a * inv.b);
}

// Two fp32 values in one operand, and arithmetic on both at once.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(lo)) | (static_cast<uint64_t>(__float_as_uint(hi)) << 32);
}
__device__ __forceinline__ float first(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float second(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// (Beside add2 not to be used where the product has to be rounded by itself: the two become one operation.)
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

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
  float* part;             // [2 * CTAs][8 * NT * (D + 4)]
};

// Floats of one partial result of 8 * NT columns: outputs, then (unit, sum, -) of each column.
template <int D, int NT>
__host__ __device__ constexpr int kv8_slot() {
  return 8 * NT * (D + 4);
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

// Tokens that the rows of a tile see: the furthest row's.  By groups of kLanes threads with
// one tile, each thread its rows, four loads in flight.
template <int NT, int kLanes>
__device__ __forceinline__ int tile_limit(const Kv8Params& p, int b, int tile, int len) {
  const int r0 = tile * 8 * NT / p.G;
  const int r1 = min(p.cols - 1, tile * 8 * NT + 8 * NT - 1) / p.G;
  int vis = 0;
#pragma unroll 1
  for (int r = r0 + (threadIdx.x & (kLanes - 1)); r <= r1; r += 4 * kLanes)
#pragma unroll
    for (int k = 0; k < 4; ++k) vis = max(vis, row_limit(p, b, min(r + k * kLanes, r1), len));
  if constexpr (kLanes > 1)
    for (int o = 1; o < kLanes; o <<= 1) vis = max(vis, __shfl_xor_sync(0xffffffffu, vis, o));
  return vis;
}

template <int NT, int kLanes>
__device__ __forceinline__ Entry make_entry(const Kv8Params& p, int e) {
  Entry t;
  t.b = e / p.tiles;
  t.tile = e - t.b * p.tiles;
  const int len = p.seq_lens[t.b];
  t.len = len >= 0 && len <= p.max_len ? len : 0;
  t.vis = p.q_pos ? tile_limit<NT, kLanes>(p, t.b, t.tile, t.len) : t.len;
  const int whole = t.len / kPage;
  t.n8 = min(whole, (t.vis + kPage - 1) / kPage);
  t.pages = max(1, t.n8 + (t.vis > whole * kPage ? 1 : 0));
  return t;
}

// By whole warps.
template <int NT>
__device__ __forceinline__ Entry entry_of(const Kv8Params& p, int e) {
  return make_entry<NT, 32>(p, e);
}

// First element of column `col` of the tile; null when the tile has fewer columns.
__device__ __forceinline__ const uint16_t* column(const Kv8Params& p, const Entry& t, int h,
                                                  int col, int D) {
  if (col >= p.cols) return nullptr;
  const int row = col / p.G, g = col - row * p.G;
  return p.q + ((static_cast<size_t>(t.b) * p.m_rows + row) * p.hq + h * p.G + g) * D;
}

// Inclusive prefix sum over the CTA's threads, and the sum of all; scratch: a word per warp.
template <int kWarps>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) v += scratch[w];
    all += scratch[w];
  }
  __syncthreads();
  return v;
}

// This CTA's equal share [at, end) of the pages of all units laid end to end, the unit
// that holds its first page, and that unit's own first page.  false: no pages.
struct Share {
  int64_t at, end, share, unit0;
  int e, h;
  Entry t;
};

// (Its loops rolled: code that a CTA runs once costs its fetches.  Not out of line: there the
// parameters are read through memory, 2% of the 65-row case.)
template <int NT, int kWarps>
__device__ __forceinline__ Share find_share(const Kv8Params& p, int min_share, bool& any) {
  // threads of an entry, for its rows' positions; entries at a time
  constexpr int kLanes = NT > 2 ? 8 : 1, kAtOnce = 32 * kWarps / kLanes;
  __shared__ int64_t scratch[kWarps];
  __shared__ Entry found;
  __shared__ int found_number;
  __shared__ int64_t found_before;
  const int own_e = threadIdx.x / kLanes;
  Share s{};
  int64_t before = 0, total = 0;
  // pass 0: the sum; pass 1: the entry that holds `at`, kAtOnce at a time (of no more
  // entries than that, with what pass 0 found)
  Entry own{};
  int64_t v = 0, incl = 0, all = 0;
  const bool few = p.entries <= kAtOnce;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
    for (int e0 = 0; e0 < p.entries; e0 += kAtOnce) {
      if (pass == 0 || !few) {
        own = make_entry<NT, kLanes>(p, min(e0 + own_e, p.entries - 1));
        v = e0 + own_e < p.entries && threadIdx.x % kLanes == 0 ? static_cast<int64_t>(own.pages) * p.hkv : 0;
        incl = block_scan<kWarps>(v, scratch, all);
      }
      if (pass == 0) {
        total += all;
      } else {
        if (s.at < before + all) {   // one thread's
          if (before + incl - v <= s.at && s.at < before + incl) {
            found = own;
            found_number = e0 + own_e;
            found_before = before + incl - v;
          }
          break;
        }
        before += all;
      }
    }
    if (pass == 0) {   // at least, and in multiples of, min_share
      const int64_t step = static_cast<int64_t>(gridDim.x) * min_share;
      s.share = max(static_cast<int64_t>(1), (total + step - 1) / step) * min_share;
      s.at = blockIdx.x * s.share;
      s.end = min(total, s.at + s.share);
      any = s.at < s.end;
      if (!any) return s;
    }
  }
  __syncthreads();
  s.e = found_number;
  s.t = found;
  // (the entry's pages are fewer than 2^31 for all heads of a cache that exists)
  s.h = static_cast<int>((s.at - found_before) / s.t.pages);
  s.unit0 = found_before + static_cast<int64_t>(s.h) * s.t.pages;
  return s;
}

// mbar_wait with the rare part out of line.
static __device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity, int32_t* status) {
  return mbar_wait(bar, parity, status);
}
__device__ __forceinline__ bool wait_copy(uint64_t* bar, uint32_t parity, int32_t* status) {
  return mbar_try_wait(bar, parity) || wait_longer(bar, parity, status);
}

// Many query columns (tiles of 128) on the tensor-memory MMAs: kv8_rows.cu.
constexpr int kRowsNT = 16;
oscar_status run_kv8_rows(const Kv8Params& p, int head_dim, bool e4m3, int64_t ctas, int min_share,
                          cudaStream_t st);

}  // namespace oscar
