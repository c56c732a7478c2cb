// Attention over the 8-bit cache (kv8_layout.cuh): decode and several query rows
// per sequence, split over the context.
//
//   out[b][m][hq] = sum_t softmax_t(q . k_t / sqrt(d)) v_t,  t <= position of row m,
// with k_t = code * s_K(page, head), v_t = code * s_V(page, head) for tokens in
// whole pages and bf16 keys and values for the tokens of the tail.
//
// The codes go to the tensor cores as exact fp16 operands (two byte permutes per
// four int8 codes, one conversion per two e4m3 codes), keys as the A operand of
// q.K and values, transposed, as the A operand of p.V; 8 query columns (row, query
// head) fill the N dimension:
//   logit = s_K * (sum_c (u_c - 128) q_c),  the -128 sum_c q_c as the initial
//     accumulator (int8); q enters as fp16 scaled by a power of two per column,
//     which keeps all 8 bits of every bf16 within 2^-21 of the column's largest.
//   o += (p s_V) code,  p s_V rounded once to fp16 (2^-12 relative, unbiased), in a unit of
//     each column's own (kv8_units.cuh) that leaves it its
//     11 bits down to 2^-20 of the column's largest p s_V.  int8 value
//     codes lose their 128 before the MMA (one fp16 add per two codes): summed
//     with it over hundreds of pages, the accumulator's truncation of sums of
//     p s_V (code + 128) is a bias of 2e-3 of the output where values cancel.
// Softmax statistics, accumulators and the merges are fp32.  Tail tokens are exact
// in bf16 on the K side and use fp32 p on the V side.
//
// Work split, by what there is of units, each a run of pages (kv8_plan has the rule).
// A unit is (sequence, 8 query columns, KV head), or 128 columns where the estimates of
// kv8_plan find that faster (kv8_rows.cu).
//   - many short units: a team of 1, 2, 4 or 8 warps per unit.
//   - few units, moderate lengths: a thread-block cluster per unit.  Each of its CTAs
//     (16 warps, one CTA per SM) takes an equal run of the unit's pages, and the CTAs
//     merge through distributed shared memory: one launch, no workspace.
//   - else the units are laid end to end, and every CTA (8 warps, two per SM) takes an
//     equal share of the pages, found from the lengths on the device: ragged batches
//     finish together.  A CTA whose share ends inside a unit leaves a partial (at most
//     two per CTA, so the workspace does not grow with the batch); a second kernel
//     merges those units.
// Within a CTA the warps take pages in turn, each through its own ring of bulk copies,
// and merge through shared memory at a unit's end; the ring already fills for the
// next unit meanwhile.
//
// Bound by HBM: 2d + 1 bytes per token and KV head.  Measured, 8 KV heads, d = 128: 64
// sequences of 4096-8192 tokens 135 us, 5990 GB/s (shares); one of 131071 tokens 48.3 us, 5580
// GB/s (clusters of 16 for 7 heads would leave one for a second round, so 12; 96 of 152 SMs);
// one of 32768 18.8 us, 3590 GB/s, of which 5 us are the launch, the first pages and the merge.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "kv8_units.cuh"

namespace oscar {

enum Kv8Mode { kShares, kCluster, kTeams };

template <int D, Kv8Mode kMode>
struct Kv8Cfg {
  using F = Kv8Fmt<D>;
  static constexpr int kWarps = kMode == kCluster ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = kMode != kCluster ? 2 : 1;   // per SM
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kWarpRing = kStages * F::kBlock;
  static constexpr int kStride = D + 4;                     // floats per column when merging
  static constexpr int kMerge = kWarps * 8 * kStride * 4;
  static constexpr int kStat = kWarps * 8 * 4;              // one of m, k, l
  static constexpr int kSlot = kv8_slot<D, 1>();
  static constexpr int kMergeOff = kWarps * kWarpRing;
  static constexpr int kStatOff = kMergeOff + kMerge;
  static constexpr int kUnitOff = kStatOff + 3 * kStat;     // float2: units that the parts are brought to
  static constexpr int kPartOff = kUnitOff + kWarps * 8 * 8;   // a cluster's CTA: its partial
  static constexpr int kBarOff = kPartOff + (kMode == kCluster ? kSlot * 4 : 0);
  static constexpr int kBytes = kBarOff + kWarps * kStages * 8;
  static_assert(kWarpRing >= F::kTailBytes, "a warp's ring holds a tail block");
};

// The columns of one unit as a lane sees them: operands for column gid, factors and limits for
// columns 2tig and 2tig + 1.
template <int D>
struct Query {
  uint32_t b[D / 16][2];
  float fac[2];     // log2-domain logit per unit of q.code, before s_K; of the int8 codes' 2^24 it
                    // has 2^18, and s_K gets 2^6, as neither takes all without overflow
  float init[2];    // -128 sum q (int8)
  int vis[2];
  int vis_min;      // smallest over the unit's columns
};

template <int D, bool kE4m3>
__device__ __forceinline__ void load_query(const Kv8Params& p, const Entry& t, int h, int lane,
                                           Query<D>& q) {
  const int gid = lane >> 2, tig = lane & 3;
  const int col = t.tile * 8 + gid;
  const uint16_t* src = column(p, t, h, col, D);
  int vis = 0x7fffffff;
  if (src) vis = p.q_pos ? row_limit(p, t.b, col / p.G, t.len) : t.len;
  uint4 raw[D / 32];
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const uint4* s = reinterpret_cast<const uint4*>(src + 64 * j + 16 * tig);
    raw[2 * j] = src ? s[0] : make_uint4(0, 0, 0, 0);
    raw[2 * j + 1] = src ? s[1] : make_uint4(0, 0, 0, 0);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      amax = fmaxf(amax, fmaxf(fabsf(bf16_lo_value(w[x])), fabsf(bf16_hi_value(w[x]))));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // the largest magnitude goes to [2^7, 2^8)
  const int up = scale_up(__float_as_uint(amax) >> 16);
  const float mul = power_of_two(up);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // four channels: one k-step of this lane
      const float x0 = bf16_lo_value(w[2 * half]) * mul, x1 = bf16_hi_value(w[2 * half]) * mul;
      const float x2 = bf16_lo_value(w[2 * half + 1]) * mul;
      const float x3 = bf16_hi_value(w[2 * half + 1]) * mul;
      // the pairs of kv8_operands
      const uint32_t b0 = kE4m3 ? pack_half2(x0, x1) : pack_half2(x0, x2);
      const uint32_t b1 = kE4m3 ? pack_half2(x2, x3) : pack_half2(x1, x3);
      q.b[2 * i + half][0] = b0;
      q.b[2 * i + half][1] = b1;
      sum += (half_lo(b0) + half_hi(b0)) + (half_lo(b1) + half_hi(b1));
    }
  }
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  const float fac = p.scale_log2 * power_of_two(-up) * (kE4m3 ? 1.f : 262144.f);
  const float init = kE4m3 ? 0.f : sum * (-128.f / 16777216.f);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    q.fac[c] = __shfl_sync(0xffffffffu, fac, 8 * tig + 4 * c);
    q.init[c] = __shfl_sync(0xffffffffu, init, 8 * tig + 4 * c);
    q.vis[c] = __shfl_sync(0xffffffffu, vis, 8 * tig + 4 * c);
  }
  q.vis_min = __reduce_min_sync(0xffffffffu, vis);
}

// A warp's running result for its columns.  o: accumulator tiles, element
// [2i + y][r + 2x] is channel 32i + 4gid + 2y + x of column 2tig + r, in units of 2^(m + k).
// l: the sum of p = 2^(logit - m).
template <int D>
struct Running {
  float o[D / 16][4];
  float m[2], k[2], l[2];
};
// Weights w = p 2^(log2 s_V - k) reach 2^(kLag + kLift): k lies kLift below the largest p s_V when it is set.
constexpr float kLift = 6.f;

template <int D>
__device__ __forceinline__ void reset(Running<D>& s) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s.o[i][0] = s.o[i][1] = s.o[i][2] = s.o[i][3] = 0.f;
  s.m[0] = s.m[1] = kNoUnit.m;
  s.k[0] = s.k[1] = kNoUnit.k;
  s.l[0] = s.l[1] = 0.f;
}

// w and p of a tile of tokens with values of scale 2^off, p added to the sums.  lg: logits, rows gid,
// gid + 8 of the tile in the accumulator layout.  Where a logit passes its column's m by more than kLag, or
// a weight 2^(kLag + kLift), m and k are raised first: l changes with m, o with m + k.  (Both columns at
// once where there is an instruction for it: 24 columns over 32k tokens 33.2 to 32.5 us.)
template <int D>
__device__ __forceinline__ void weigh(Running<D>& s, const float (&lg)[4], float off, float (&w)[4]) {
  float e[4], up[2];   // exponents of p; of a weight's factor beside it
  bool over = false;
  const uint64_t less = two(-1.f, -1.f), m2 = two(s.m[0], s.m[1]);
  const uint64_t e0 = fma2(m2, less, two(lg[0], lg[1])), e1 = fma2(m2, less, two(lg[2], lg[3]));
  const uint64_t u2 = fma2(two(s.k[0], s.k[1]), less, two(off, off));
  e[0] = first(e0); e[1] = second(e0); e[2] = first(e1); e[3] = second(e1);
  up[0] = first(u2); up[1] = second(u2);
#pragma unroll
  for (int c = 0; c < 2; ++c) over |= fmaxf(e[c], e[2 + c]) > fminf(kLag, kLag + kLift - up[c]);
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float top = fmaxf(lg[c], lg[2 + c]);
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float m = fmaxf(top, s.m[c]), down = s.m[c] - m;
      // the unit as it is, seen from m; and what this page needs
      const float k0 = s.k[c] + down, k = fmaxf(fmaxf(k0, top - m + off - kLift), kNoUnit.k);
      s.l[c] *= fast_exp2(down);
      const float a = fast_exp2(k0 - k);
      s.m[c] = m;
      s.k[c] = k;
      e[c] = lg[c] - m;
      e[2 + c] = lg[2 + c] - m;
      up[c] = off - k;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        s.o[i][c] *= a;
        s.o[i][2 + c] *= a;
      }
    }
  }
  // (finite: it meets p of 0 where it is large)
  const uint64_t scale = two(fast_exp2(fminf(up[0], 126.f)), fast_exp2(fminf(up[1], 126.f)));
  const uint64_t p0 = two(fast_exp2(e[0]), fast_exp2(e[1])), p1 = two(fast_exp2(e[2]), fast_exp2(e[3]));
  const uint64_t l = add2(two(s.l[0], s.l[1]), add2(p0, p1)), w0 = mul2(p0, scale), w1 = mul2(p1, scale);
  s.l[0] = first(l);
  s.l[1] = second(l);
  w[0] = first(w0);
  w[1] = second(w0);
  w[2] = first(w1);
  w[3] = second(w1);
}

// One page of codes at `st`.
template <int D, bool kE4m3>
__device__ __forceinline__ void page(const uint8_t* st, int page0, int lane, const Query<D>& q,
                                     Running<D>& s) {
  using F = Kv8Fmt<D>;
  const int gid = lane >> 2;
  const uint4* kb = reinterpret_cast<const uint4*>(st);
  float lg[4];
  lg[0] = lg[2] = q.init[0];
  lg[1] = lg[3] = q.init[1];
  const float2 sc = *reinterpret_cast<const float2*>(st + F::kScales);
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const uint4 k0 = kb[(2 * j) * 32 + lane], k1 = kb[(2 * j + 1) * 32 + lane];
    const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t a0, a1, a2, a3;
      kv8_operands<kE4m3>(w0[w], a0, a2);
      kv8_operands<kE4m3>(w1[w], a1, a3);
      mma_f16(lg, a0, a1, a2, a3, q.b[4 * j + w][0], q.b[4 * j + w][1]);
    }
  }
  const float sk = kE4m3 ? sc.x : sc.x * 64.f;
  const float f0 = logit_factor(sk, q.fac[0]), f1 = logit_factor(sk, q.fac[1]);
  // (rounded by themselves, not on the way to a difference, so that equal logits stay equal)
#pragma unroll
  for (int r = 0; r < 4; ++r) lg[r] = __fmul_rn(lg[r], r & 1 ? f1 : f0);
  if (page0 + kPage > q.vis_min) {
    const int t = page0 + 2 * gid;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (t >= q.vis[c]) lg[c] = -INFINITY;
      if (t + 1 >= q.vis[c]) lg[2 + c] = -INFINITY;
    }
  }
  float w[4];
  weigh<D>(s, lg, fast_log2(sc.y), w);   // (a page of zeros: log2 0 = -inf, weights of 0)
  // rows gid of the logits were tokens 2 gid and 2 gid + 1: transposed, the two
  // registers hold tokens (4tig, 4tig + 2) and (4tig + 1, 4tig + 3) of column gid
  uint32_t b0 = movmatrix_trans(pack_half2(w[0], w[1]));
  uint32_t b1 = movmatrix_trans(pack_half2(w[2], w[3]));
  if constexpr (kE4m3) {   // pairs (4tig, 4tig + 1), (4tig + 2, 4tig + 3)
    const uint32_t lo = __byte_perm(b0, b1, 0x5410);
    b1 = __byte_perm(b0, b1, 0x7632);
    b0 = lo;
  }
  const uint4* vb = reinterpret_cast<const uint4*>(st + F::kCodes);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const uint4 v = vb[i * 32 + lane];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      uint32_t a0, a1, a2, a3;
      kv8_signed_operands<kE4m3>(w[2 * y], a0, a2);
      kv8_signed_operands<kE4m3>(w[2 * y + 1], a1, a3);
      mma_f16(s.o[2 * i + y], a0, a1, a2, a3, b0, b1);
    }
  }
}

// Takes the int8 codes' 2^-24 off the accumulators.
template <int D, bool kE4m3>
__device__ __forceinline__ void unscale(Running<D>& s) {
  if constexpr (!kE4m3) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) s.o[i][r] *= 16777216.f;
  }
}

// The largest finite magnitude of a pair of bf16, or `top`.
__device__ __forceinline__ uint32_t finite_max(uint32_t top, uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  return max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
}
__device__ __forceinline__ uint32_t bf16_times(uint32_t w, __nv_bfloat162 x) {
  const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), x);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// The tail: n bf16 tokens from position page0 at `st`; unscaled accumulators.  q.K in bf16
// (exact products).  Its values enter times a power of two that brings the largest finite one to
// [2^7, 2^8), as if they were codes of the scale that undoes it.  w.V in bf16 with w as a pair of
// bf16 (2^-17); when a value is not finite, or a column does not see all n tokens, in
// fp32 on the CUDA cores instead, which keeps a NaN or an infinity of a token out of
// the rows that do not see it.
template <int D>
__device__ void tail_tokens(const Kv8Params& p, const Entry& t, int h, const uint8_t* st, int page0,
                            int n, int lane, const Query<D>& q, Running<D>& s) {
  using F = Kv8Fmt<D>;
  const int gid = lane >> 2, tig = lane & 3;
  const uint4* kb = reinterpret_cast<const uint4*>(st);
  float lg[4] = {};
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    const int c0 = ((2 * j) * 32 + lane) * 2, c1 = ((2 * j + 1) * 32 + lane) * 2;
#pragma unroll
    for (int x = 0; x < 2; ++x) {   // 8 channels: two k-steps
      const uint4 k0 = kb[c0 + x], k1 = kb[c1 + x];
      const uint16_t* src = column(p, t, h, t.tile * 8 + gid, D);
      const uint4 qv = src ? *reinterpret_cast<const uint4*>(src + 64 * j + 16 * tig + 8 * x)
                           : make_uint4(0, 0, 0, 0);
      mma_bf16(lg, k0.x, k1.x, k0.y, k1.y, qv.x, qv.y);
      mma_bf16(lg, k0.z, k1.z, k0.w, k1.w, qv.z, qv.w);
    }
  }
  const uint4* vb = kb + 2 * D;   // 16 * d keys before them
  // tokens 4tig, 4tig + 1 and 4tig + 2, 4tig + 3 of a channel's words, where there are any
  const int have = n - 4 * tig;
  const uint32_t m01 = (have > 0 ? 0xffffu : 0u) | (have > 1 ? 0xffff0000u : 0u);
  const uint32_t m23 = (have > 2 ? 0xffffu : 0u) | (have > 3 ? 0xffff0000u : 0u);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint4 v = vb[((i >> 1) * 32 + lane) * 2 + (i & 1)];
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & m01 & 0x7fff7fffu, v.y & m23 & 0x7fff7fffu),
                                 __vmaxu2(v.z & m01 & 0x7fff7fffu, v.w & m23 & 0x7fff7fffu)));
  }
  uint32_t finite = max(top & 0xffffu, top >> 16);
  const bool plain = __all_sync(0xffffffffu, finite < 0x7f80u);
  if (!plain) {
    finite = 0;
#pragma unroll 1
    for (int i = 0; i < D / 16; ++i) {
      const uint4 v = vb[((i >> 1) * 32 + lane) * 2 + (i & 1)];
      finite = finite_max(finite_max(finite, v.x & m01), v.y & m23);
      finite = finite_max(finite_max(finite, v.z & m01), v.w & m23);
    }
  }
  finite = __reduce_max_sync(0xffffffffu, finite);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int seen = min(n, q.vis[c] - page0);   // tokens of the tail this column sees
    lg[c] = 2 * gid < seen ? __fmul_rn(lg[c], p.scale_log2) : -INFINITY;
    lg[2 + c] = 2 * gid + 1 < seen ? __fmul_rn(lg[2 + c], p.scale_log2) : -INFINITY;
  }
  const int up = scale_up(finite);
  const float mul = power_of_two(up);
  float w[4];
  // (values that are all zeros need no weight; beside a NaN or an infinity, any)
  weigh<D>(s, lg, finite || !plain ? static_cast<float>(-up) : -INFINITY, w);
  if (q.vis_min >= page0 + n && plain) {
    const __nv_bfloat162 mul2 = __float2bfloat162_rn(mul);
    uint32_t bh[2], bl[2];
    const uint32_t h0 = pack_bf162(w[0], w[1]), h1 = pack_bf162(w[2], w[3]);
    const uint32_t l0 = pack_bf162(w[0] - bf16_lo_value(h0), w[1] - bf16_hi_value(h0));
    const uint32_t l1 = pack_bf162(w[2] - bf16_lo_value(h1), w[3] - bf16_hi_value(h1));
    const uint32_t t0 = movmatrix_trans(h0), t1 = movmatrix_trans(h1);
    const uint32_t u0 = movmatrix_trans(l0), u1 = movmatrix_trans(l1);
    bh[0] = __byte_perm(t0, t1, 0x5410);
    bh[1] = __byte_perm(t0, t1, 0x7632);
    bl[0] = __byte_perm(u0, u1, 0x5410);
    bl[1] = __byte_perm(u0, u1, 0x7632);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint4 v = vb[((i >> 1) * 32 + lane) * 2 + (i & 1)];
      // slots without a token may hold anything
      v.x = bf16_times(v.x & m01, mul2);
      v.y = bf16_times(v.y & m23, mul2);
      v.z = bf16_times(v.z & m01, mul2);
      v.w = bf16_times(v.w & m23, mul2);
      mma_bf16(s.o[i], v.x, v.z, v.y, v.w, bh[0], bh[1]);
      mma_bf16(s.o[i], v.x, v.z, v.y, v.w, bl[0], bl[1]);
    }
    return;
  }
  const uint16_t* ve = reinterpret_cast<const uint16_t*>(st) + F::kTailHalf;
  for (int i = 0; i < n; ++i) {
    float v[D / 16][2];
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {   // the lane's channels 32 (c/4) + 4 gid + c%4
      const int chunk = kv8_value_chunk(i >> 2, (c >> 2) * 8 + gid);
      v[c >> 1][c & 1] = bf16_to_float(ve[chunk * 16 + 4 * (c & 3) + (i & 3)]) * mul;
    }
    const float w0 = __shfl_sync(0xffffffffu, (i & 1) ? w[2] : w[0], 4 * (i >> 1) + tig);
    const float w1 = __shfl_sync(0xffffffffu, (i & 1) ? w[3] : w[1], 4 * (i >> 1) + tig);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      if (w0 != 0.f) {
        s.o[k][0] = fmaf(w0, v[k][0], s.o[k][0]);
        s.o[k][2] = fmaf(w0, v[k][1], s.o[k][2]);
      }
      if (w1 != 0.f) {
        s.o[k][1] = fmaf(w1, v[k][0], s.o[k][1]);
        s.o[k][3] = fmaf(w1, v[k][1], s.o[k][3]);
      }
    }
  }
}

// A warp's ring of page copies: n_in issued, n_out consumed since the kernel's start, so
// the phases run on from unit to unit.  A tail block takes the whole ring (and one
// barrier's turn), so it comes when the pages before it have been consumed.
struct Ring {
  uint8_t* base;
  uint64_t* bars;
  uint32_t n_in, n_out, shown;   // shown: bit per stage, the id was valid
  int next_id;
  bool alive;                    // false after a copy that did not arrive in time
  bool tail_issued;
};

template <typename C>
__device__ __forceinline__ void copy_in(const Kv8Params& p, bool ok, const uint8_t* src, int bytes,
                                        uint8_t* dst, int lane, Ring& r) {
  const int s = r.n_in % C::kStages;
  r.shown = (r.shown & ~(1u << s)) | (static_cast<uint32_t>(ok) << s);
  if (lane == 0) {
    if (!ok && p.status) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
    mbar_arrive_expect_tx(r.bars + s, bytes);
    bulk_g2s(dst, src, bytes, r.bars + s);
  }
  ++r.n_in;
}

// The copy of page pg (a refused id copies page 0, which is then not looked at); `step`
// pages on is the warp's next.
template <typename C>
__device__ __forceinline__ void issue(const Kv8Params& p, const Entry& t, int h, int pg, int end,
                                      int step, int lane, Ring& r) {
  const bool ok = r.next_id >= 0 && r.next_id < p.n_pages;
  const int64_t block = static_cast<int64_t>(ok ? r.next_id : 0) * p.hkv + h;
  copy_in<C>(p, ok, p.pool + block * C::F::kBlock, C::F::kBlock,
             r.base + r.n_in % C::kStages * C::F::kBlock, lane, r);
  if (pg + step < end) r.next_id = p.page_table[static_cast<size_t>(t.b) * p.max_pages + pg + step];
}

template <typename C>
__device__ __forceinline__ void issue_tail(const Kv8Params& p, const Entry& t, int h, int lane, Ring& r) {
  const int64_t id = p.tail_ids ? p.tail_ids[t.b] : t.b;
  const bool ok = id >= 0 && id < p.n_tails;
  copy_in<C>(p, ok, p.tail + ((ok ? id : 0) * p.hkv + h) * C::F::kTailBytes, C::F::kTailBytes, r.base,
             lane, r);
  r.tail_issued = true;
}

// Waits for the oldest copy; false when it did not come in time, with no copy left in flight.
template <typename C>
__device__ __forceinline__ bool copied(const Kv8Params& p, Ring& r, int& s) {
  s = r.n_out % C::kStages;
  const bool got = mbar_wait(r.bars + s, (r.n_out / C::kStages) & 1, p.status);
  ++r.n_out;
  if (__all_sync(0xffffffffu, got)) return true;
  for (; r.n_out < r.n_in; ++r.n_out)
    wait_longer(r.bars + r.n_out % C::kStages, (r.n_out / C::kStages) & 1, p.status);
  r.alive = false;
  return false;
}

// A warp's part of pages [p0, p1) of a unit: pages first, first + step, ... below end, and
// the tail if it is this warp's.
struct Part {
  int first, end;
  bool tail;
};

__device__ __forceinline__ Part part_of(const Entry& t, int p0, int p1, int warp, int step) {
  Part a;
  a.first = p0 + warp;
  a.end = min(p1, t.n8);
  a.tail = p1 > t.n8 && t.vis > t.len / kPage * kPage && warp == (t.n8 - p0) % step;
  return a;
}

// Starts the first copies of a warp's part (its ring is empty).
template <typename C>
__device__ __forceinline__ void start_part(const Kv8Params& p, const Entry& t, int h, const Part& a,
                                           int step, int lane, Ring& r) {
  r.tail_issued = false;
  if (!r.alive) return;
  if (a.first < a.end) {
    r.next_id = p.page_table[static_cast<size_t>(t.b) * p.max_pages + a.first];
#pragma unroll
    for (int i = 0; i < C::kStages; ++i)
      if (a.first + i * step < a.end) issue<C>(p, t, h, a.first + i * step, a.end, step, lane, r);
  } else if (a.tail) {
    issue_tail<C>(p, t, h, lane, r);
  }
}

// What outputs in units of 2^(u.m + u.k) are times, and sums of p in units of 2^u.m, to be the result: 0 for
// a row that sees nothing (l = 0).
__device__ __forceinline__ float output_factor(float k, float l) { return l == 0.f ? 0.f : fast_exp2(k) / l; }

// Channels ch .. ch + 3 of an output row.
__device__ __forceinline__ void store_row(const Kv8Params& p, int b, int h, int gcol, int ch, int D,
                                          float4 o, float f) {
  const int row = gcol / p.G, g = gcol - row * p.G;
  uint16_t* dst = p.out + ((static_cast<size_t>(b) * p.m_rows + row) * p.hq + h * p.G + g) * D + ch;
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(pack_bf162(o.x * f, o.y * f), pack_bf162(o.z * f, o.w * f));
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;\n" ::: "memory");
}

// Address of this CTA's shared-memory word `p` in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_address(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a));
  return v;
}

// Merges the partials of a cluster's CTAs (8 columns in `slot` of each; stats: room for 8 float4 of each);
// every CTA writes its share of the unit's outputs.
template <int D>
__device__ __forceinline__ void merge_cluster(const Kv8Params& p, const Entry& t, int h,
                                              const float* slot, float4* stats) {
  cluster_sync();
  const int n = p.cluster, rank = blockIdx.x % n;
  if (threadIdx.x < 8 * n)
    stats[threadIdx.x] = cluster_load4(cluster_address(slot + 8 * D + 4 * (threadIdx.x & 7), threadIdx.x >> 3));
  __syncthreads();
  const int per = (8 * D / 4 + n - 1) / n;      // float4 of each CTA
  const int i = rank * per + threadIdx.x;
  if (threadIdx.x < per && i < 8 * D / 4) {
    const int col = i / (D / 4), ch = 4 * (i % (D / 4)), gcol = t.tile * 8 + col;
    if (gcol < p.cols) {
      float m = kLowest, k = kLowest, l = 0.f;
      for (int r = 0; r < n; ++r) m = fmaxf(m, stats[8 * r + col].x);
      for (int r = 0; r < n; ++r) k = fmaxf(k, (stats[8 * r + col].x - m) + stats[8 * r + col].y);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int r = 0; r < n; ++r) {
        const float4 part = stats[8 * r + col];
        const float4 x = cluster_load4(cluster_address(slot + col * D + ch, r));
        const float down = part.x - m, a = fast_exp2(down + part.y - k);
        l = fmaf(fast_exp2(down), part.z, l);
        o.x = fmaf(a, x.x, o.x); o.y = fmaf(a, x.y, o.y);
        o.z = fmaf(a, x.z, o.z); o.w = fmaf(a, x.w, o.w);
      }
      store_row(p, t.b, h, gcol, ch, D, o, output_factor(k, l));
    }
  }
  cluster_sync();   // no CTA leaves while its shared memory is read
}

// A barrier of the `team` warps that serve a unit (teams: barrier 1 + number of the team).
template <Kv8Mode kMode>
__device__ __forceinline__ void team_sync(int team, int number) {
  if constexpr (kMode != kTeams) {
    __syncthreads();
  } else if (team == 1) {
    __syncwarp();
  } else {
    asm volatile("bar.sync %0, %1;\n" ::"r"(1 + number), "r"(32 * team) : "memory");
  }
}

template <int D, bool kE4m3, Kv8Mode kMode>
__global__ void __launch_bounds__((Kv8Cfg<D, kMode>::kThreads), (Kv8Cfg<D, kMode>::kCtas))
kv8_attention_kernel(const __grid_constant__ Kv8Params p, int min_share) {
  using C = Kv8Cfg<D, kMode>;
  constexpr int kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  // the warps of a unit (all, or a team of them) and this one's place among them
  const int team = kMode == kTeams ? p.team : kWarps;
  const int number = kMode == kTeams ? (tid >> 5) / team : 0;
  const int warp = (tid >> 5) - number * team;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  float* sm_m = reinterpret_cast<float*>(smem + C::kStatOff) + number * team * 8;
  float* sm_k = sm_m + kWarps * 8;
  float* sm_l = sm_k + kWarps * 8;
  float2* sm_unit = reinterpret_cast<float2*>(smem + C::kUnitOff) + number * 8;
  float* merge = reinterpret_cast<float*>(smem + C::kMergeOff) + number * team * 8 * C::kStride;
  if (tid < kWarps * C::kStages) mbar_init(bars + tid, 1);
  fence_mbar_init();
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  // this team's pages [at, end) of all units laid end to end, and its first unit
  int e = 0, h = 0;
  int64_t at = 0, end = 0, share = 0, unit0 = 0;   // unit0: first page of the current unit
  Entry t;
  if constexpr (kMode == kTeams) {   // a whole unit
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kWarps / team) + number;
    if (unit >= static_cast<int64_t>(p.entries) * p.hkv) return;
    e = static_cast<int>(unit / p.hkv);
    h = static_cast<int>(unit - static_cast<int64_t>(e) * p.hkv);
    t = entry_of<1>(p, e);
    end = t.pages;
  } else if constexpr (kMode == kCluster) {   // this CTA's run of the cluster's unit
    const int unit = blockIdx.x / p.cluster, rank = blockIdx.x - unit * p.cluster;
    e = unit / p.hkv;
    h = unit - e * p.hkv;
    t = entry_of<1>(p, e);
    at = static_cast<int64_t>(t.pages) * rank / p.cluster;
    end = static_cast<int64_t>(t.pages) * (rank + 1) / p.cluster;
  } else {
    bool any;
    const Share sh = find_share<1, kWarps>(p, min_share, any);
    if (!any) {
      if (tid == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    at = sh.at;
    end = sh.end;
    share = sh.share;
    unit0 = sh.unit0;
    e = sh.e;
    h = sh.h;
    t = sh.t;
  }

  Ring ring{smem + (tid >> 5) * C::kWarpRing, bars + (tid >> 5) * C::kStages, 0, 0, 0, 0, true, false};
  int4 owned = make_int4(0, 0, 0, 0);
  int p0 = static_cast<int>(at - unit0);
  int p1 = static_cast<int>(min(static_cast<int64_t>(t.pages), end - unit0));
  Part mine = part_of(t, p0, p1, warp, team);
  start_part<C>(p, t, h, mine, team, lane, ring);

  for (;;) {
    Query<D> q;
    load_query<D, kE4m3>(p, t, h, lane, q);
    Running<D> s;
    reset<D>(s);
    if (p0 == 0 && h == 0 && t.tile == 0 && warp == 0 && lane == 0 && p.status) {
      const int len = p.seq_lens[t.b];
      if (len < 0 || len > p.max_len) atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
    }
    if (p.q_pos && p0 == 0 && h == 0 && warp == 0 && lane < 8 && p.status) {
      const int row = (t.tile * 8 + lane) / p.G;
      if (row < p.m_rows && p.q_pos[static_cast<size_t>(t.b) * p.m_rows + row] >= t.len)
        atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
    }
    for (int pg = mine.first; pg < mine.end && ring.alive; pg += team) {
      int st;
      if (!copied<C>(p, ring, st)) break;
      // (a refused id's stands for nothing, whatever it holds)
      if ((ring.shown >> st) & 1u) page<D, kE4m3>(ring.base + st * C::F::kBlock, pg * kPage, lane, q, s);
      __syncwarp();
      if (pg + C::kStages * team < mine.end)
        issue<C>(p, t, h, pg + C::kStages * team, mine.end, team, lane, ring);
    }
    unscale<D, kE4m3>(s);
    if (mine.tail && ring.alive) {
      if (!ring.tail_issued) issue_tail<C>(p, t, h, lane, ring);
      int st;
      if (copied<C>(p, ring, st) && ((ring.shown >> st) & 1u))
        tail_tokens<D>(p, t, h, ring.base, t.len / kPage * kPage, t.len % kPage, lane, q, s);
      __syncwarp();
    }

    // the next unit of this CTA: its copies start before this one is merged
    const Entry tc = t;
    const int hc = h, c0 = p0, c1 = p1;
    const int64_t u0 = unit0;
    const bool more = kMode == kShares && u0 + c1 < end;
    if (more) {
      unit0 = u0 + tc.pages;
      if (++h == p.hkv) {
        h = 0;
        t = entry_of<1>(p, ++e);
      }
      p0 = 0;
      p1 = static_cast<int>(min(static_cast<int64_t>(t.pages), end - unit0));
      mine = part_of(t, p0, p1, warp, team);
      start_part<C>(p, t, h, mine, team, lane, ring);
    }

    if (gid == 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sm_m[warp * 8 + 2 * tig + c] = s.m[c];
        sm_k[warp * 8 + 2 * tig + c] = s.k[c];
      }
    }
    team_sync<kMode>(team, number);
    const bool complete = c0 == 0 && c1 == tc.pages;
    float* slot = kMode == kCluster
        ? reinterpret_cast<float*>(smem + C::kPartOff)
        : p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * C::kSlot;
    // the parts of a column in the unit of the largest m, and the k with which it lies as high as the highest
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 2 * tig + c;
      float m = kLowest, k = kLowest;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (kMode != kTeams || w < team) m = fmaxf(m, sm_m[w * 8 + col]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (kMode != kTeams || w < team) k = fmaxf(k, (sm_m[w * 8 + col] - m) + sm_k[w * 8 + col]);
      const float down = s.m[c] - m, a = fast_exp2(down + s.k[c] - k);
      float l = s.l[c] * fast_exp2(down);
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (gid == 0) sm_l[warp * 8 + col] = l;
      if (warp == 0 && gid == 0) sm_unit[col] = make_float2(m, k);
      float* dst = merge + (warp * 8 + col) * C::kStride + 4 * gid;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        *reinterpret_cast<float4*>(dst + 32 * i) =
            make_float4(s.o[2 * i][c] * a, s.o[2 * i][2 + c] * a,
                        s.o[2 * i + 1][c] * a, s.o[2 * i + 1][2 + c] * a);
    }
    team_sync<kMode>(team, number);
    for (int i = warp * 32 + lane; i < 8 * D / 4; i += 32 * team) {
      const int col = i / (D / 4), ch = 4 * (i % (D / 4));
      const int gcol = tc.tile * 8 + col;
      if (kMode != kCluster && gcol >= p.cols) continue;
      const float2 unit = sm_unit[col];
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (kMode == kTeams && w >= team) break;
        l += sm_l[w * 8 + col];
        const float4 x = *reinterpret_cast<const float4*>(merge + (w * 8 + col) * C::kStride + ch);
        o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
      }
      if (kMode != kCluster && (kMode == kTeams || complete)) {
        store_row(p, tc.b, hc, gcol, ch, D, o, output_factor(unit.y, l));
      } else {
        *reinterpret_cast<float4*>(slot + col * D + ch) = o;
        if (ch == 0)
          *reinterpret_cast<float4*>(slot + 8 * D + 4 * col) = make_float4(unit.x, unit.y, l, 0.f);
      }
    }
    if (kMode != kTeams) __syncthreads();   // before the buffers are written again
    if constexpr (kMode == kCluster) {
      merge_cluster<D>(p, tc, hc, slot, reinterpret_cast<float4*>(merge));
      return;
    }
    if constexpr (kMode == kTeams) return;
    if (!complete && c0 == 0)   // the unit goes on in the next CTAs: they hold its other parts
      owned = make_int4(e, hc, static_cast<int>((u0 + tc.pages - 1) / share) - blockIdx.x + 1, 0);
    if (!more) break;
  }
  if (tid == 0) p.info[blockIdx.x] = owned;
}

// Merges the units that lie in several CTAs.  Block: (CTA in which the unit starts, columns);
// kSplit warps share the parts of a column, a lane has D / 32 channels.
template <int D>
__global__ void __launch_bounds__(256) kv8_merge_kernel(const __grid_constant__ Kv8Params p) {
  constexpr int kSplit = 4;   // warps of a column: few columns, with many parts each
  constexpr int kSlot = kv8_slot<D, 1>(), kPer = D / 32;
  __shared__ float partial[8][D];
  pdl_wait();
  pdl_trigger();
  const int4 own = p.info[blockIdx.x];
  const int n = own.z;
  if (n == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = warp % kSplit;
  const int b = own.x / p.tiles, tile = own.x - b * p.tiles;
  const int col = blockIdx.y * (8 / kSplit) + warp / kSplit, gcol = tile * 8 + col;
  const bool live = col < 8 && gcol < p.cols;
  float acc[kPer] = {};
  float m = kLowest, k = kLowest, l = 0.f;
  if (live) {
    // part 0: the CTA's own second slot; part j: the first slot of the j-th CTA after it
    auto slot = [&](int j) {
      return p.part + (2 * (blockIdx.x + static_cast<size_t>(j)) + (j == 0 ? 1 : 0)) * kSlot;
    };
    auto stats = [&](int j) {   // unit and sum of part j
      return j < n ? *reinterpret_cast<const float4*>(slot(j) + 8 * D + 4 * col)
                   : make_float4(kNoUnit.m, kNoUnit.k, 0.f, 0.f);
    };
    for (int j = lane; j < n; j += 32) m = fmaxf(m, stats(j).x);
    m = warp_max(m);
    for (int j = lane; j < n; j += 32) {
      const float4 part = stats(j);
      k = fmaxf(k, (part.x - m) + part.y);
    }
    k = warp_max(k);
    for (int j0 = 0; j0 < n; j0 += 32) {
      const float4 part = stats(j0 + lane);
      const float down = part.x - m, w = fast_exp2(down + part.y - k);
      l = fmaf(fast_exp2(down), part.z, l);
      const int here = min(32, n - j0);
#pragma unroll 8
      for (int j = sub; j < here; j += kSplit) {
        const float a = __shfl_sync(0xffffffffu, w, j);
        const float* x = slot(j0 + j) + col * D + kPer * lane;
        if constexpr (kPer == 4) {
          const float4 v = *reinterpret_cast<const float4*>(x);
          acc[0] = fmaf(a, v.x, acc[0]); acc[1] = fmaf(a, v.y, acc[1]);
          acc[2] = fmaf(a, v.z, acc[2]); acc[3] = fmaf(a, v.w, acc[3]);
        } else {
          const float2 v = *reinterpret_cast<const float2*>(x);
          acc[0] = fmaf(a, v.x, acc[0]); acc[1] = fmaf(a, v.y, acc[1]);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) partial[warp][kPer * lane + k] = acc[k];
  __syncthreads();
  if (sub != 0) return;
#pragma unroll
  for (int s = 1; s < kSplit; ++s)
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] += partial[warp + s][kPer * lane + k];
  if (!live) return;
  const float f = output_factor(k, l);
  const int row = gcol / p.G, g = gcol - row * p.G;
  uint32_t* dst = reinterpret_cast<uint32_t*>(
      p.out + ((static_cast<size_t>(b) * p.m_rows + row) * p.hq + own.y * p.G + g) * D + kPer * lane);
#pragma unroll
  for (int k = 0; k < kPer; k += 2) dst[k / 2] = pack_bf162(acc[k] * f, acc[k + 1] * f);
}

// The same for tiles of 128 columns, whose partial results lie by fours of channels, 128 columns
// each: a lane per column, a warp per 8 channels, four parts in flight (eight: 2 us more where a
// unit has few).
template <int D>
__global__ void __launch_bounds__(4 * D) kv8_merge_rows_kernel(const __grid_constant__ Kv8Params p) {
  constexpr int kSlot = kv8_slot<D, kRowsNT>(), kFlight = 4;
  pdl_wait();
  pdl_trigger();
  const int4 own = p.info[blockIdx.x];
  const int n = own.z;
  if (n == 0) return;
  const int ch = 8 * (threadIdx.x >> 5), col = 32 * blockIdx.y + (threadIdx.x & 31);
  const int b = own.x / p.tiles, tile = own.x - b * p.tiles, gcol = tile * 128 + col;
  if (gcol >= p.cols) return;
  float acc[8] = {};
  Unit u = kNoUnit;
  float l = 0.f;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += kFlight) {
    float4 part[kFlight];
    float4 v[kFlight][2];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      // part 0: the CTA's own second slot; part j: the first slot of the j-th CTA after it
      const int i = j0 + j;
      part[j] = make_float4(kNoUnit.m, kNoUnit.k, 0.f, 0.f);
      v[j][0] = v[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i >= n) continue;
      const float* slot = p.part + (2 * (blockIdx.x + static_cast<size_t>(i)) + (i == 0 ? 1 : 0)) * kSlot;
      part[j] = *reinterpret_cast<const float4*>(slot + 128 * D + 4 * col);
      v[j][0] = *reinterpret_cast<const float4*>(slot + 128 * ch + 4 * col);
      v[j][1] = *reinterpret_cast<const float4*>(slot + 128 * ch + 512 + 4 * col);
    }
    float m = u.m, k = kLowest;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) m = fmaxf(m, part[j].x);
    k = (u.m - m) + u.k;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) k = fmaxf(k, (part[j].x - m) + part[j].y);
    const float shift = fast_exp2(0.5f * ((u.m - m) + u.k - k)), old = shift * shift;
    u = {m, k};
    l = l * shift * shift;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= old;
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const float half = fast_exp2(0.5f * ((part[j].x - m) + part[j].y - k)), w = half * half;
      l = fmaf(half * part[j].z, half, l);
      acc[0] = fmaf(w, v[j][0].x, acc[0]);
      acc[1] = fmaf(w, v[j][0].y, acc[1]);
      acc[2] = fmaf(w, v[j][0].z, acc[2]);
      acc[3] = fmaf(w, v[j][0].w, acc[3]);
      acc[4] = fmaf(w, v[j][1].x, acc[4]);
      acc[5] = fmaf(w, v[j][1].y, acc[5]);
      acc[6] = fmaf(w, v[j][1].z, acc[6]);
      acc[7] = fmaf(w, v[j][1].w, acc[7]);
    }
  }
  const Inverse inv = inverse_of(l);
  const int row = gcol / p.G, g = gcol - row * p.G;
  *reinterpret_cast<uint4*>(p.out + ((static_cast<size_t>(b) * p.m_rows + row) * p.hq + own.y * p.G + g) * D + ch) =
      make_uint4(over_sum(acc[0], acc[1], inv), over_sum(acc[2], acc[3], inv),
                 over_sum(acc[4], acc[5], inv), over_sum(acc[6], acc[7], inv));
}

template <typename Kern, typename... Args>
cudaError_t launch_kv8(Kern kernel, int cluster, dim3 grid, int threads, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Pages of a CTA's share, at least and a multiple of: one per warp, or a tile of 128 tokens.
// (16: 64 long sequences 133.3 us for 134.3, 36 columns over 40 sequences 83.6 for 82.3; 32: 87.9.)
constexpr int kMinShare = 8;
constexpr int kMaxCluster = 16;
constexpr int kTeamPages = 128;

// How many clusters of 1 .. 16 CTAs (one per SM) the current device holds at once;
// a GPC's SMs bound them (a GB300: 7 of 16, 8 of 12, 15 of 9, 36 of 4, 152 of 1).
struct ClusterSizes {
  int active[kMaxCluster + 1];
};

// (The kernel for d = 128 stands for all: every cluster kernel fills an SM.)
ClusterSizes count_clusters() {
  using C = Kv8Cfg<128, kCluster>;
  const auto kernel = kv8_attention_kernel<128, false, kCluster>;
  ClusterSizes s{};
  if (!oscar_host::allow_smem(reinterpret_cast<const void*>(kernel), C::kBytes, true)) return s;
  for (int c = 1; c <= kMaxCluster; ++c) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(c);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(c));
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&s.active[c], kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      s.active[c] = 0;
    }
  }
  return s;
}

// Counted once per device.  (Threads that are the first at once all count, to the same end.)
ClusterSizes cluster_sizes() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][kMaxCluster + 1];   // [0]: whether the others are
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return {};
  if (dev >= kDevices) return count_clusters();
  ClusterSizes s{};
  if (known[dev][0].load(std::memory_order_acquire)) {
    for (int c = 1; c <= kMaxCluster; ++c) s.active[c] = known[dev][c].load(std::memory_order_relaxed);
    return s;
  }
  s = count_clusters();
  for (int c = 1; c <= kMaxCluster; ++c) known[dev][c].store(s.active[c], std::memory_order_relaxed);
  known[dev][0].store(1, std::memory_order_release);
  return s;
}

struct Kv8Plan {
  bool rows;           // tiles of 128 columns (kv8_rows.cu), else of 8
  int cluster, team;   // cluster > 0: CTAs per unit; team > 0: warps per unit
  int64_t tiles, entries, ctas;
  size_t info, total;   // workspace bytes: the CTAs' records, all
  size_t most;          // no call of fewer sequences, rows or tokens takes more than this
};

// CTAs that share the pages of `units`, and the workspace bytes of their records and parts.
inline int64_t share_ctas(bool rows, int64_t units, int64_t pages, int64_t sms) {
  return std::min(std::min<int64_t>(kMaxCtas, rows ? sms : 2 * sms), (units * pages + kMinShare - 1) / kMinShare);
}
inline size_t record_bytes(int64_t ctas) { return (static_cast<size_t>(ctas) * sizeof(int4) + 255) / 256 * 256; }
inline size_t share_bytes(bool rows, int d, int64_t ctas) {
  return record_bytes(ctas) + static_cast<size_t>(ctas) * 2 * (rows ? 128 : 8) * (d + 4) * sizeof(float);
}

// Several sequences are taken as three quarters of the longest: the host does not know the
// lengths.
inline double visited(int64_t batch, int64_t units, int64_t pages) {
  return (batch > 1 ? 0.75 : 1.0) * static_cast<double>(units) * static_cast<double>(pages);
}

// Estimates in us.  Tiles of 8 columns: shares run at the memory's rate, 0.00064 us a page over
// all units (d = 128), and cost a second kernel and longer first and last waves, 6 us; a
// cluster's CTA streams its pages at 0.06 us each.
inline double shares_us(int d, int64_t batch, int64_t units, int64_t pages) {
  return 6.0 + (0.00036 + 0.00028 / 128 * d) * visited(batch, units, pages);
}
inline double cluster_us(int d, int64_t pages, int c) {
  return (0.04 + 0.02 / 128 * d) * static_cast<double>(pages) / c;
}

// Tiles of 128: a start of 24 us (18 for d = 64), 0.08 us for each unit, 0.15 us for each of
// the CTAs that a unit is spread over, whose parts are merged, and 0.001 us a page.  Measured,
// tiles of 8 against tiles of 128, in us (int8): d = 128, 8 KV heads, one sequence of 32k: 24
// columns 32.7, 38.5; 32 columns 38.2, 38.6; 48 columns 68, 39.5; 64 sequences of 2000-4000: 16
// columns 130, 164; 24 columns 183, 166; one sequence, 256 columns: 500 tokens 10.5, 21.8; 2000
// tokens 19.8, 26.2; 4000 tokens 50, 26.5; d = 64, 2 KV heads, 40 sequences of 1000-2000: 64
// columns 46.5, 29; one of 32k: 96 columns 23.7, 33.7.
inline double rows_us(int d, int64_t batch, int64_t units, int64_t pages, int64_t sms) {
  return 12.0 + 12.0 / 128 * d + 0.08 * static_cast<double>(units) +
         0.15 * static_cast<double>(std::min(sms / units, pages / kMinShare)) +
         (0.00065 + 0.00038 / 128 * d) * visited(batch, units, pages);
}

// The largest cluster of which the device holds one per unit at a time; 0: shares are faster,
// as they touch only the tokens there are, or there is none.  Measured, 8 KV heads: one
// sequence of 32k 18.6 us against 23.9, of 128k 48.7 against 54 (both in one run).
inline int cluster_of(int d, int64_t batch, int64_t units, int64_t pages) {
  const ClusterSizes s = cluster_sizes();
  int c = kMaxCluster;
  while (c > 0 && s.active[c] < units) --c;
  if (c == 0) return 0;
  c = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c, pages / 8)));   // half the warps busy
  return cluster_us(d, pages, c) < shares_us(d, batch, units, pages) ? c : 0;
}

// Warps per unit where units are many and short: as many as give every warp slot of the
// device (16 an SM) about one unit.  0: not this form.  Shares pay a merge and a fill of
// the rings per unit, teams the spread of lengths; at d = 128, 8 KV heads, teams against
// shares: 256 sequences of 100-200 tokens 22.8 us against 55.1, 100 of 500-1000 36.5
// against 45.3, 40 of 1000-2000 33.8 both, 40 of 2000-4000 58.6 against 50.3.
inline int team_of(int64_t units, int64_t pages, int64_t sms) {
  if (units <= sms || pages > kTeamPages) return 0;
  int team = 8;
  while (team > 1 && (units * team > 16 * sms || team > pages)) team /= 2;
  return team;
}

// false: sizes outside the supported range.
inline bool kv8_plan(const oscar_kv8_desc* c, int64_t batch, int64_t m_rows, int64_t max_len,
                     Kv8Plan* out) {
  Kv8Plan p{};
  const int64_t cols = m_rows * (c->num_q_heads / c->num_kv_heads);
  const int64_t tiles8 = (cols + 7) / 8, tiles128 = (cols + 127) / 128;
  // (positions, and those of the pages behind the last, fit int32)
  if (max_len > (1 << 30) || cols > (1 << 30) || batch * tiles8 > (1 << 30) || batch * tiles8 * c->num_kv_heads > 0x7fffffff)
    return false;
  const int d = c->head_dim, h = c->num_kv_heads;
  const int64_t pages = std::max<int64_t>(1, (max_len + kPage - 1) / kPage);
  const int64_t sms = oscar_host::sm_count(), units8 = batch * tiles8 * h;
  p.team = team_of(units8, pages, sms);
  if (!p.team) p.cluster = cluster_of(d, batch, units8, pages);
  const double narrow = p.cluster ? 6.0 + cluster_us(d, pages, p.cluster) : shares_us(d, batch, units8, pages);
  p.rows = cols > 8 && rows_us(d, batch, batch * tiles128 * h, pages, sms) < narrow;
  if (p.rows) p.team = p.cluster = 0;
  p.tiles = p.rows ? tiles128 : tiles8;
  p.entries = batch * p.tiles;
  const int64_t units = p.entries * h;
  p.ctas = p.team      ? (units * p.team + 7) / 8
           : p.cluster ? units * p.cluster
                       : share_ctas(p.rows, units, pages, sms);
  p.info = record_bytes(p.ctas);
  p.total = p.cluster || p.team ? 16 : share_bytes(p.rows, d, p.ctas);
  // a smaller call may take another form: shares in narrow tiles at most, or in wide ones
  p.most = share_bytes(false, d, share_ctas(false, units8, pages, sms));
  if (cols > 8) p.most = std::max(p.most, share_bytes(true, d, share_ctas(true, batch * tiles128 * h, pages, sms)));
  *out = p;
  return true;
}

template <int D, bool kE4m3, Kv8Mode kMode>
oscar_status launch_attention(const Kv8Params& p, const Kv8Plan& pl, cudaStream_t st) {
  using C = Kv8Cfg<D, kMode>;
  const auto kernel = kv8_attention_kernel<D, kE4m3, kMode>;
  if (!oscar_host::allow_smem(reinterpret_cast<const void*>(kernel), C::kBytes, kMode == kCluster))
    return OSCAR_ERR_CUDA;
  return launch_kv8(kernel, kMode == kCluster ? pl.cluster : 1, dim3(static_cast<unsigned>(pl.ctas)),
                    C::kThreads, C::kBytes, st, p, kMinShare) == cudaSuccess
             ? OSCAR_OK : OSCAR_ERR_CUDA;
}

template <int D>
oscar_status launch_merge(const Kv8Params& p, const Kv8Plan& pl, cudaStream_t st) {
  const unsigned ctas = static_cast<unsigned>(pl.ctas);
  cudaError_t e;
  if (pl.rows)
    e = launch_kv8(kv8_merge_rows_kernel<D>, 1, dim3(ctas, (std::min(p.cols, 128) + 31) / 32), 4 * D, 0, st, p);
  else   // four warps a column
    e = launch_kv8(kv8_merge_kernel<D>, 1, dim3(ctas, (std::min(p.cols, 8) + 1) / 2), 256, 0, st, p);
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

template <int D, bool kE4m3>
oscar_status run_kv8(const Kv8Params& p, const Kv8Plan& pl, cudaStream_t st) {
  if (pl.team) return launch_attention<D, kE4m3, kTeams>(p, pl, st);
  if (pl.cluster) return launch_attention<D, kE4m3, kCluster>(p, pl, st);
  const oscar_status s = pl.rows ? run_kv8_rows(p, D, kE4m3, pl.ctas, kMinShare, st)
                                 : launch_attention<D, kE4m3, kShares>(p, pl, st);
  if (s != OSCAR_OK) return s;
  return launch_merge<D>(p, pl, st);
}

}  // namespace oscar

namespace oscar_host {

oscar_status check_kv8(const oscar_kv8_desc* c) {
  if (!c) return OSCAR_ERR_INVALID_ARG;
  if (c->num_kv_heads < 1 || c->num_q_heads < 1 || c->max_pages_per_seq < 1 || c->num_pages < 1 ||
      c->num_tails < 1)
    return OSCAR_ERR_INVALID_ARG;
  if (!head_dim_ok(c->head_dim)) return OSCAR_ERR_UNSUPPORTED;
  if (c->format != OSCAR_KV8_INT8 && c->format != OSCAR_KV8_E4M3) return OSCAR_ERR_UNSUPPORTED;
  if (c->num_q_heads % c->num_kv_heads) return OSCAR_ERR_INVALID_ARG;
  if (!c->pool || !c->tail || !c->page_table) return OSCAR_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(c->pool) | reinterpret_cast<uintptr_t>(c->tail)) & 15)
    return OSCAR_ERR_INVALID_ARG;
  return OSCAR_OK;
}

}  // namespace oscar_host

using namespace oscar;

extern "C" {

size_t oscar_kv8_workspace_size(const oscar_kv8_desc* desc, int32_t batch, int32_t m_rows,
                                int32_t max_seq_len) {
  Kv8Plan pl;
  if (oscar_host::check_kv8(desc) != OSCAR_OK || batch < 1 || m_rows < 1 || max_seq_len < 1 ||
      !kv8_plan(desc, batch, m_rows, max_seq_len, &pl))
    return 0;
  return pl.most;
}

oscar_status oscar_kv8_attention(const oscar_kv8_desc* desc, const void* q, const int32_t* seq_lens,
                                 const int32_t* q_pos, int32_t batch, int32_t m_rows,
                                 int32_t max_seq_len, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const oscar_status s = oscar_host::check_kv8(desc);
  if (s != OSCAR_OK) return s;
  if (batch < 0 || m_rows < 0 || max_seq_len < 1 || (!q_pos && m_rows > 1))
    return OSCAR_ERR_INVALID_ARG;
  if (batch == 0 || m_rows == 0) return OSCAR_OK;
  if (!q || !seq_lens || !out || !workspace) return OSCAR_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) |
       reinterpret_cast<uintptr_t>(workspace)) & 15)
    return OSCAR_ERR_INVALID_ARG;
  // whole pages go through the table, the last tokens through the tail
  if (max_seq_len > static_cast<int64_t>(desc->max_pages_per_seq) * kPage + kPage - 1)
    return OSCAR_ERR_INVALID_ARG;
  Kv8Plan pl;
  if (!kv8_plan(desc, batch, m_rows, max_seq_len, &pl)) return OSCAR_ERR_UNSUPPORTED;
  if (workspace_bytes < pl.total) return OSCAR_ERR_WORKSPACE;
  Kv8Params p{};
  p.hkv = desc->num_kv_heads;
  p.hq = desc->num_q_heads;
  p.G = p.hq / p.hkv;
  p.max_pages = desc->max_pages_per_seq;
  p.n_pages = desc->num_pages;
  p.n_tails = desc->num_tails;
  p.pool = static_cast<const uint8_t*>(desc->pool);
  p.tail = static_cast<const uint8_t*>(desc->tail);
  p.page_table = desc->page_table;
  p.tail_ids = desc->tail_ids;
  p.status = desc->status;
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.seq_lens = seq_lens;
  p.q_pos = q_pos;
  p.m_rows = m_rows;
  p.cols = m_rows * p.G;
  p.tiles = static_cast<int>(pl.tiles);
  p.entries = static_cast<int>(pl.entries);
  p.max_len = max_seq_len;
  p.cluster = pl.cluster;
  p.team = pl.team;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(desc->head_dim)));
  p.info = static_cast<int4*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.info);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = desc->format == OSCAR_KV8_E4M3;
  if (desc->head_dim == 128)
    return e4m3 ? run_kv8<128, true>(p, pl, st) : run_kv8<128, false>(p, pl, st);
  return e4m3 ? run_kv8<64, true>(p, pl, st) : run_kv8<64, false>(p, pl, st);
}

}  // extern "C"
