// Attention over the 4-bit cache (kv4_layout.cuh): decode and several query rows per sequence,
// split over the context.
//
//   out[b][m][hq] = sum_t softmax_t(q . k_t / sqrt(d)) v_t,  t <= position of row m,
// with k_t = code s(channel) g_K(page, head), v_t = code s(token, 16 channels) g_V(page, head) for
// tokens in whole pages and bf16 keys and values for the tokens of the tail.
//
// The arithmetic and the units of weights are those of the 8-bit cache (kv8_attention.cu), with
// code * s, exact in fp16, where that one has codes, and g for its scale: the only roundings are
// q (exact down to 2^-21 of a column's largest), p g_V (11 bits, unbiased) and the output.  The
// division of work is that one's too, but that a unit counts for kLead pages more in shares.
//
// What differs: with half the bytes a page, HBM does not bound the loop.  A page of d = 128 takes a warp 64 conversions and 64
// products of codes, 24 conversions of scales and 16 MMAs, 340 instructions in all with its part of queries and merges,
// which would fill an SM's issue slots for 85 cycles where HBM's share of an SM brings a page in 100.  Neither is at its
// limit (64 sequences: issue slots 61% busy, ALU 54%, HBM 64%): the latency of few warps is, four a scheduler, which
// issue once in 6.5 cycles each.
//   - A warp takes two pages at a time: one wait, one softmax step for 32 tokens, and two independent chains of
//     instructions (64 sequences of 4096-8192 tokens 107 us for 115, one of 131071 43 for 54, at the time).
//   - Tiles of 8, 16 or 24 query columns: what was converted serves all of them, and every page is read once.  Of 20
//     columns, 16 sequences of 2000-9001 tokens 64.3 us, as three tiles apart 82; 64 of 2000-4000 124 and 170.  (For more
//     columns, several such tiles, or tiles of 128: kv8_rows.cu.)
//   - The units of weights, queries and merges are the 8-bit cache's, per tile of 8 columns.
//
// Measured, 32/8 heads of 128: 64 sequences of 4096-8192 tokens 99.6 us (HBM's floor 67); one of 131071 of 64/8 heads
// 41.1 us (22.5), one of 32768 18.3 (5.6, of which 7 are launch, queries, first pages and merge); 600 tokens, 4/1 heads of
// 64, 6.5; 64 sequences of 4000-8000, 16/4 heads of 64, 38.3 (16.5).
// Tried, each against what there was at the time: a CTA's warps on the same pages, each with 16 channels of the values and
// weights through shared memory (126 us for 105 of 64 sequences, 50 for 42 of 131071 tokens: two barriers a step);
// scales converted by byte permutes and a product (118 us for 115.5); CTAs of 4 warps for one tile (131071 tokens 46 us
// for 42).
#include "kv8_tiles.cuh"

namespace oscar {

constexpr int kMaxNT = 3;      // tiles of 8 columns that share a page's operands
constexpr int kPair = 2;       // pages of a step

// In shares, a unit counts for so many pages before its own: the change to it takes a CTA that long.  (Of pages alone, 0, a
// CTA with many short units ends last: 30 sequences of 100-6000 tokens, 2 rows of 40 heads, 84.7 us for 46.5; 100 of
// 50-4000 113 for 72.5; 64 of 4096-8192 102.5 for 99.6.  8 and 16: 71 and 58, 95 and 89, 102 and 100; 72: 51, 73, 99.3.
// Of heads of 64, 64 sequences of 4000-8000 tokens, 16/4 heads, 40.8 for 38.5.)
constexpr int kLead = 40;

// CTAs per SM that divide the pages among them.
__host__ __device__ constexpr int kv4_share_ctas(int nt) { return nt == 1 ? 2 : 3; }

// The columns of a tile (kv8_tiles.cuh's Query) in shared memory, for all warps of a CTA: where there are several
// tiles, their operands would take the registers of a third of the warps.
template <int D>
struct SharedQuery {
  uint2 b[D / 16][32];
  float2 fac[32];
  int2 vis[32];
  int vis_min, pad[3];

  __device__ __forceinline__ void put(const Query<D>& q, int lane) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) b[i][lane] = make_uint2(q.b[i][0], q.b[i][1]);
    fac[lane] = make_float2(q.fac[0], q.fac[1]);
    vis[lane] = make_int2(q.vis[0], q.vis[1]);
    if (lane == 0) vis_min = q.vis_min;
  }
};
// One tile's columns as the products see them: in registers, or there.
template <int D, bool kShared>
struct Columns;
template <int D>
struct Columns<D, false> : Query<D> {
  __device__ __forceinline__ uint2 operand(int i, int) const { return make_uint2(this->b[i][0], this->b[i][1]); }
  __device__ __forceinline__ float2 factors(int) const { return make_float2(this->fac[0], this->fac[1]); }
  __device__ __forceinline__ int2 seen(int) const { return make_int2(this->vis[0], this->vis[1]); }
  __device__ __forceinline__ int seen_least() const { return this->vis_min; }
};
template <int D>
struct Columns<D, true> {
  const SharedQuery<D>* q;
  __device__ __forceinline__ uint2 operand(int i, int lane) const { return q->b[i][lane]; }
  __device__ __forceinline__ float2 factors(int lane) const { return q->fac[lane]; }
  __device__ __forceinline__ int2 seen(int lane) const { return q->vis[lane]; }
  __device__ __forceinline__ int seen_least() const { return q->vis_min; }
};

// A CTA's walk over its share of the units, as a warp keeps it in shared memory while the pages are in hand: in registers
// it would push others out of the loop.
struct Kv4Walk {
  int64_t unit0, end, share;   // first page of the current unit, end of the share, its size
  int4 owned;
  Entry t;
  int e, h, p0, p1;
};

template <int D, int NT, Kv8Mode kMode>
struct Kv4Cfg {
  using F = Kv4Fmt<D>;
  // (Shares of several column tiles by small CTAs: while one of them changes units, which takes 10 us of 12 warps
  // and three tiles, the SM's others go on.  64 sequences x 5 rows over 2000-4000 tokens 134 us for 180 before units had
  // a lead, 124 since; 64 sequences with one tile, 101 us both at the time.)
  static constexpr int kWarps = kMode == kShares ? (NT > 1 ? 4 : 8) : kMode == kTeams ? 8 : NT > 1 ? 12 : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kAtOnce = NT < 3 ? kPair : 1;        // pages whose logits are in registers
  static constexpr int kCtas = kMode == kShares ? kv4_share_ctas(NT) : kMode == kTeams ? 2 : 1;   // per SM
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kStage = kPair * F::kBlock;
  static constexpr int kWarpRing = kStages * kStage;
  static constexpr int kStride = D + 4;                     // floats per column when merging
  static constexpr int kMerge = kWarps * 8 * kStride * 4;   // 8 columns at a time
  static constexpr int kStat = kWarps * 8 * NT * 4;         // one of m, k, l
  static constexpr int kMergeOff = kWarps * kWarpRing;
  static constexpr int kStatOff = kMergeOff + kMerge;
  static constexpr int kUnitOff = kStatOff + 3 * kStat;     // float2: units that the parts are brought to
  static constexpr int kPartOff = kUnitOff + kWarps * 8 * NT * 8;   // a cluster's CTA: its partial
  static constexpr int kQueryOff = kPartOff + (kMode == kCluster ? kv8_slot<D, NT>() * 4 : 0);
  static constexpr int kBarOff = kQueryOff + (NT > 1 ? NT * static_cast<int>(sizeof(SharedQuery<D>)) : 0);
  // The tail's block goes to where the parts are merged later, so that it comes while the pages do; a team's share of that
  // may be smaller, and its tail takes the ring when the pages are through.
  static constexpr bool kTailApart = kMode != kTeams;
  static constexpr int kTailBar = kBarOff + kWarps * kStages * 8;
  static constexpr int kWalk = (kTailBar + 8 + 15) / 16 * 16;   // a warp each
  static constexpr int kBytes = kWalk + (kMode == kShares ? kWarps * static_cast<int>(sizeof(Kv4Walk)) : 0);
  static_assert(kMerge >= F::kTailBytes || !kTailApart, "a tail block fits where parts are merged");
  static_assert(kWarpRing >= F::kTailBytes, "a warp's ring holds a tail block");
  static_assert(kStage % 16 == 0 && kMergeOff % 16 == 0 && kUnitOff % 16 == 0 && kPartOff % 16 == 0, "alignment");
};

// weigh (kv8_tiles.cuh) for the tokens of N pages: logits lg[n] in the accumulator layout, value scales 2^off[n].
template <int D, int N>
__device__ __forceinline__ void weigh_pages(Running<D>& s, const float (&lg)[N][4], const float (&off)[N],
                                            float (&w)[N][4]) {
  float e[N][4], up[N][2];
  bool over = false;
  const uint64_t less = two(-1.f, -1.f), m2 = two(s.m[0], s.m[1]), k2 = two(s.k[0], s.k[1]);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint64_t e0 = fma2(m2, less, two(lg[n][0], lg[n][1])), e1 = fma2(m2, less, two(lg[n][2], lg[n][3]));
    const uint64_t u2 = fma2(k2, less, two(off[n], off[n]));
    e[n][0] = first(e0); e[n][1] = second(e0); e[n][2] = first(e1); e[n][3] = second(e1);
    up[n][0] = first(u2); up[n][1] = second(u2);
#pragma unroll
    for (int c = 0; c < 2; ++c) over |= fmaxf(e[n][c], e[n][2 + c]) > fminf(kLag, kLag + kLift - up[n][c]);
  }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float top[N], m = s.m[c];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        top[n] = fmaxf(lg[n][c], lg[n][2 + c]);
        top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 4));
        top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 8));
        top[n] = fmaxf(top[n], __shfl_xor_sync(0xffffffffu, top[n], 16));
        m = fmaxf(m, top[n]);
      }
      const float down = s.m[c] - m, k0 = s.k[c] + down;
      // the unit as it is, seen from m; and what these pages need
      float k = fmaxf(k0, kNoUnit.k);
#pragma unroll
      for (int n = 0; n < N; ++n) k = fmaxf(k, top[n] - m + off[n] - kLift);
      s.l[c] *= fast_exp2(down);
      const float a = fast_exp2(k0 - k);
      s.m[c] = m;
      s.k[c] = k;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        e[n][c] = lg[n][c] - m;
        e[n][2 + c] = lg[n][2 + c] - m;
        up[n][c] = off[n] - k;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        s.o[i][c] *= a;
        s.o[i][2 + c] *= a;
      }
    }
  }
  uint64_t l = two(s.l[0], s.l[1]);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    // (finite: it meets p of 0 where it is large)
    const uint64_t scale = two(fast_exp2(fminf(up[n][0], 126.f)), fast_exp2(fminf(up[n][1], 126.f)));
    const uint64_t p0 = two(fast_exp2(e[n][0]), fast_exp2(e[n][1])), p1 = two(fast_exp2(e[n][2]), fast_exp2(e[n][3]));
    l = add2(l, add2(p0, p1));
    const uint64_t w0 = mul2(p0, scale), w1 = mul2(p1, scale);
    w[n][0] = first(w0);
    w[n][1] = second(w0);
    w[n][2] = first(w1);
    w[n][3] = second(w1);
  }
  s.l[0] = first(l);
  s.l[1] = second(l);
}

// N pages of codes, at st and kBlock on, their tokens from first_token and first_token + step on.
template <int D, int NT, int N>
__device__ __forceinline__ void take_pages(const uint8_t* st, int first_token, int step, int lane,
                                          const Columns<D, (NT > 1)> (&q)[NT], Running<D> (&s)[NT]) {
  using F = Kv4Fmt<D>;
  const int gid = lane >> 2, tig = lane & 3;
  int page0[N];
  const uint8_t* at[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    page0[n] = first_token + n * step;
    at[n] = st + n * F::kBlock;
  }
  float lg[NT][N][4];
  float off[N], sk[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const float2 sc = *reinterpret_cast<const float2*>(at[n] + F::kScales);
    sk[n] = sc.x;
    off[n] = fast_log2(sc.y);   // (a page of zeros: -inf, weights of 0)
#pragma unroll
    for (int t = 0; t < NT; ++t) lg[t][n][0] = lg[t][n][1] = lg[t][n][2] = lg[t][n][3] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint4 k = reinterpret_cast<const uint4*>(at[n])[32 * j + lane];   // tokens 2 gid, 2 gid + 1
      const uint4 sc = reinterpret_cast<const uint4*>(at[n] + F::kKeyScales)[4 * j + tig];
      const uint32_t t0[2] = {k.x, k.y}, t1[2] = {k.z, k.w}, s4[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
      for (int w = 0; w < 2; ++w) {   // 8 channels: two k-steps
        uint32_t a[4], b[4], x[4];
        kv4_pairs(t0[w], a[0], a[1], a[2], a[3]);
        kv4_pairs(t1[w], b[0], b[1], b[2], b[3]);
        kv4_scales(s4[2 * w], x[0], x[1]);
        kv4_scales(s4[2 * w + 1], x[2], x[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = hmul2_u32(a[i], x[i]);
          b[i] = hmul2_u32(b[i], x[i]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint2 q0 = q[t].operand(4 * j + 2 * w, lane), q1 = q[t].operand(4 * j + 2 * w + 1, lane);
          mma_f16(lg[t][n], a[0], b[0], a[1], b[1], q0.x, q0.y);
          mma_f16(lg[t][n], a[2], b[2], a[3], b[3], q1.x, q1.y);
        }
      }
    }
  }
  uint32_t wb[NT][N][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float2 fac = q[t].factors(lane);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float f0 = logit_factor(sk[n], fac.x), f1 = logit_factor(sk[n], fac.y);
      // (rounded by themselves, not on the way to a difference, so that equal logits stay equal)
#pragma unroll
      for (int r = 0; r < 4; ++r) lg[t][n][r] = __fmul_rn(lg[t][n][r], r & 1 ? f1 : f0);
      if (page0[n] + kPage > q[t].seen_least()) {
        const int tk = page0[n] + 2 * gid;
        const int2 seen = q[t].seen(lane);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int vis = c ? seen.y : seen.x;
          if (tk >= vis) lg[t][n][c] = -INFINITY;
          if (tk + 1 >= vis) lg[t][n][2 + c] = -INFINITY;
        }
      }
    }
    float w[N][4];
    weigh_pages<D, N>(s[t], lg[t], off, w);
    // rows gid of the logits were tokens 2 gid and 2 gid + 1: transposed and put in order, the two
    // registers hold tokens (4tig, 4tig + 1) and (4tig + 2, 4tig + 3) of column gid
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t b0 = movmatrix_trans(pack_half2(w[n][0], w[n][1]));
      const uint32_t b1 = movmatrix_trans(pack_half2(w[n][2], w[n][3]));
      wb[t][n][0] = __byte_perm(b0, b1, 0x5410);
      wb[t][n][1] = __byte_perm(b0, b1, 0x7632);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      // channels 64i + 4 gid and on, 64i + 32 + 4 gid and on, of tokens 4 tig and on
      const uint4 v = reinterpret_cast<const uint4*>(at[n] + F::kCodes)[32 * i + lane];
      const uint2 sc = reinterpret_cast<const uint2*>(at[n] + F::kValueScales)[8 * i + 4 * (gid >> 2) + tig];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t s01, s23;
        kv4_scales(half ? sc.y : sc.x, s01, s23);
#pragma unroll
        for (int y = 0; y < 2; ++y) {   // two channels
          uint32_t a0, a1, a2, a3;
          kv4_pairs(w[2 * half + y], a0, a2, a1, a3);
          a0 = hmul2_u32(a0, s01);
          a1 = hmul2_u32(a1, s01);
          a2 = hmul2_u32(a2, s23);
          a3 = hmul2_u32(a3, s23);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            mma_f16(s[t].o[4 * i + 2 * half + y], a0, a1, a2, a3, wb[t][n][0], wb[t][n][1]);
        }
      }
    }
  }
}

// A warp's ring of copies, two pages a stage, a lane each.  Stages are used in turn, each when its step before
// has been consumed; a stage's barrier counts two arrivals.
template <typename C>
struct Ring4 {
  uint8_t* base;
  uint64_t* bars;
  int32_t* status;
  uint32_t phases;         // bit per stage
  uint32_t there;          // two bits per step in flight, the oldest lowest: pages whose copies were made
  int at, flying;          // stage of the oldest step, steps in flight
  bool alive;              // false after a copy that did not arrive in time
  // lanes 0 and 1: their pages to come of the unit's part
  const int32_t* ids;
  int left, stride, next_id;

  static __device__ __forceinline__ int after(int st) { return st + 1 == C::kStages ? 0 : st + 1; }

  // The next step, into the stage behind those in flight; `src` is the KV head's first block.
  __device__ __forceinline__ void issue(const Kv8Params& p, const uint8_t* src, int st, int lane) {
    bool ok = false;
    if (lane < kPair) {
      ok = left > 0 && next_id >= 0 && next_id < p.n_pages;
      mbar_arrive_expect_tx(bars + st, ok ? C::F::kBlock : 0);
      if (ok)
        bulk_g2s(base + st * C::kStage + lane * C::F::kBlock,
                 src + static_cast<int64_t>(next_id) * p.hkv * C::F::kBlock, C::F::kBlock, bars + st);
      else if (left > 0 && status)
        atomicOr(status, OSCAR_DEVERR_PAGE_ID);
      ids += stride;
      if (--left > 0) next_id = *ids;
    }
    there |= __ballot_sync(0xffffffffu, ok) << (2 * flying);
    ++flying;
  }
  __device__ __forceinline__ void issue_tail(const Kv8Params& p, const Entry& t, int h, int lane) {
    const int64_t id = p.tail_ids ? p.tail_ids[t.b] : t.b;
    const bool ok = id >= 0 && id < p.n_tails;
    if (lane < kPair) {
      mbar_arrive_expect_tx(bars + at, ok && lane == 0 ? C::F::kTailBytes : 0);
      if (lane == 0) {
        if (ok) bulk_g2s(base, p.tail + (id * p.hkv + h) * C::F::kTailBytes, C::F::kTailBytes, bars + at);
        else if (status) atomicOr(status, OSCAR_DEVERR_PAGE_ID);
      }
    }
    there = ok;
    flying = 1;
  }
  // Starts a warp's part of a unit (nothing is in flight): as many steps as there are stages, or the tail.
  __device__ __forceinline__ void start(const Kv8Params& p, const Entry& t, int h, const Part& a, int step, int lane) {
    there = 0;
    flying = 0;
    if (!alive) return;
    const int pages = a.first < a.end ? (a.end - a.first + step - 1) / step : 0;
    ids = p.page_table + static_cast<size_t>(t.b) * p.max_pages + a.first + lane * step;
    stride = kPair * step;
    left = (pages - lane + 1) / kPair;   // (of lanes 0 and 1)
    if (lane < kPair && left > 0) next_id = *ids;
    const uint8_t* src = p.pool + static_cast<int64_t>(h) * C::F::kBlock;
    int st = at;
#pragma unroll 1
    for (int i = 0; i < C::kStages && kPair * i < pages; ++i, st = after(st)) issue(p, src, st, lane);
    if (!C::kTailApart && pages == 0 && a.tail) issue_tail(p, t, h, lane);
  }
  // Waits for the oldest step and takes it off; which of its copies were made; ~0u: it did not come in time, and no
  // copy is left in flight.
  __device__ __forceinline__ uint32_t take() {
    const bool got = wait_copy(bars + at, (phases >> at) & 1u, status);
    if (__all_sync(0xffffffffu, got)) {
      phases ^= 1u << at;
      const uint32_t mask = there & 3u;
      there >>= 2;
      --flying;
      return mask;
    }
    for (int st = at; flying > 0; --flying, st = after(st)) wait_longer(bars + st, (phases >> st) & 1u, status);
    alive = false;
    return ~0u;
  }
};

// The rest of a wait for the tail's block: false when it did not come in time.  (Parts are put there next, so it has
// another while not to be in flight any more.)
static __device__ __noinline__ bool wait_tail(uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_wait(bar, parity, status)) return true;
  mbar_wait(bar, parity, status);
  return false;
}

// merge_cluster for NT tiles of 8 columns.
template <int D, int NT>
__device__ __forceinline__ void merge_cluster4(const Kv8Params& p, const Entry& t, int h, const float* slot, float4* stats) {
  cluster_sync();
  const int n = p.cluster, rank = blockIdx.x % n;
  constexpr int kOne = kv8_slot<D, 1>();
  for (int i = threadIdx.x; i < 8 * NT * n; i += blockDim.x) {
    const int col = i % (8 * NT);
    stats[i] = cluster_load4(cluster_address(slot + col / 8 * kOne + 8 * D + 4 * (col % 8), i / (8 * NT)));
  }
  __syncthreads();
  constexpr int kAll = 8 * NT * D / 4;          // float4 of a unit
  const int per = (kAll + n - 1) / n, end = min(kAll, (rank + 1) * per);
  for (int i = rank * per + threadIdx.x; i < end; i += blockDim.x) {
    const int col = i / (D / 4), ch = 4 * (i % (D / 4)), gcol = t.tile * 8 * NT + col;
    if (gcol >= p.cols) continue;
    float m = kLowest, k = kLowest, l = 0.f;
    for (int r = 0; r < n; ++r) m = fmaxf(m, stats[8 * NT * r + col].x);
    for (int r = 0; r < n; ++r) k = fmaxf(k, (stats[8 * NT * r + col].x - m) + stats[8 * NT * r + col].y);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < n; ++r) {
      const float4 part = stats[8 * NT * r + col];
      const float4 x = cluster_load4(cluster_address(slot + col / 8 * kOne + col % 8 * D + ch, r));
      const float down = part.x - m, a = fast_exp2(down + part.y - k);
      l = fmaf(fast_exp2(down), part.z, l);
      o.x = fmaf(a, x.x, o.x); o.y = fmaf(a, x.y, o.y);
      o.z = fmaf(a, x.z, o.z); o.w = fmaf(a, x.w, o.w);
    }
    store_row(p, t.b, h, gcol, ch, D, o, output_factor(k, l));
  }
  cluster_sync();   // no CTA leaves while its shared memory is read
}

template <int D, int NT, Kv8Mode kMode>
__global__ void __launch_bounds__((Kv4Cfg<D, NT, kMode>::kThreads), (Kv4Cfg<D, NT, kMode>::kCtas))
kv4_attention_kernel(const __grid_constant__ Kv8Params p, int min_share) {
  using C = Kv4Cfg<D, NT, kMode>;
  constexpr int kWarps = C::kWarps, kCols = 8 * NT, kOne = kv8_slot<D, 1>();
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  // the warps of a unit (all, or a team of them) and this one's place among them
  const int team = kMode == kTeams ? p.team : kWarps;
  const int number = kMode == kTeams ? (tid >> 5) / team : 0;
  const int warp = (tid >> 5) - number * team;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  float* sm_m = reinterpret_cast<float*>(smem + C::kStatOff) + number * team * kCols;
  float* sm_k = sm_m + kWarps * kCols;
  float* sm_l = sm_k + kWarps * kCols;
  float2* sm_unit = reinterpret_cast<float2*>(smem + C::kUnitOff) + number * kCols;
  float* merge = reinterpret_cast<float*>(smem + C::kMergeOff) + number * team * 8 * C::kStride;
  uint64_t* tail_bar = reinterpret_cast<uint64_t*>(smem + C::kTailBar);
  uint32_t tail_phase = 0;
  if (tid < kWarps * C::kStages) mbar_init(bars + tid, kPair);
  if (tid == 0) mbar_init(tail_bar, 1);
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
    t = entry_of<NT>(p, e);
    end = t.pages;
  } else if constexpr (kMode == kCluster) {   // this CTA's run of the cluster's unit
    const int unit = blockIdx.x / p.cluster, rank = blockIdx.x - unit * p.cluster;
    e = unit / p.hkv;
    h = unit - e * p.hkv;
    t = entry_of<NT>(p, e);
    at = static_cast<int64_t>(t.pages) * rank / p.cluster;
    end = static_cast<int64_t>(t.pages) * (rank + 1) / p.cluster;
  } else {
    bool any;
    const Share sh = find_share<NT, kWarps, kLead>(p, min_share, any);
    // (a share that ends in a unit's lead has no page of it)
    if (!any || sh.end - sh.unit0 <= kLead) {
      if (tid == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
      return;
    }
    at = max(sh.at, sh.unit0 + kLead);
    end = sh.end;
    share = sh.share;
    unit0 = sh.unit0 + kLead;   // (a unit's first page stands behind its lead)
    e = sh.e;
    h = sh.h;
    t = sh.t;
  }

  Ring4<C> ring{smem + (tid >> 5) * C::kWarpRing, bars + (tid >> 5) * C::kStages, p.status, 0, 0, 0, 0, true,
                nullptr, 0, 0, 0};
  int4 owned = make_int4(0, 0, 0, 0);
  int p0 = static_cast<int>(at - unit0);
  int p1 = static_cast<int>(min(static_cast<int64_t>(t.pages), end - unit0));
  Part mine = part_of(t, p0, p1, warp, team);
  ring.start(p, t, h, mine, team, lane);

  for (;;) {
    Columns<D, (NT > 1)> q[NT];
    Running<D> s[NT];
    if constexpr (NT > 1) {   // a warp a tile, for all
      SharedQuery<D>* shared = reinterpret_cast<SharedQuery<D>*>(smem + C::kQueryOff);
      if (warp < NT) {
        Query<D> one;
        load_query<D, kCodeE2m1>(p, t, h, t.tile * kCols + 8 * warp, lane, one);
        shared[warp].put(one, lane);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) q[n].q = shared + n;
      __syncthreads();
    } else {
      load_query<D, kCodeE2m1>(p, t, h, t.tile * kCols, lane, q[0]);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) reset<D>(s[n]);
    if (p0 == 0 && h == 0 && t.tile == 0 && warp == 0 && lane == 0 && p.status) {
      const int len = p.seq_lens[t.b];
      if (len < 0 || len > p.max_len) atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
    }
    if (p.q_pos && p0 == 0 && h == 0 && warp == 0 && lane < kCols && p.status) {
      const int row = (t.tile * kCols + lane) / p.G;
      if (row < p.m_rows && p.q_pos[static_cast<size_t>(t.b) * p.m_rows + row] >= t.len)
        atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
    }
    // the tail's block, for all warps: each takes a tile of its columns, those with the fewest pages
    bool tail_there = false;
    const bool tail_asked = C::kTailApart && p1 > t.n8 && t.vis > t.len / kPage * kPage;
    const int tail_tile = tail_asked ? (warp + kWarps - (max(t.n8, p0) - p0) % kWarps) % kWarps : kWarps;
    if (tail_asked) {
      const int64_t id = p.tail_ids ? p.tail_ids[t.b] : t.b;
      tail_there = id >= 0 && id < p.n_tails;
      if (tid == 0) {
        fence_proxy_async();   // (parts of the unit before were read there)
        mbar_arrive_expect_tx(tail_bar, tail_there ? C::F::kTailBytes : 0);
        if (tail_there)
          bulk_g2s(smem + C::kMergeOff, p.tail + (id * p.hkv + h) * C::F::kTailBytes, C::F::kTailBytes, tail_bar);
        else if (p.status)
          atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
      }
    }
    Kv4Walk* walk = reinterpret_cast<Kv4Walk*>(smem + C::kWalk) + (tid >> 5);
    if constexpr (kMode == kShares) {
      if (lane == 0) *walk = {unit0, end, share, owned, t, e, h, p0, p1};
    }
    const uint8_t* src = p.pool + static_cast<int64_t>(h) * C::F::kBlock;
    // (from start on, a step is issued for each that is taken, while there are more)
    int left = mine.first < mine.end ? (mine.end - mine.first + kPair * team - 1) / (kPair * team) : 0;
    bool tail_here = mine.tail && left == 0;
#pragma unroll 1
    for (int page0 = mine.first * kPage; left > 0 && ring.alive; --left, page0 += kPair * team * kPage) {
      const uint32_t there = ring.take();
      if (there == ~0u) break;
      // (a refused id's stands for nothing)
      const uint8_t* st = ring.base + ring.at * C::kStage;
      if constexpr (C::kAtOnce == kPair) {
        if (there == 3u) {
          take_pages<D, NT, kPair>(st, page0, team * kPage, lane, q, s);
        } else if (there) {   // the last of an odd number, or beside a refused id (as a pair: 32768 tokens 18.9 us for 18.3)
          const int n = there >> 1;
          take_pages<D, NT, 1>(st + n * C::F::kBlock, page0 + n * team * kPage, 0, lane, q, s);
        }
      } else {
#pragma unroll 1
        for (int n = 0; n < kPair; ++n)
          if ((there >> n) & 1u) take_pages<D, NT, 1>(st + n * C::F::kBlock, page0 + n * team * kPage, 0, lane, q, s);
      }
      __syncwarp();
      if (left > C::kStages) ring.issue(p, src, ring.at, lane);
      ring.at = ring.after(ring.at);
    }
    if constexpr (kMode == kShares) {
      __syncwarp();
      asm volatile("" ::: "memory");   // (from there)
      unit0 = walk->unit0;
      end = walk->end;
      share = walk->share;
      owned = walk->owned;
      t = walk->t;
      e = walk->e;
      h = walk->h;
      p0 = walk->p0;
      p1 = walk->p1;
    }
    const uint8_t* tail_block = ring.base;
    if constexpr (C::kTailApart) {
      if (tail_asked) {
        const bool got = __all_sync(0xffffffffu, mbar_try_wait(tail_bar, tail_phase) || wait_tail(tail_bar, tail_phase, p.status));
        tail_phase ^= 1u;
        tail_there = tail_there && got;
      }
      tail_block = smem + C::kMergeOff;
    } else if (mine.tail && ring.alive) {
      if (!tail_here) ring.issue_tail(p, t, h, lane);
      tail_there = ring.take() == 1u;
      ring.at = ring.after(ring.at);
    }
    if (tail_there) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (C::kTailApart && n != tail_tile) continue;
        Query<D> seen;   // (of which only this is looked at)
        const int2 vis = q[n].seen(lane);
        seen.vis[0] = vis.x;
        seen.vis[1] = vis.y;
        seen.vis_min = q[n].seen_least();
        tail_tokens<D>(p, t, h, t.tile * kCols + 8 * n, tail_block, t.len / kPage * kPage, t.len % kPage, lane, seen, s[n]);
      }
    }
    __syncwarp();

    // the next unit of this CTA: its copies start before this one is merged
    const Entry tc = t;
    const int hc = h, c0 = p0, c1 = p1;
    const int64_t u0 = unit0;
    const bool more = kMode == kShares && u0 + tc.pages + kLead < end;
    if (more) {
      unit0 = u0 + tc.pages + kLead;
      if (++h == p.hkv) {
        h = 0;
        t = entry_of<NT>(p, ++e);
      }
      p0 = 0;
      p1 = static_cast<int>(min(static_cast<int64_t>(t.pages), end - unit0));
      mine = part_of(t, p0, p1, warp, team);
      ring.start(p, t, h, mine, team, lane);
    }

    if (gid == 0) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sm_m[warp * kCols + 8 * n + 2 * tig + c] = s[n].m[c];
          sm_k[warp * kCols + 8 * n + 2 * tig + c] = s[n].k[c];
        }
    }
    team_sync<kMode>(team, number);
    const bool complete = c0 == 0 && c1 == tc.pages;
    float* slot = kMode == kCluster
        ? reinterpret_cast<float*>(smem + C::kPartOff)
        : p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * (NT * kOne);
#pragma unroll
    for (int n = 0; n < NT; ++n) {   // 8 columns at a time
      // the parts of a column in the unit of the largest m, and the k with which it lies as high as the highest
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 2 * tig + c, at_col = 8 * n + col;
        float m = kLowest, k = kLowest;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          if (kMode != kTeams || w < team) m = fmaxf(m, sm_m[w * kCols + at_col]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          if (kMode != kTeams || w < team) k = fmaxf(k, (sm_m[w * kCols + at_col] - m) + sm_k[w * kCols + at_col]);
        const float down = s[n].m[c] - m, a = fast_exp2(down + s[n].k[c] - k);
        float l = s[n].l[c] * fast_exp2(down);
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (gid == 0) sm_l[warp * kCols + at_col] = l;
        if (warp == 0 && gid == 0) sm_unit[at_col] = make_float2(m, k);
        float* dst = merge + (warp * 8 + col) * C::kStride + 4 * gid;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          *reinterpret_cast<float4*>(dst + 32 * i) =
              make_float4(s[n].o[2 * i][c] * a, s[n].o[2 * i][2 + c] * a,
                          s[n].o[2 * i + 1][c] * a, s[n].o[2 * i + 1][2 + c] * a);
      }
      team_sync<kMode>(team, number);
      for (int i = warp * 32 + lane; i < 8 * D / 4; i += 32 * team) {
        const int col = i / (D / 4), ch = 4 * (i % (D / 4));
        const int gcol = tc.tile * kCols + 8 * n + col;
        if (kMode != kCluster && gcol >= p.cols) continue;
        const float2 unit = sm_unit[8 * n + col];
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          if (kMode == kTeams && w >= team) break;
          l += sm_l[w * kCols + 8 * n + col];
          const float4 x = *reinterpret_cast<const float4*>(merge + (w * 8 + col) * C::kStride + ch);
          o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
        }
        if (kMode != kCluster && (kMode == kTeams || complete)) {
          store_row(p, tc.b, hc, gcol, ch, D, o, output_factor(unit.y, l));
        } else {
          *reinterpret_cast<float4*>(slot + n * kOne + col * D + ch) = o;
          if (ch == 0)
            *reinterpret_cast<float4*>(slot + n * kOne + 8 * D + 4 * col) = make_float4(unit.x, unit.y, l, 0.f);
        }
      }
      if (kMode != kTeams) __syncthreads();   // before the buffers are written again
    }
    if constexpr (kMode == kCluster) {
      merge_cluster4<D, NT>(p, tc, hc, slot, reinterpret_cast<float4*>(merge));
      return;
    }
    if constexpr (kMode == kTeams) return;
    if (!complete && c0 == 0)   // the unit goes on in the next CTAs: they hold its other parts
      owned = make_int4(e, hc, static_cast<int>((u0 + tc.pages - 1) / share) - blockIdx.x + 1, 0);
    if (!more) break;
  }
  if (tid == 0) p.info[blockIdx.x] = owned;
}

struct Kv4Plan {
  int nt;              // tiles of 8 columns that share pages; 0: tiles of 128 columns (kv8_rows.cu)
  int cluster, team;   // cluster > 0: CTAs per unit; team > 0: warps per unit
  int64_t tiles, entries, ctas;
  size_t info, total;   // workspace bytes: the CTAs' records, all
  size_t most;          // no call of fewer sequences, rows or tokens takes more than this
};

// CTAs that share the pages of `units`.
inline int64_t share_ctas4(int nt, int64_t units, int64_t pages, int64_t sms) {
  return std::min(std::min<int64_t>(kMaxCtas, kv4_share_ctas(nt) * sms), (units * (pages + kLead) + kMinShare - 1) / kMinShare);
}

// Estimates in us of nt column tiles (kv8_plan says what they stand for).  A page costs d = 64 two thirds of what it costs
// d = 128.  Fitted to these, 32/8 heads of 128, in us ("-": more units than SMs; nt = 1, 2, 3 in turn):
//                                      shares             clusters           teams   128 columns
//   1 x 1 row over 512, 8000           8.2, 12.0          6.9, 9.7
//   1 x 1 row over 32768, 131071       18.0, 40.1         17.2, 46.6
//   16 x 1 row over 4000-8000          35.8               35.9               283
//   64 x 1 row over 500-1000           29.6               -                  22.9
//   40 x 1 row over 1000-2000          29.1               -                  34.2
//   100 x 1 row over 50-4000           72.6               -                  147
//   256 x 1 row over 100-200           51.3               -                  21.2
//   1 x 3 rows over 32768              24.3, 24.5         27.3, 22.5                 37.9
//   1 x 5 rows over 32768              31.2, 33.8, 33.3   31.2, 35.5, 29.5           38.1
//   1 x 16 rows over 32768             62.1, 50.4, 58.9   64.7, 48.7, 56.1           40.2
//   16 x 5 rows over 2000-9001         82.2, 73.1, 64.5   -, -, 69.7         305     79.0
//   16 x 5 rows over 9000-9001         111, 101, 87.5     -, -, 74.5                 94.8
//   64 x 3 rows over 2000-4000         117, 82.1          -                  153     169
//   64 x 4 rows over 200-400           46.0, 37.7         -                  24.9    76.1
//   1 x 64 rows over 500               18.3, 20.5, 23.9   -, 11.4, 13.3      11.1    21.7
// The rule takes the fastest of each row but two: for 1 x 64 rows clusters (11.4 us for 11.1), and for 16 x 5 rows of one
// length shares (87.5 for 74.5), as the host takes a batch's lengths for three quarters of the longest on average.
inline double page_us4(int d) { return 0.35 + 0.65 / 128 * d; }
inline double shares_us4(int d, int nt, int64_t batch, int64_t units, int64_t pages) {
  const double start[] = {11.5, 14, 19}, page[] = {0.00044, 0.00062, 0.00085}, unit[] = {0.015, 0.015, 0.04};
  return start[nt - 1] + page[nt - 1] * page_us4(d) * visited(batch, units, pages) + unit[nt - 1] * static_cast<double>(units);
}
inline double cluster_us4(int d, int nt, int64_t pages, int c) {
  const double start[] = {7, 8, 8}, page[] = {0.063, 0.095, 0.115};
  return start[nt - 1] + page[nt - 1] * page_us4(d) * static_cast<double>(pages) / c;
}
inline double team_us4(int d, int64_t units, int64_t pages, int64_t sms) {
  return 7 + 0.095 * page_us4(d) * static_cast<double>(units) * static_cast<double>(pages) / static_cast<double>(sms);
}
inline double rows_us4(int d, int64_t batch, int64_t units, int64_t pages, int64_t sms) {
  return rows_us(d, batch, units, pages, sms) - 0.00008 / 128 * d * visited(batch, units, pages);
}

inline int cluster_of4(int d, int nt, int64_t batch, int64_t units, int64_t pages) {
  const ClusterSizes s = cluster_sizes();   // (every cluster kernel fills an SM)
  int c = kMaxCluster;
  while (c > 0 && s.active[c] < units) --c;
  if (c == 0) return 0;
  c = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(c, pages / 8)));   // half the warps busy
  return cluster_us4(d, nt, pages, c) < shares_us4(d, nt, batch, units, pages) ? c : 0;
}

// false: sizes outside the supported range.
inline bool kv4_plan(const oscar_kv8_desc* c, int64_t batch, int64_t m_rows, int64_t max_len, Kv4Plan* out) {
  Kv4Plan p{};
  const int64_t cols = m_rows * (c->num_q_heads / c->num_kv_heads);
  const int64_t tiles8 = (cols + 7) / 8, tiles128 = (cols + 127) / 128;
  // (positions, and those of the pages behind the last, fit int32)
  if (max_len > (1 << 30) || cols > (1 << 30) || batch * tiles8 > (1 << 30) || batch * tiles8 * c->num_kv_heads > 0x7fffffff)
    return false;
  const int d = c->head_dim, h = c->num_kv_heads;
  const int64_t pages = std::max<int64_t>(1, (max_len + kPage - 1) / kPage);
  const int64_t sms = oscar_host::sm_count(), units8 = batch * tiles8 * h;
  double best = 0;
  for (int nt = 1; nt <= kMaxNT && (nt == 1 || tiles8 > nt - 1); ++nt) {
    Kv4Plan x{};
    x.nt = nt;
    x.tiles = (tiles8 + nt - 1) / nt;
    const int64_t units = batch * x.tiles * h;
    x.cluster = cluster_of4(d, nt, batch, units, pages);
    double us = x.cluster ? cluster_us4(d, nt, pages, x.cluster) : shares_us4(d, nt, batch, units, pages);
    const int team = nt == 1 ? team_of(units, pages, sms) : 0;
    if (team && team_us4(d, units, pages, sms) < us) {
      us = team_us4(d, units, pages, sms);
      x.team = team;
      x.cluster = 0;
    }
    if (nt == 1 || us < best) {
      best = us;
      p = x;
    }
  }
  if (cols > 8 && rows_us4(d, batch, batch * tiles128 * h, pages, sms) < best) {
    p = Kv4Plan{};
    p.tiles = tiles128;
  }
  p.entries = batch * p.tiles;
  const int64_t units = p.entries * h;
  p.ctas = p.team      ? (units * p.team + 7) / 8
           : p.cluster ? units * p.cluster
           : p.nt      ? share_ctas4(p.nt, units, pages, sms)
                       : share_ctas(true, units, pages, sms);
  p.info = record_bytes(p.ctas);
  p.total = p.cluster || p.team ? 16 : part_bytes(p.nt ? 8 * p.nt : 128, d, p.ctas);
  // a smaller call may take another form: shares of any number of columns up to these, or wide tiles
  for (int nt = 1; nt <= kMaxNT && (nt == 1 || tiles8 > nt - 1); ++nt)
    p.most = std::max(p.most, part_bytes(8 * nt, d, share_ctas4(nt, units8, pages, sms)));
  if (cols > 8) p.most = std::max(p.most, share_bytes(true, d, share_ctas(true, batch * tiles128 * h, pages, sms)));
  *out = p;
  return true;
}

template <int D, int NT, Kv8Mode kMode>
oscar_status launch_attention4(const Kv8Params& p, const Kv4Plan& pl, cudaStream_t st) {
  using C = Kv4Cfg<D, NT, kMode>;
  const auto kernel = kv4_attention_kernel<D, NT, kMode>;
  if (!oscar_host::allow_smem(reinterpret_cast<const void*>(kernel), C::kBytes, kMode == kCluster))
    return OSCAR_ERR_CUDA;
  return launch_kv8(kernel, kMode == kCluster ? pl.cluster : 1, dim3(static_cast<unsigned>(pl.ctas)),
                    C::kThreads, C::kBytes, st, p, kMinShare) == cudaSuccess
             ? OSCAR_OK : OSCAR_ERR_CUDA;
}

template <int D, int NT>
oscar_status run_tiles4(const Kv8Params& p, const Kv4Plan& pl, cudaStream_t st) {
  if constexpr (NT == 1)
    if (pl.team) return launch_attention4<D, 1, kTeams>(p, pl, st);
  if (pl.cluster) return launch_attention4<D, NT, kCluster>(p, pl, st);
  const oscar_status s = launch_attention4<D, NT, kShares>(p, pl, st);
  if (s != OSCAR_OK) return s;
  // four warps a column
  return launch_kv8(kv8_merge_kernel<D, NT>, 1, dim3(static_cast<unsigned>(pl.ctas), (std::min(p.cols, 8 * NT) + 1) / 2),
                    256, 0, st, p) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

template <int D>
oscar_status run_kv4(const Kv8Params& p, const Kv4Plan& pl, cudaStream_t st) {
  switch (pl.nt) {
    case 1: return run_tiles4<D, 1>(p, pl, st);
    case 2: return run_tiles4<D, 2>(p, pl, st);
    case 3: return run_tiles4<D, 3>(p, pl, st);
    default: break;
  }
  const oscar_status s = run_kv8_rows(p, D, kCodeE2m1, pl.ctas, kMinShare, st);
  if (s != OSCAR_OK) return s;
  return launch_kv8(kv8_merge_rows_kernel<D>, 1, dim3(static_cast<unsigned>(pl.ctas), (std::min(p.cols, 128) + 31) / 32),
                    4 * D, 0, st, p) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // namespace oscar

namespace oscar_host {

oscar_status check_kv4(const oscar_kv4_desc* c, oscar_kv8_desc* as8) {
  if (!c) return OSCAR_ERR_INVALID_ARG;
  *as8 = {c->num_kv_heads, c->num_q_heads, c->head_dim, c->max_pages_per_seq, c->num_pages, c->num_tails,
          c->pool, c->tail, c->page_table, c->tail_ids, c->status, oscar::kCodeInt8};
  const oscar_status s = check_kv8(as8);
  as8->format = oscar::kCodeE2m1;
  return s;
}

}  // namespace oscar_host

using namespace oscar;

extern "C" {

size_t oscar_kv4_workspace_size(const oscar_kv4_desc* desc, int32_t batch, int32_t m_rows,
                                int32_t max_seq_len) {
  oscar_kv8_desc c;
  Kv4Plan pl;
  if (oscar_host::check_kv4(desc, &c) != OSCAR_OK || batch < 1 || m_rows < 1 || max_seq_len < 1 ||
      !kv4_plan(&c, batch, m_rows, max_seq_len, &pl))
    return 0;
  return pl.most;
}

oscar_status oscar_kv4_attention(const oscar_kv4_desc* desc, const void* q, const int32_t* seq_lens,
                                 const int32_t* q_pos, int32_t batch, int32_t m_rows,
                                 int32_t max_seq_len, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  oscar_kv8_desc c;
  oscar_status s = oscar_host::check_kv4(desc, &c);
  if (s != OSCAR_OK) return s;
  bool work;
  s = check_attention(&c, q, seq_lens, q_pos, batch, m_rows, max_seq_len, out, workspace, &work);
  if (s != OSCAR_OK || !work) return s;
  Kv4Plan pl;
  if (!kv4_plan(&c, batch, m_rows, max_seq_len, &pl)) return OSCAR_ERR_UNSUPPORTED;
  if (workspace_bytes < pl.total) return OSCAR_ERR_WORKSPACE;
  const Kv8Params p = attention_params(&c, q, seq_lens, q_pos, m_rows, max_seq_len, out, workspace, pl.tiles,
                                       pl.entries, pl.cluster, pl.team, pl.info);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c.head_dim == 128 ? run_kv4<128>(p, pl, st) : run_kv4<64>(p, pl, st);
}

}  // extern "C"
