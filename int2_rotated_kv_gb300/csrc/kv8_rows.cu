// Attention over the 8-bit cache for many query columns of a KV head (a chunk of
// prefill, a long verification): tiles of 128 (row, query head) columns on tcgen05.
//
// Same mathematics, unit division and partial results as kv8_attention.cu, for the 4-bit cache too (kv4_attention.cu),
// whose operands are code * s.  Per tile
// of 128 tokens (8 pages):
//   S = Q K^T   M = 128 columns of queries, N = 128 tokens, K = d   (Q, K in shared memory)
//   w = 2^(s_K fac S + log2 s_V - m - k)   (a thread per query; kv8_units.cuh has unit and ranges)
//   O += w V    M = 128, N = d, K = 128 tokens      (w in tensor memory, V in shared memory)
// Here the bound is arithmetic, so the codes are turned into fp16 operands once per
// tile and CTA (exact: integers up to 127, or e4m3 values) and the MMAs run from
// shared and tensor memory.  The value scale of a page rides in the exponent: w is
// p s_V, rounded once to fp16, and the sum of p is that of w / s_V.
//
// One CTA per SM, 18 warps:
//   0-3, 4-7      softmax of even and odd tiles ("streams", each with its own S, w, O in
//                 tensor memory, own maxima and sums, merged at the unit's end): reads S
//                 twice, for the maximum and for w, which overwrites S;
//   8-11, 12-15   pages -> fp16 K tiles and V tiles, 128-byte swizzled, two of each, and
//                 the queries of a unit.  A warp has two pages of every tile, whose codes it
//                 holds in registers from one tile to the next.  (As bulk copies of 2 KB, 24 a
//                 tile, the copies alone took 3400 cycles a tile; by cp.async the 65-row case
//                 takes 121 us.)
//   16, 17        MMAs of a stream, from one lane each.
// Every wait is bounded; a CTA that gives up finishes its copies and MMAs first.
// Tensor memory: S0, S1 (128 columns each), O0, O1 (d each); w in the first half of S.
// What bounds it: the latency of its roles.  Per tile of 128 tokens the MMAs take 1024 cycles
// at d = 128 and shared memory 1536 (fp16 tiles written once and read by the MMAs, Q read per
// tile); a tile takes 2400, in which a K warp is busy for 1950 and a stream's chain S, softmax,
// O is longer than its share.  Measured, d = 128, 8 KV heads, G = 4: 2048 rows over 32768 tokens
// 1050 us, 1047 TFLOP/s; 4 sequences x 65 rows over 6000-16385 tokens 86.7 us, 550 TFLOP/s of
// rows that exist (260 columns are 3 tiles: a third of the work is for 4 of them).  4 bits: 1000 rows
// over 17000 tokens 308 us, 905 TFLOP/s.
// Registers: 96 a thread for 18 warps.  Whatever is spilled in a role's loop costs more than
// it saves elsewhere (16 registers' worth: 7 of 98 us), and code that is fetched cold costs its
// fetches, so what runs once per unit is out of line or rolled.
// Tried: one pass over S with the maximum of 32 (16) columns checked before their weights,
// 1895 (1694) us where two passes take 1479, as every check waits for a vote; three V tiles,
// 1420 us for 1185: shared memory that a tile more takes is L1's; setmaxnreg, no gain; value
// codes through a ring of asynchronous copies, 91 us for 86, or asked into L1 two tiles ahead,
// 94; a page's successor requested before the other page is converted, 113.

#include "kv8_units.cuh"
#include "tcgen05.cuh"

namespace oscar {

constexpr int kRWarps = 18;
constexpr int kRThreads = 32 * kRWarps;
constexpr int kRTile = 128;        // tokens of a tile
constexpr int kRHidden = 0x7fff0000;   // position of a page slot that holds no page

template <int D>
struct RowsSmem {
  using F = Kv8Fmt<D>;
  static constexpr int kTile16 = kRTile * D * 2;           // fp16 K or V tile, or Q
  static constexpr int kK = 0;
  static constexpr int kV = 2 * kTile16;
  static constexpr int kQ = 4 * kTile16;
  static constexpr int kMeta = 5 * kTile16;                  // float4 [4][8]: s_K, log2 s_V, 2^-12/s_V, position
  static constexpr int kFac = kMeta + 512;                 // float [2][128]
  static constexpr int kMl = kFac + 1024;                  // float4 [2][2][128]: unit and sum
  static constexpr int kBad = kMl + 8192;                  // int [4]: tails that are not finite
  static constexpr int kOdd = kBad + 16;                   // int [2][2]: see note_odd
  static constexpr int kBars = kBad + 64;
  static constexpr int kMisc = kBars + 40 * 8;
  static constexpr int kBytes = kMisc + 64;
  static constexpr int kAlloc = kBytes + 1024;             // the base is rounded up to 1024 bytes
  static_assert(kMeta % 16 == 0, "metadata is read by 16 bytes");
};

struct RowsBars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];   // fp16 tiles, by tile number
  uint64_t sfull[2], pfull[4], wdone[2];               // S ready, w ready, w used, by stream
  uint64_t qfull[2], oempty[2];                        // by unit: queries ready, O read
  uint64_t qempty, odone, mlfull, last[2];
};
static_assert(sizeof(RowsBars) <= 40 * 8, "barriers fit");

// One unit's pages of this CTA and their tiles.
struct Walk {
  int e, h, p0, p1, n8, tiles;
  bool tail;
  int64_t unit0, end;
  Entry t;

  __device__ __forceinline__ void set() {
    p1 = static_cast<int>(min(static_cast<int64_t>(t.pages), end - unit0));
    n8 = max(0, min(p1, t.n8) - p0);
    tail = p1 > t.n8 && t.vis > t.len / kPage * kPage;
    tiles = (n8 + (tail ? 1 : 0) + 7) / 8;
  }
  __device__ __forceinline__ void start(const Share& s) {
    e = s.e;
    h = s.h;
    t = s.t;
    unit0 = s.unit0;
    end = s.end;
    p0 = static_cast<int>(s.at - s.unit0);
    set();
  }
  __device__ __forceinline__ bool next(const Kv8Params& p) {
    if (unit0 + p1 >= end) return false;
    *this = after(p, *this);
    return true;
  }
  static __device__ __noinline__ Walk after(const Kv8Params& p, Walk u) {
    u.unit0 += u.t.pages;
    if (++u.h == p.hkv) {
      u.h = 0;
      u.t = entry_of<kRowsNT>(p, ++u.e);
    }
    u.p0 = 0;
    u.set();
    return u;
  }
  // The tail's page slot in tile i; -1: none.
  __device__ __forceinline__ int tail_slot(int i) const { return tail && i == tiles - 1 ? n8 - 8 * i : -1; }
};

// Blocks of a unit's pages as a warp holds them: four tiles' (32 pages), a lane each, and the
// next four's page ids on their way.
struct PageBlocks {
  const int32_t* row;
  int now, ahead;   // -1: no page, or (in `now`) an id out of range

  __device__ __forceinline__ PageBlocks(const Kv8Params& p, const Walk& u, int lane) {
    row = p.page_table + static_cast<size_t>(u.t.b) * p.max_pages + u.p0;
    now = -1;
    ahead = lane < u.n8 ? row[lane] : -1;
  }
  // to be called for every tile in order
  __device__ __forceinline__ void tile(const Kv8Params& p, const Walk& u, int i, int lane) {
    if (i % 4) return;
    const bool ok = ahead >= 0 && ahead < p.n_pages;
    if (!ok && 8 * i + lane < u.n8 && p.status) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
    now = ok ? ahead * p.hkv + u.h : -1;   // (2^31 blocks are more than a cache can have)
    const int pg = 8 * i + 32 + lane;
    ahead = pg < u.n8 ? row[pg] : -1;
  }
  __device__ __forceinline__ int block(int i, int slot) const {
    return __shfl_sync(0xffffffffu, now, (8 * i + slot) & 31);
  }
};

// 16 bytes; volatile: where it stands, well ahead of its use.
__device__ __forceinline__ uint4 load16(const uint8_t* src) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "l"(src));
  return x;
}

__device__ __forceinline__ uint2 load8(const uint8_t* src) {
  uint2 x;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n" : "=r"(x.x), "=r"(x.y) : "l"(src));
  return x;
}

// Four codes as fp16 pairs in order, exact.
template <bool kE4m3>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (kE4m3) {
    kv8_operands<true>(w, a, b);
  } else {   // 1024 + code + 128 as fp16 bytes, less 1152
    const __half2 less = __floats2half2_rn(-1152.f, -1152.f);
    const uint32_t x = __byte_perm(w, 0x64646464u, 0x4140), y = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 s = __hadd2(*reinterpret_cast<const __half2*>(&x), less);
    const __half2 t = __hadd2(*reinterpret_cast<const __half2*>(&y), less);
    a = *reinterpret_cast<const uint32_t*>(&s);
    b = *reinterpret_cast<const uint32_t*>(&t);
  }
}

// A lane's chunk c of a page's key codes is chunk 32 c + lane (a load of 16 bytes a lane reads
// 512 in a row): token 2 (lane / 4) + c % 2, channels 16 (lane % 4) + 64 (c / 2) and on.  Its
// place in the page's 16 rows of the swizzled tile; half: 8 channels of it.  Every other four
// lanes store their halves in the other order, so that the eight of a store phase, in two
// rows, meet all the banks.
__device__ __forceinline__ uint32_t key_place(int lane, int c, int half) {
  const int t = 2 * (lane >> 2) + (c & 1);
  return (c >> 1) * (kRTile * 128) + 128 * t + 16 * ((2 * (lane & 3) + half) ^ (t & 7));
}

template <bool kE4m3>
__device__ __forceinline__ void store_keys(uint8_t* dst, int c, int lane, uint4 x) {
  const int turn = (lane >> 2) & 1;
  uint32_t o[8];
  code_pairs<kE4m3>(turn ? x.z : x.x, o[0], o[1]);
  code_pairs<kE4m3>(turn ? x.w : x.y, o[2], o[3]);
  code_pairs<kE4m3>(turn ? x.x : x.z, o[4], o[5]);
  code_pairs<kE4m3>(turn ? x.y : x.w, o[6], o[7]);
  *reinterpret_cast<uint4*>(dst + key_place(lane, c, turn)) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(dst + key_place(lane, c, turn ^ 1)) = make_uint4(o[4], o[5], o[6], o[7]);
}

// Its chunk c of value codes: channels 32 c + 4 (lane / 4) and on, tokens 4 (lane % 4) and on.
// Where four tokens of the channel that it stores k-th lie, as fp16, in a 64-token atom's rows
// (channels), page slot w of four.  Every other pair of channel groups stores its channels in
// the order 2, 3, 0, 1, for the banks as above.
__device__ __forceinline__ int value_channel(int lane, int k) { return k ^ ((lane >> 2) & 2); }
__device__ __forceinline__ uint32_t value_place(int lane, int c, int w, int k) {
  const int ch = 4 * (lane >> 2) + value_channel(lane, k), tg = lane & 3;
  return (32 * c + ch) * 128 + 16 * ((2 * w + (tg >> 1)) ^ (ch & 7)) + 8 * (tg & 1);
}

template <bool kE4m3>
__device__ __forceinline__ void store_values(uint8_t* dst, int c, int w, int lane, uint4 x) {
  const bool turn = value_channel(lane, 0);
  const uint32_t in[4] = {turn ? x.z : x.x, turn ? x.w : x.y, turn ? x.x : x.z, turn ? x.y : x.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint2 o;
    code_pairs<kE4m3>(in[k], o.x, o.y);
    *reinterpret_cast<uint2*>(dst + value_place(lane, c, w, k)) = o;
  }
}

// A lane's chunk j of a page's 4-bit key codes, tokens 2 (lane / 4) and that + 1, channels 64 j + 16 (lane % 4)
// and on, times the scales of the channels: chunks 2 j and 2 j + 1 of the 8-bit order.
__device__ __forceinline__ void store_keys4(uint8_t* dst, int j, int lane, uint4 x, uint4 sc) {
  const int turn = (lane >> 2) & 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {   // 8 channels of both tokens, the other 8
    const int half = turn ^ k;
    uint32_t s[4];
    kv4_scales(half ? sc.z : sc.x, s[0], s[1]);
    kv4_scales(half ? sc.w : sc.y, s[2], s[3]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t o[4];
      kv4_pairs(half ? (e ? x.w : x.y) : (e ? x.z : x.x), o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dst + key_place(lane, 2 * j + e, half)) =
          make_uint4(hmul2_u32(o[0], s[0]), hmul2_u32(o[1], s[1]), hmul2_u32(o[2], s[2]), hmul2_u32(o[3], s[3]));
    }
  }
}

// Its chunk i of 4-bit value codes, tokens 4 (lane % 4) and on, channels 64 i + 4 (lane / 4) and on and those 32 further:
// chunks 2 i and 2 i + 1 of the 8-bit order.
__device__ __forceinline__ void store_values4(uint8_t* dst, int i, int w, int lane, uint4 x, uint2 sc) {
  const bool turn = value_channel(lane, 0);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t s01, s23;
    kv4_scales(half ? sc.y : sc.x, s01, s23);
    const uint32_t lo = half ? x.z : x.x, hi = half ? x.w : x.y;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      uint32_t o[4];
      kv4_pairs(turn != (k != 0) ? hi : lo, o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint2*>(dst + value_place(lane, 2 * i + half, w, k)) =
          make_uint2(hmul2_u32(o[0], s01), hmul2_u32(o[1], s23));
      *reinterpret_cast<uint2*>(dst + value_place(lane, 2 * i + half, w, k + 1)) =
          make_uint2(hmul2_u32(o[2], s01), hmul2_u32(o[3], s23));
    }
  }
}

__device__ __forceinline__ uint32_t half_pair(uint32_t w, float mul) {
  return pack_half2(bf16_lo_value(w) * mul, bf16_hi_value(w) * mul);
}

// The largest finite magnitude in a tail's values (which: 0 keys, 1 values) among its
// first n tokens, by one warp from global memory; bad: something there is not finite.
template <int D>
__device__ __forceinline__ uint32_t tail_magnitude(const uint16_t* area, int which, int n, int lane,
                                                   bool& bad) {
  uint32_t top = 0;
  bool odd = false;
#pragma unroll 1
  for (int c = lane; c < D; c += 32) {   // chunks of 16 elements
    const uint4* s = reinterpret_cast<const uint4*>(area + 16 * c);
    const uint4 a = s[0], b = s[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // the tokens of the two halves of word i
      const int t0 = which ? 4 * (c & 3) + 2 * (i & 1) : 2 * ((c & 31) >> 2) + ((c >> 5) & 1);
      const int t1 = which ? t0 + 1 : t0;
      const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
      if (t0 < n) {
        if (lo < 0x7f80u) top = max(top, lo); else odd = true;
      }
      if (t1 < n) {
        if (hi < 0x7f80u) top = max(top, hi); else odd = true;
      }
    }
  }
  bad = __any_sync(0xffffffffu, odd);
  return __reduce_max_sync(0xffffffffu, top);
}

// The tail's element block (keys, then values) of a unit; ok: its id is in range.
template <int D>
__device__ __forceinline__ const uint16_t* tail_block(const Kv8Params& p, int b, int h, bool& ok) {
  const int64_t id = p.tail_ids ? p.tail_ids[b] : b;
  ok = id >= 0 && id < p.n_tails;
  return reinterpret_cast<const uint16_t*>(p.tail) + ((ok ? id : 0) * p.hkv + h) * (2 * Kv8Fmt<D>::kTailHalf);
}

// The tail's keys as 16 fp16 rows at dst, scaled by a power of two; returns what the softmax
// needs of the slot, and sets *bad when a value there is not finite.  Once per unit.
template <int D>
__device__ __noinline__ float4 tail_keys(const Kv8Params& p, int b, int h, int len, uint8_t* dst,
                                         int lane, volatile int* bad) {
  bool ok, odd;
  const uint16_t* area = tail_block<D>(p, b, h, ok);
  const int n = len % kPage;
  const int up = scale_up(tail_magnitude<D>(area, 0, n, lane, odd));
  const uint32_t top_v = tail_magnitude<D>(area + Kv8Fmt<D>::kTailHalf, 1, n, lane, odd);
  const int up_v = top_v ? scale_up(top_v) : static_cast<int>(-kZeroLog2);
  const float mul = power_of_two(up);
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const uint4 x = reinterpret_cast<const uint4*>(area)[2 * (32 * c + lane) + half];
      *reinterpret_cast<uint4*>(dst + key_place(lane, c, half)) =
          make_uint4(half_pair(x.x, mul), half_pair(x.y, mul), half_pair(x.z, mul), half_pair(x.w, mul));
    }
  }
  if (lane == 0) {
    *bad = odd && ok;
    if (!ok && p.status) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
  }
  return make_float4(power_of_two(-up), static_cast<float>(-up_v), power_of_two(up_v) * kSumUnit,
                     __int_as_float(ok ? len / kPage * kPage : kRHidden));
}

// The tail's values into page slot w of the atom at dst; what is not finite, or not a token,
// becomes 0 (the epilogue adds the former).
template <int D>
__device__ __noinline__ void tail_values(const Kv8Params& p, int b, int h, int len, uint8_t* dst, int w,
                                        int lane) {
  bool ok, odd;
  const uint16_t* area = tail_block<D>(p, b, h, ok) + Kv8Fmt<D>::kTailHalf;
  const int n = len % kPage;
  const float mul = power_of_two(scale_up(tail_magnitude<D>(area, 1, n, lane, odd)));
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      const uint16_t* four = area + 16 * (32 * c + lane) + 4 * value_channel(lane, k);
      uint2 x = *reinterpret_cast<const uint2*>(four);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t& v = j < 2 ? x.x : x.y;
        const uint32_t mask = j & 1 ? 0xffff0000u : 0xffffu;
        if (4 * (lane & 3) + j >= n || (v & mask & 0x7fff7fffu) >= (0x7f807f80u & mask)) v &= ~mask;
      }
      *reinterpret_cast<uint2*>(dst + value_place(lane, c, w, k)) = make_uint2(half_pair(x.x, mul), half_pair(x.y, mul));
    }
  }
}

// The largest finite magnitude of a column's part; out of line, as nearly never needed.
template <int kWords>
__device__ __noinline__ uint32_t finite_magnitude(const uint4* src) {
  uint32_t top = 0;
#pragma unroll 1
  for (int i = 0; i < 8 * kWords; ++i) {
    const uint32_t x = reinterpret_cast<const uint16_t*>(src)[i] & 0x7fffu;
    if (x < 0x7f80u) top = max(top, x);
  }
  return top;
}

// Sixteen query columns of a unit (the w-th of eight parts) as fp16 rows of the operand at
// dst, each scaled by a power of two; facs gets what a logit in the log2 domain is per unit of
// S.  Two lanes a column, all their loads in flight at once.
template <int D>
__device__ __noinline__ void load_queries(const Kv8Params& p, int b, int h, int tile, int w, int lane,
                                          uint8_t* dst, float* facs) {
  constexpr int kWords = D / 16;   // 16-byte words of a lane
  const int rr = 16 * w + (lane >> 1), part = lane & 1, col = tile * 128 + rr;
  const int row = col / p.G, g = col - row * p.G;
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + ((static_cast<size_t>(b) * p.m_rows + row) * p.hq + h * p.G + g) * D) + part * kWords;
  uint4 q[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) q[i] = col < p.cols ? src[i] : make_uint4(0, 0, 0, 0);
  uint32_t pair = 0;   // magnitudes as pairs of 16-bit integers
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    pair = __vmaxu2(__vmaxu2(__vmaxu2(pair, q[i].x & 0x7fff7fffu), __vmaxu2(q[i].y & 0x7fff7fffu, q[i].z & 0x7fff7fffu)),
                    q[i].w & 0x7fff7fffu);
  uint32_t top = max(pair & 0xffffu, pair >> 16);
  if (top >= 0x7f80u) top = finite_magnitude<kWords>(src);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  const int up = scale_up(top);
  const float mul = power_of_two(up);
  if (part == 0) facs[rr] = p.scale_log2 * power_of_two(-up);
#pragma unroll
  for (int i = 0; i < kWords; ++i)
    *reinterpret_cast<uint4*>(dst + tc_sw128_offset(rr, 8 * (part * kWords + i), kRTile)) =
        make_uint4(half_pair(q[i].x, mul), half_pair(q[i].y, mul), half_pair(q[i].z, mul), half_pair(q[i].w, mul));
}

// 2^x; unlike fast_exp2 free to move among its neighbours.
__device__ __forceinline__ float rows_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;\n" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The largest exponent s_K fac S + log2 s_V of a thread's row over a tile's visible tokens.
// Two pages' 32 columns at a time, the next two pages' on their way.  kCareful: where the tile has a
// token that a row does not see, the unit odd scales (note_odd), or a row a steep maximum (kSteep).
template <bool kCareful>
__device__ __forceinline__ float rows_max(uint32_t ts, const float4* mt, float fac, int vis) {
  float big = -INFINITY;
  auto pages = [&](const uint32_t (&s)[32], int j0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 pm = mt[j0 + j];
      const int seen = vis - __float_as_int(pm.w);
      float x[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = !kCareful || k < seen ? __uint_as_float(s[16 * j + k]) : -INFINITY;
#pragma unroll
      for (int k = 0; k < 5; ++k) x[k] = max3(x[k], x[k + 5], x[k + 10]);
      const float top = fmaxf(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[15]));
      // (a hidden page's -inf times a scale of 0 would be NaN)
      big = fmaxf(big, kCareful && top == -INFINITY ? top : fmaf(top, kCareful ? logit_factor(pm.x, fac) : pm.x * fac, pm.y));
    }
  };
  uint32_t a[32], b[32];
  tc_request32(ts, a);
#pragma unroll 1
  for (int j = 0; j < 8; j += 4) {
    tc_wait_ld(a);
    tc_request32(ts + 16 * j + 32, b);
    pages(a, j);
    tc_wait_ld(b);
    tc_request32(ts + (j == 0 ? 64 : 0), a);   // (the last one is not looked at)
    pages(b, j + 2);
  }
  tc_wait_ld(a);
  return big;
}

// w = 2^(s_K fac S + log2 s_V - m - k) of the row, as fp16 over the columns of S that have been
// read; returns the sum of w / s_V.  Where |m| is at most kSteep, log2 s_V - m is off by 2^-14 at most
// as one number (and k is 0); else logits are rounded by themselves, so that equal ones stay equal.
template <bool kCareful>
__device__ __forceinline__ float rows_weights(uint64_t* half, uint32_t ts, const float4* mt, float fac, int vis, Unit un) {
  float l = 0.f;
  auto pages = [&](const uint32_t (&s)[32], int j0) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t out[8];
      const float4 pm = mt[j0 + j];
      const float f = kCareful ? logit_factor(pm.x, fac) : pm.x * fac, off = pm.y - (kCareful ? un.k : un.m);
      const uint64_t f2 = two(f, f), off2 = two(off, off), m2 = two(-un.m, -un.m);
      const int seen = vis - __float_as_int(pm.w);
      uint64_t sum[2];
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float s0 = __uint_as_float(s[16 * j + k]), s1 = __uint_as_float(s[16 * j + k + 1]);
        const uint64_t e = kCareful ? add2(add2(two(__fmul_rn(s0, f), __fmul_rn(s1, f)), m2), off2)
                                    : fma2(two(s0, s1), f2, off2);
        float x0 = rows_exp2(first(e)), x1 = rows_exp2(second(e));
        if constexpr (kCareful) {
          x0 = k < seen ? x0 : 0.f;
          x1 = k + 1 < seen ? x1 : 0.f;
        }
        const uint64_t x = two(x0, x1);
        sum[(k >> 1) & 1] = k < 4 ? x : add2(sum[(k >> 1) & 1], x);
        out[k / 2] = pack_half2(x0, x1);
      }
      tc_st8(ts + 8 * (j0 + j), out);
      const uint64_t all = add2(sum[0], sum[1]);
      if (!kCareful || seen > 0) l = fmaf(first(all) + second(all), pm.z, l);
    }
  };
  uint32_t a[32], b[32];
  tc_request32(ts, a);
#pragma unroll 1
  for (int j = 0; j < 8; j += 4) {
    tc_wait_ld(a);
    tc_request32(ts + 16 * j + 32, b);
    pages(a, j);
    tc_wait_ld(b);
    tc_request32(ts + (j == 0 ? 64 : 0), a);   // (the last one is not looked at)
    pages(b, j + 2);
    if (j == 0) {
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) tc_arrive(half);
    }
  }
  tc_wait_ld(a);
  return l;
}

// Unit `seg` has a value scale outside the window of is_odd, or keys whose scale times a column's
// factor (2^110 at most) may overflow: its number into the first word of two, and into the second for a
// scale above the window.  Two units' words, as the pages are ahead of the softmax by one.
constexpr float kOddKeys = 131072.f;
static __device__ __noinline__ void note_odd(volatile int* odd_scale, uint32_t seg, float log2_scale) {
  volatile int* odd = odd_scale + 2 * (seg & 1);
  if (log2_scale > 0.f) odd[1] = static_cast<int>(seg) + 1;
  odd[0] = static_cast<int>(seg) + 1;
}

// p of the row's visible tokens whose weights underflow in rows_weights, times 2^kSumLog2: for
// units with odd scales; high: one above the window of is_odd, else only pages below it can
// lose any.  The same exponents as there, so each token counts once.
__device__ __forceinline__ float rows_lost(uint32_t ts, const float4* mt, float fac, int vis, float m, float k, bool high) {
  float l = 0.f;
#pragma unroll 1
  for (int j = 0; j < 8; ++j) {
    const float4 pm = mt[j];
    if (!high && !is_odd(pm.y)) continue;   // (the same for all lanes)
    const float f = logit_factor(pm.x, fac), off = pm.y - k;
    const int seen = vis - __float_as_int(pm.w);
    uint32_t s[16];
    tc_request16(ts + 16 * j, s);
    tc_wait_ld(s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = __fmul_rn(__uint_as_float(s[i]), f) - m;
      if (i < seen && rows_exp2(x + off) == 0.f) l += whole_exp2(x - k + static_cast<float>(kSumLog2));
    }
  }
  return l;
}

// The unit that a row's visible tokens of a tile need: their largest logit, and the largest
// logit + log2 s_V less that.
__device__ __forceinline__ Unit steep_max(uint32_t ts, const float4* mt, float fac, int vis) {
  Unit u{-INFINITY, 0.f};
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    float best = -INFINITY;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      const float4 pm = mt[j];
      const int seen = vis - __float_as_int(pm.w);
      uint32_t s[16];
      tc_request16(ts + 16 * j, s);
      tc_wait_ld(s);
      float raw = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < seen) raw = fmaxf(raw, __uint_as_float(s[i]));
      if (raw > -INFINITY) raw = __fmul_rn(raw, logit_factor(pm.x, fac));
      best = fmaxf(best, pass == 0 ? raw : (raw - u.m) + pm.y);
    }
    if (pass == 0) u.m = best;
    else u.k = u.m == -INFINITY ? 0.f : best;
  }
  return u;
}

// A row's O in tensor memory times a.
template <int D>
__device__ __forceinline__ void rescale_output(uint32_t to, float a) {
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t o[16];
    tc_request16(to + 16 * c, o);
    tc_wait_ld(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
    tc_st16(to + 16 * c, o);
  }
}

struct RowState {
  float m, k, l;   // unit and sum
};
// A row's unit and sum before the weights of a tile of an odd unit, or of one with a steep row.  (Out of
// line: in line it costs the common path 1 to 2% in registers.)
enum { kBegun = 1, kIsSteep = 2, kIsOdd = 4, kIsHigh = 8 };
template <int D>
__device__ __noinline__ RowState settle(RowState r, float big, uint32_t ts, uint32_t to, const float4* mt, float fac,
                                        int vis, int what) {
  Unit next{big, 0.f};
  if (what & kIsSteep) next = steep_max(ts, mt, fac, vis);
  const float x = above(Unit{r.m, r.k}, next.m, next.k);
  const bool over = x > kLag;
  const float half = over ? rows_exp2(-0.5f * x) : 1.f, a = half * half;
  if (over) {
    r.m = next.m;
    r.k = next.k;
  }
  r.l = r.l * half * half;
  if ((what & kBegun) && __any_sync(0xffffffffu, over)) rescale_output<D>(to, a);
  if (what & kIsOdd) r.l += rows_lost(ts, mt, fac, vis, r.m, r.k, what & kIsHigh);
  return r;
}

template <int D, int kCode>
__global__ void __launch_bounds__(kRThreads, 1)
kv8_rows_kernel(const __grid_constant__ Kv8Params p, int min_share) {
  using S = RowsSmem<D>;
  using F = KvFmt<D, kCode>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  RowsBars* bar = reinterpret_cast<RowsBars*>(smem + S::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  float4* meta = reinterpret_cast<float4*>(smem + S::kMeta);
  float* facs = reinterpret_cast<float*>(smem + S::kFac);
  float4* mls = reinterpret_cast<float4*>(smem + S::kMl);
  volatile int* bad_tail = reinterpret_cast<volatile int*>(smem + S::kBad);
  volatile int* odd_scale = reinterpret_cast<volatile int*>(smem + S::kOdd);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->kfull[i], 4);
      mbar_init(&bar->kempty[i], 1);
      mbar_init(&bar->vfull[i], 4);
      mbar_init(&bar->vempty[i], 1);
      mbar_init(&bar->sfull[i], 1);
      mbar_init(&bar->pfull[i], 4);
      mbar_init(&bar->pfull[2 + i], 4);
      mbar_init(&bar->wdone[i], 1);
      mbar_init(&bar->last[i], 1);
      mbar_init(&bar->qfull[i], 8);
      mbar_init(&bar->oempty[i], 8);
    }
    mbar_init(&bar->qempty, 2);
    mbar_init(&bar->odone, 2);
    mbar_init(&bar->mlfull, 8);
    *abort_flag = 0;
    for (int i = 0; i < 4; ++i) odd_scale[i] = 0;
    fence_mbar_init();
  }
  if (warp == 16) tc_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  bool any;
  const Share sh = find_share<kRowsNT, kRWarps>(p, min_share, any);
  if (!any && tid == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
  Walk u;
  if (any) u.start(sh);
  // A wait of a warp together (one answer for all lanes); false: give up.
  // No barrier completes a second phase before all that wait for the first have passed.
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    const bool ok = __all_sync(0xffffffffu, wait_copy(b, parity & 1u, p.status) && !*abort_flag);
    if (!ok) *abort_flag = 1;
    return ok;
  };
  auto arrive = [&](uint64_t* b) {
    __syncwarp();
    if (lane == 0) tc_arrive(b);
  };

  if (any && (warp == 16 || warp == 17)) {
    // ------------------------------------------------------------------ MMAs
    // a stream's, so that neither waits behind the other; lane 0 issues
    constexpr uint32_t id_s = tc_idesc_f16(kRTile, kRTile), id_o = tc_idesc_f16(kRTile, D);
    constexpr int kAtom = kRTile * 128;   // 64 channels of K or Q
    constexpr int kAtomV = D * 128;       // 64 tokens of V
    const int st = __shfl_sync(0xffffffffu, warp, 0) - 16;   // (known to be one for the warp)
    const bool leader = tc_elect();
    uint32_t g0 = 0, seg = 0;             // tiles before this unit, units with tiles
    uint32_t count = 0;                   // tiles of the stream whose O has been issued
    bool ok = true;
    for (bool go = true; go && ok; go = u.next(p)) {
      if (u.tiles == 0) continue;
      if (!(ok = wait(&bar->qfull[seg & 1], seg >> 1))) break;
      for (int i = st; i < u.tiles && ok; i += 2) {
        const uint32_t g = g0 + i, buf = __shfl_sync(0xffffffffu, g & 1, 0);
        // S of the tile, once w of the stream's tile before, which lies in it, has been used
        ok = wait(&bar->kfull[buf], g >> 1) && (count == 0 || wait(&bar->wdone[st], count - 1));
        if (!ok) break;
        if (leader) {
          tc_fence_after();
          const uint32_t a0 = sb + S::kQ, b0 = sb + S::kK + buf * S::kTile16;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kAtom + (kk & 3) * 32;
            tc_mma(tmem + st * kRTile, tc_desc_sw128(a0 + off), tc_desc_sw128(b0 + off), id_s, kk != 0);
          }
          tc_commit(&bar->sfull[st]);
          tc_commit(&bar->kempty[buf]);
        }
        __syncwarp();
        // O, once the unit before has been read
        ok = wait(&bar->pfull[st], count) && wait(&bar->vfull[buf], g >> 1) &&
             (i > 1 || seg == 0 || wait(&bar->oempty[(seg - 1) & 1], (seg - 1) >> 1));
        if (!ok) break;
        ++count;
        const int later = __shfl_sync(0xffffffffu, i > 1 ? 1 : 0, 0);
        if (leader) {
          tc_fence_after();
          const uint32_t v0 = sb + S::kV + buf * S::kTile16;
#pragma unroll
          for (int kk = 0; kk < kRTile / 32; ++kk)
            tc_mma_ts(tmem + 2 * kRTile + st * D, tmem + st * kRTile + 8 * kk,
                      tc_desc_sw128(v0 + (kk >> 2) * kAtomV + (kk & 3) * 32), id_o, kk != 0 || later);
        }
        __syncwarp();
        ok = wait(&bar->pfull[2 + st], count - 1);
        if (!ok) break;
        if (leader) {
          tc_fence_after();
          const uint32_t v0 = sb + S::kV + buf * S::kTile16;
#pragma unroll
          for (int kk = kRTile / 32; kk < kRTile / 16; ++kk)
            tc_mma_ts(tmem + 2 * kRTile + st * D, tmem + st * kRTile + 8 * kk,
                      tc_desc_sw128(v0 + (kk >> 2) * kAtomV + (kk & 3) * 32), id_o, 1);
          tc_commit(&bar->vempty[buf]);
          tc_commit(&bar->wdone[st]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (leader) {   // the stream's MMAs of the unit: its queries may go, its O is complete
        tc_commit(&bar->qempty);
        tc_commit(&bar->odone);
      }
      __syncwarp();
      g0 += u.tiles;
      ++seg;
    }
    if (!ok && leader) {   // MMAs in flight finish before the CTA ends
      tc_commit(&bar->last[st]);
      mbar_wait(&bar->last[st], 0, p.status);
    }
  } else if (any && warp >= 12 && warp < 16) {
    // ---------------------------------------------------- values as fp16 operands
    const int w = warp - 12;   // page slots w and w + 4 of every tile
    uint32_t g = 0, seg = 0;
    for (bool go = true, ok = true; go && ok; go = u.next(p)) {
      if (u.tiles == 0) continue;
      PageBlocks blocks(p, u, lane);
      constexpr int kChunks = F::kCodes / 512;   // 16 bytes a lane
      uint4 x[2][kChunks];
      uint2 vs[2][kCode == kCodeE2m1 ? kChunks : 1];   // their scales (4 bits)
      // the codes of this warp's pages of tile i
      auto request = [&](int i) {
        blocks.tile(p, u, i, lane);
        const int b[2] = {blocks.block(i, w), blocks.block(i, w + 4)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* src = p.pool + static_cast<int64_t>(b[half]) * F::kBlock + F::kCodes + 16 * lane;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) x[half][c] = b[half] >= 0 ? load16(src + 512 * c) : make_uint4(0, 0, 0, 0);
          if constexpr (kCode == kCodeE2m1) {
            const uint8_t* sc = p.pool + static_cast<int64_t>(b[half]) * F::kBlock + F::kValueScales +
                32 * (lane >> 4) + 8 * (lane & 3);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) vs[half][c] = b[half] >= 0 ? load8(sc + 64 * c) : make_uint2(0, 0);
          }
        }
      };
      if (!wait(&bar->qempty, seg + 1)) break;
      if (seg > 1 && !wait(&bar->oempty[seg & 1], (seg - 2) >> 1)) break;
      load_queries<D>(p, u.t.b, u.h, u.t.tile, 4 + w, lane, smem + S::kQ, facs + (seg & 1) * 128);
      fence_proxy_async();
      arrive(&bar->qfull[seg & 1]);
      request(0);   // (earlier, it would be spilled around the queries: 7 us of 98)
      for (int i = 0; i < u.tiles; ++i, ++g) {
        const uint32_t buf = g & 1;
        uint8_t* dst = smem + S::kV + buf * S::kTile16;
        if (!(ok = wait(&bar->vempty[buf], (g >> 1) + 1))) break;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if constexpr (kCode == kCodeE2m1) store_values4(dst + half * (D * 128), c, w, lane, x[half][c], vs[half][c]);
            else store_values<kCode == kCodeE4m3>(dst + half * (D * 128), c, w, lane, x[half][c]);
          }
        const int slot = u.tail_slot(i);
        if (i + 1 < u.tiles) {
          request(i + 1);
        } else if (slot >= 0 && (slot & 3) == w) {   // over the zeros that stood for it
          __syncwarp();
          tail_values<D>(p, u.t.b, u.h, u.t.len, dst + (slot >> 2) * (D * 128), w, lane);
        }
        fence_proxy_async();
        arrive(&bar->vfull[buf]);
      }
      ++seg;
    }
  } else if (any && warp >= 8 && warp < 12) {
    // ------------------------------------------- queries and keys as fp16 operands
    const int w = warp - 8;   // page slots w and w + 4 of every tile
    uint32_t g = 0, seg = 0;
    for (bool go = true, ok = true; go && ok; go = u.next(p)) {
      if (u.tiles == 0) continue;
      PageBlocks blocks(p, u, lane);
      constexpr int kChunks = F::kCodes / 512;   // 16 bytes a lane
      uint4 x[2][kChunks];
      uint4 ks[2][kCode == kCodeE2m1 ? kChunks : 1];   // their scales (4 bits)
      float2 sc;      // lanes 0 and 1: scales of the two pages
      bool shown;     // and whether there is one
      // codes and scales of this warp's pages of tile i
      auto request = [&](int i) {
        blocks.tile(p, u, i, lane);
        const int b[2] = {blocks.block(i, w), blocks.block(i, w + 4)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint8_t* src = p.pool + static_cast<int64_t>(b[half]) * F::kBlock + 16 * lane;
#pragma unroll
          for (int c = 0; c < kChunks; ++c) x[half][c] = b[half] >= 0 ? load16(src + 512 * c) : make_uint4(0, 0, 0, 0);
          if constexpr (kCode == kCodeE2m1) {
            const uint8_t* s = p.pool + static_cast<int64_t>(b[half]) * F::kBlock + F::kKeyScales + 16 * (lane & 3);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) ks[half][c] = b[half] >= 0 ? load16(s + 64 * c) : make_uint4(0, 0, 0, 0);
          }
        }
        const int mine = lane ? b[1] : b[0];
        shown = mine >= 0;
        if (lane < 2 && shown)
          sc = __ldg(reinterpret_cast<const float2*>(p.pool + static_cast<int64_t>(mine) * F::kBlock + F::kScales));
      };
      if (!wait(&bar->qempty, seg + 1)) break;
      // and the unit before the last has been read (what is kept by unit comes round again)
      if (seg > 1 && !wait(&bar->oempty[seg & 1], (seg - 2) >> 1)) break;
      load_queries<D>(p, u.t.b, u.h, u.t.tile, w, lane, smem + S::kQ, facs + (seg & 1) * 128);
      fence_proxy_async();
      arrive(&bar->qfull[seg & 1]);
      request(0);   // (earlier, it would be spilled around the queries: 7 us of 98)
      for (int i = 0; i < u.tiles; ++i, ++g) {
        const uint32_t buf = g & 1;
        uint8_t* dst = smem + S::kK + buf * S::kTile16 + 2048 * w;
        if (!(ok = wait(&bar->kempty[buf], (g >> 1) + 1))) break;
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            if constexpr (kCode == kCodeE2m1) store_keys4(dst + 8192 * half, c, lane, x[half][c], ks[half][c]);
            else store_keys<kCode == kCodeE4m3>(dst + 8192 * half, c, lane, x[half][c]);
          }
        if (lane < 2) {   // what the softmax needs of the two pages
          const int slot = 4 * lane + w;
          const float scale = fmaxf(sc.y, kZeroScale), off = fast_log2(scale);
          meta[(g & 3) * 8 + slot] =
              shown ? make_float4(sc.x, off, fast_inverse(scale) * kSumUnit,
                                  __int_as_float((u.p0 + 8 * i + slot) * kPage))
                    : make_float4(0.f, -INFINITY, 0.f, __int_as_float(kRHidden));   // weight 0 without a mask
          if (shown && (is_odd(off) || sc.x > kOddKeys)) note_odd(odd_scale, seg, off);
        }
        const int slot = u.tail_slot(i);
        if (i + 1 < u.tiles) {
          request(i + 1);
        } else if (slot >= 0 && (slot & 3) == w) {   // over the zeros that stood for it
          __syncwarp();
          const float4 m = tail_keys<D>(p, u.t.b, u.h, u.t.len, dst + 8192 * (slot >> 2), lane, bad_tail + (seg & 3));
          if (lane == 0) {
            meta[(g & 3) * 8 + slot] = m;
            if (is_odd(m.y) || m.x > kOddKeys) note_odd(odd_scale, seg, m.y);
          }
        }
        fence_proxy_async();
        arrive(&bar->kfull[buf]);
      }
      ++seg;
    }
  } else if (any && warp < 8) {
    // --------------------------------------------------------------- softmax
    const int st = warp >> 2;                      // stream: even or odd tiles
    const int rr = 32 * (warp & 3) + lane;         // query column of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const uint32_t ts = lanes + st * kRTile, to = lanes + 2 * kRTile + st * D;
    uint32_t g0 = 0, seg = 0, count = 0;
    int4 owned = make_int4(0, 0, 0, 0);
    for (bool go = true; go; go = u.next(p)) {
      const int gcol = u.t.tile * 128 + rr;
      const int row = gcol < p.cols ? gcol / p.G : 0;
      int vis = kRHidden;   // a column that does not exist hides nothing that is there
      if (gcol < p.cols) vis = p.q_pos ? row_limit(p, u.t.b, row, u.t.len) : u.t.len;
      if (u.p0 == 0 && u.h == 0 && p.status && st == 0) {
        const int len = p.seq_lens[u.t.b];
        if (u.t.tile == 0 && rr == 0 && (len < 0 || len > p.max_len))
          atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
        if (p.q_pos && gcol < p.cols && p.q_pos[static_cast<size_t>(u.t.b) * p.m_rows + row] >= u.t.len)
          atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
      }
      RowState r{kLowest, 0.f, 0.f};
      Unit top{kLowest, 0.f};
      float a0 = 0.f, a1 = 0.f;
      if (u.tiles > 0) {
        if (!wait(&bar->qfull[seg & 1], seg >> 1)) break;
        const float fac = facs[(seg & 1) * 128 + rr];
        const bool idle = __all_sync(0xffffffffu, gcol >= p.cols);
        int vis_least = __reduce_min_sync(0xffffffffu, vis);   // -1 once a row's maximum is steep
        const int unit = static_cast<int>(seg) + 1;
        const volatile int* odd = odd_scale + 2 * (seg & 1);
        bool ok = true;
        for (int i = st; i < u.tiles; i += 2) {
          if (!(ok = wait(&bar->sfull[st], count))) break;
          ++count;
          tc_fence_after();
          const float4* mt = meta + ((g0 + i) & 3) * 8;
          if (idle) {   // no column of this warp exists: its rows of w and O may hold anything
            tc_fence_before();
            arrive(&bar->pfull[st]);
            arrive(&bar->pfull[2 + st]);
            continue;
          }
          const bool is_odd_unit = __any_sync(0xffffffffu, odd[0] == unit);   // (one answer for all lanes)
          const bool careful = (u.p0 + 8 * i + 8) * kPage > vis_least || is_odd_unit;   // (always with a tail)
          const float big = careful ? rows_max<true>(ts, mt, fac, vis) : rows_max<false>(ts, mt, fac, vis);
          const bool over = big - r.m > kLag;
          if (__any_sync(0xffffffffu, over) || is_odd_unit || vis_least < 0) {
            if (__any_sync(0xffffffffu, over && fabsf(big) > kSteep)) vis_least = -1;
            if (is_odd_unit || vis_least < 0) {
              r = settle<D>(r, big, ts, to, mt, fac, vis,
                            (i > 1 ? kBegun : 0) | (vis_least < 0 ? kIsSteep : 0) | (is_odd_unit ? kIsOdd : 0) |
                                (__any_sync(0xffffffffu, odd[1] == unit) ? kIsHigh : 0));
            } else {   // (k is 0)
              const float half = over ? rows_exp2(0.5f * (r.m - big)) : 1.f;
              r.m = over ? big : r.m;
              r.l = r.l * half * half;
              if (i > 1) rescale_output<D>(to, half * half);   // O so far (its last MMA finished before this S began)
            }
          }
          r.l += careful || vis_least < 0 ? rows_weights<true>(&bar->pfull[st], ts, mt, fac, vis, Unit{r.m, r.k})
                                          : rows_weights<false>(&bar->pfull[st], ts, mt, fac, vis, Unit{r.m, r.k});
          tc_wait_st();
          tc_fence_before();
          arrive(&bar->pfull[2 + st]);
        }
        if (!ok) break;
        // the other stream's unit and sum
        float4* ml = mls + (seg & 1) * 256;
        ml[128 * st + rr] = make_float4(r.m, r.k, r.l, 0.f);
        arrive(&bar->mlfull);
        if (!wait(&bar->mlfull, seg) || !wait(&bar->odone, seg)) break;
        tc_fence_after();
        const float4 other = ml[128 * (1 - st) + rr];
        top = higher(Unit{r.m, r.k}, other.x, other.y);
        const float mine = rows_exp2(0.5f * above(top, r.m, r.k)), theirs = rows_exp2(0.5f * above(top, other.x, other.y));
        r.l = r.l * mine * mine + other.z * theirs * theirs;
        a0 = st ? theirs * theirs : mine * mine;
        a1 = st ? mine * mine : theirs * theirs;
      }
      // channels [st * D/2, (st + 1) * D/2) of this column
      const bool complete = u.p0 == 0 && u.p1 == u.t.pages;
      float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (u.p0 == 0 ? 1 : 0)) * kv8_slot<D, kRowsNT>();
      const int tail0 = u.t.len / kPage * kPage;
      const bool odd = u.tail && u.tiles > 0 && bad_tail[seg & 3];
      const int64_t tail_id = p.tail_ids ? p.tail_ids[u.t.b] : u.t.b;
      const uint16_t* tail = reinterpret_cast<const uint16_t*>(p.tail + (tail_id * p.hkv + u.h) * F::kTailBytes) +
          F::kTailHalf;
      const Inverse inv = inverse_of(r.l);
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {   // 16 channels
        const int ch = st * (D / 2) + 16 * c;
        float o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = 0.f;
        if (u.tiles > 0) {
          uint32_t x[16];
          tc_request16(lanes + 2 * kRTile + ch, x);
          tc_wait_ld(x);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(x[k]) * a0;
        }
        if (u.tiles > 1) {
          uint32_t x[16];
          tc_request16(lanes + 2 * kRTile + D + ch, x);
          tc_wait_ld(x);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = fmaf(__uint_as_float(x[k]), a1, o[k]);
        }
        if (odd) {   // values of the tail that are not finite, to the rows that see them
#pragma unroll 1
          for (int t = 0; t < u.t.len - tail0 && tail0 + t < vis; ++t)
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int e = kv8_value_chunk(t >> 2, (ch + k) >> 2) * 16 + 4 * (k & 3) + (t & 3);
              const float x = bf16_to_float(tail[e]);
              if (!isfinite(x)) o[k] += x;
            }
        }
        if (gcol < p.cols) {
          if (complete) {
            uint16_t* dst = p.out + ((static_cast<size_t>(u.t.b) * p.m_rows + row) * p.hq + u.h * p.G +
                                     (gcol - row * p.G)) * D + ch;
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              *reinterpret_cast<uint4*>(dst + k) =
                  make_uint4(over_sum(o[k], o[k + 1], inv), over_sum(o[k + 2], o[k + 3], inv),
                             over_sum(o[k + 4], o[k + 5], inv), over_sum(o[k + 6], o[k + 7], inv));
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(slot + 128 * (ch + k) + 4 * rr) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            if (ch == 0) *reinterpret_cast<float4*>(slot + 128 * D + 4 * rr) = make_float4(top.m, top.k, r.l, 0.f);
          }
        }
      }
      if (!complete && u.p0 == 0)
        owned = make_int4(u.e, u.h, static_cast<int>((u.unit0 + u.t.pages - 1) / sh.share) - blockIdx.x + 1, 0);
      if (u.tiles > 0) {
        tc_fence_before();
        arrive(&bar->oempty[seg & 1]);
        g0 += u.tiles;
        ++seg;
      }
    }
    if (tid == 0) p.info[blockIdx.x] = *abort_flag ? make_int4(0, 0, 0, 0) : owned;
  }

  // ---- after a give-up the MMAs' own thread has waited for those in flight
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

template <int D, int kCode>
oscar_status launch_rows(const Kv8Params& p, int64_t ctas, int min_share, cudaStream_t st) {
  const auto kernel = kv8_rows_kernel<D, kCode>;
  if (!oscar_host::allow_smem(reinterpret_cast<const void*>(kernel), RowsSmem<D>::kAlloc))
    return OSCAR_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kRThreads);
  cfg.dynamicSmemBytes = RowsSmem<D>::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, min_share) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

oscar_status run_kv8_rows(const Kv8Params& p, int head_dim, int code, int64_t ctas, int min_share,
                          cudaStream_t st) {
  const bool wide = head_dim == 128;
  switch (code) {
    case kCodeE4m3:
      return wide ? launch_rows<128, kCodeE4m3>(p, ctas, min_share, st) : launch_rows<64, kCodeE4m3>(p, ctas, min_share, st);
    case kCodeE2m1:
      return wide ? launch_rows<128, kCodeE2m1>(p, ctas, min_share, st) : launch_rows<64, kCodeE2m1>(p, ctas, min_share, st);
    default:
      return wide ? launch_rows<128, kCodeInt8>(p, ctas, min_share, st) : launch_rows<64, kCodeInt8>(p, ctas, min_share, st);
  }
}

}  // namespace oscar
