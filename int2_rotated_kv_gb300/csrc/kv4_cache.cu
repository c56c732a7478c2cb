// Placement into the 4-bit cache and reading back (kv4_layout.cuh).
//
//   a = max |x| over the 16 tokens and d channels of a page (finite values), g = fl32(a / 2688);
//   per block of 16 (a channel's 16 tokens for keys, 16 channels of a token for values)
//   s = e4m3(fl32(max|x| fl32(448 / a))), code = e2m1(fl32(x fl32(fl32(2688 / a) / s))).
// As in the 8-bit cache a page is coded once, when its 16 tokens are there, and they lie in
// the sequence's bf16 tail block until then.
//
// One warp does one (page, KV head, keys or values), its 16 x d values in registers: a lane has 4
// channels of all tokens (of 8 tokens for d = 64), so that maxima over tokens stay in a lane and
// those over 16 channels take two shuffles; the codes cross lanes once, to be stored 16 bytes a lane.
//
// Bound by HBM at long prompts: 4 d + 1.125 d + 1 bytes per token and KV head.  24 prompts of 2500-5000 tokens, 8 KV heads
// of 128: placing 87 us, 5.4 TB/s, with the issue slots 64% busy; reading back 77, 6.1 TB/s; 16 prefixes of 4097-8192
// tokens read back 74 us, 6.25 TB/s.  A token of 64 sequences: 6.2 and 4.2 us, a chain of lengths, ids and values.
// Placing is near its instructions' bound too: products two at a time, maxima of pairs of bf16 and each block's scale
// found by one lane took placing and reading back of the prompts from 183 to 165 us.
#include "kv4_layout.cuh"
#include "kv8_spans.cuh"

namespace oscar {

// A lane's values: channels 4 cg .. 4 cg + 3 (two words) of tokens t0 .. t0 + kTokens - 1.
template <int D>
struct Lane4 {
  static constexpr int kTokens = D / 8;
  static __device__ __forceinline__ int cg(int lane) { return lane % (D / 4); }
  static __device__ __forceinline__ int t0(int lane) { return lane / (D / 4) * kTokens; }
};

// The values of page pg: tokens before s.t0 from the tail, the others from the rows.
template <int D>
__device__ __forceinline__ void load_values(const Kv8CacheParams& p, const Span& s, int h, int kv, int pg,
                                            const uint16_t* tail, int lane,
                                            uint32_t (&x)[Lane4<D>::kTokens][2]) {
  const int cg = Lane4<D>::cg(lane), t0 = Lane4<D>::t0(lane);
  const int64_t stride = kv ? p.v_stride : p.k_stride;
  // row of the page's token 0 (not read where the token comes from the tail)
  const uint16_t* base = (kv ? p.v : p.k) + (s.r0 + (static_cast<int64_t>(pg) * kPage - s.t0)) * stride + h * D + 4 * cg;
  const int old = s.t0 - pg * kPage;   // tokens of the page that lie in the tail
  if (old <= 0) {
    const uint16_t* row = base + t0 * stride;
#pragma unroll
    for (int i = 0; i < Lane4<D>::kTokens; ++i, row += stride) {
      const uint2 w = *reinterpret_cast<const uint2*>(row);
      x[i][0] = w.x;
      x[i][1] = w.y;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < Lane4<D>::kTokens; ++i) {
    const int t = t0 + i;
    if (t >= old) {
      const uint2 w = *reinterpret_cast<const uint2*>(base + t * stride);
      x[i][0] = w.x;
      x[i][1] = w.y;
    } else if (kv == 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(tail + kv8_key_chunk(t, cg >> 2) * 16 + 4 * (cg & 3));
      x[i][0] = w.x;
      x[i][1] = w.y;
    } else {
      const uint16_t* w = tail + kv8_value_chunk(t >> 2, cg) * 16 + (t & 3);
      x[i][0] = w[0] | (static_cast<uint32_t>(w[4]) << 16);
      x[i][1] = w[8] | (static_cast<uint32_t>(w[12]) << 16);
    }
  }
}

// The larger magnitudes of two pairs of bf16, signs undefined; NaN where there is one.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// NaN become 0, infinities the largest finite magnitude.  Out of line, as nearly never needed, and by value, which
// leaves the caller's in registers.
template <int kTokens>
struct Values {
  uint32_t x[kTokens][2];
};
template <int kTokens>
__device__ __noinline__ Values<kTokens> finite_values(Values<kTokens> v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w = v.x[i][j];
      if ((w & 0x7fffu) > 0x7f80u) w &= 0xffff0000u;
      if ((w & 0x7fff0000u) > 0x7f800000u) w &= 0xffffu;
      v.x[i][j] = w;
      const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
      top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
  const uint32_t amax = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
  for (int i = 0; i < kTokens; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w = v.x[i][j];
      if ((w & 0x7fffu) == 0x7f80u) w = (w & 0xffff8000u) | amax;
      if ((w & 0x7fff0000u) == 0x7f800000u) w = (w & 0x8000ffffu) | (amax << 16);
      v.x[i][j] = w;
    }
  return v;
}
template <int kTokens>
__device__ __forceinline__ void make_finite(uint32_t (&x)[kTokens][2]) {
  Values<kTokens> v;
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    v.x[i][0] = x[i][0];
    v.x[i][1] = x[i][1];
  }
  v = finite_values(v);
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    x[i][0] = v.x[i][0];
    x[i][1] = v.x[i][1];
  }
}

// Scale byte of a block whose largest magnitude is m (bf16 bits), and what its values are times to
// be codes: 0 for a block that is stored as zeros.
struct PageScale {
  float to_block, to_code;   // fl32(448 / a), fl32(2688 / a)
};
__device__ __forceinline__ uint32_t block_scale(uint32_t m, PageScale g, float& r) {
  const float y = __fmul_rn(__uint_as_float(m << 16), g.to_block);
  uint16_t two;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(two) : "f"(0.f), "f"(y));
  const uint32_t byte = two & 0xffu;
  uint32_t lo, hi;
  kv4_scales(byte, lo, hi);
  const float s = half_lo(lo);
  r = s > 0.f ? __fdiv_rn(g.to_code, s) : 0.f;
  return byte;
}

// Codes of eight values x (pairs of bf16) times r (pairs of fp32).
__device__ __forceinline__ uint32_t codes8(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint64_t r0, uint64_t r1,
                                           uint64_t r2, uint64_t r3) {
  const uint64_t y0 = mul2(two(bf16_lo_value(x0), bf16_hi_value(x0)), r0);
  const uint64_t y1 = mul2(two(bf16_lo_value(x1), bf16_hi_value(x1)), r1);
  const uint64_t y2 = mul2(two(bf16_lo_value(x2), bf16_hi_value(x2)), r2);
  const uint64_t y3 = mul2(two(bf16_lo_value(x3), bf16_hi_value(x3)), r3);
  const float y[8] = {first(y0), second(y0), first(y1), second(y1), first(y2), second(y2), first(y3), second(y3)};
  return kv4_codes8(y);
}

// v[k] of lane l among four neighbours becomes lane k's v[l].
__device__ __forceinline__ void transpose_quad(uint32_t (&v)[4], int lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & bit) continue;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k | bit], bit);
      if (up) v[k] = got;
      else v[k | bit] = got;
    }
  }
}

// The page's scales from its largest magnitude (bf16 bits); its own goes to `at`.
__device__ __forceinline__ PageScale page_scale(uint32_t amax, float* at, int lane) {
  const float a = __uint_as_float(amax << 16);
  const bool live = a >= kKv4Least;
  if (lane < 2)   // the scale and, two words on, a spare one
    at[2 * lane] = lane == 0 && live ? __fdiv_rn(a, kKv4Top) : 0.f;
  return {live ? __fdiv_rn(kKv4BlockTop, a) : 0.f, live ? __fdiv_rn(kKv4Top, a) : 0.f};
}

// Largest magnitudes of blocks m (pairs) of a warp's page, and the page's; false: something is not finite.
template <int kPairs>
__device__ __forceinline__ bool page_max(uint32_t (&m)[kPairs], uint32_t& amax) {
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    m[i] &= 0x7fff7fffu;
    all = __vmaxu2(all, m[i]);
  }
  amax = __reduce_max_sync(0xffffffffu, max(all & 0xffffu, all >> 16));
  return amax < 0x7f80u;
}

// Codes and scales of a page's keys.
template <int D>
__device__ __forceinline__ void store_keys(const Kv8CacheParams& p, uint8_t* blk, int lane, uint32_t (&x)[Lane4<D>::kTokens][2]) {
  constexpr int kTokens = Lane4<D>::kTokens;
  const int cg = Lane4<D>::cg(lane), t0 = Lane4<D>::t0(lane);
  uint32_t m[2], amax;   // of channels (0, 1), (2, 3)
  auto maxima = [&] {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < kTokens; ++i) m[j] = larger(m[j], x[i][j]);
    }
    return page_max(m, amax);
  };
  if (!maxima()) {
    report(p, OSCAR_DEVERR_NONFINITE);
    make_finite(x);
    maxima();
  }
  if constexpr (D == 64) {   // and of the other lane's tokens
    m[0] = __vmaxu2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 16));
    m[1] = __vmaxu2(m[1], __shfl_xor_sync(0xffffffffu, m[1], 16));
  }
  const PageScale g = page_scale(amax, reinterpret_cast<float*>(blk + Kv4Fmt<D>::kScales), lane);
  float r[4];
  uint32_t scales = block_scale(m[0] & 0xffffu, g, r[0]);
  scales |= block_scale(m[0] >> 16, g, r[1]) << 8;
  scales |= block_scale(m[1] & 0xffffu, g, r[2]) << 16;
  scales |= block_scale(m[1] >> 16, g, r[3]) << 24;
  const uint64_t r01 = two(r[0], r[1]), r23 = two(r[2], r[3]);
  if (t0 == 0) *reinterpret_cast<uint32_t*>(blk + Kv4Fmt<D>::kKeyScales + 4 * cg) = scales;
  // two tokens of 4 channels a word; the four lanes of 16 channels share theirs out
  const int l = lane & 3;
  uint4* out = reinterpret_cast<uint4*>(blk) + (cg >> 4) * 32 + ((cg >> 2) & 3);
#pragma unroll
  for (int half = 0; half < kTokens / 8; ++half) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 8 * half + 2 * k;
      w[k] = codes8(x[i][0], x[i][1], x[i + 1][0], x[i + 1][1], r01, r23, r01, r23);
    }
    transpose_quad(w, lane);
    out[4 * (t0 / 2 + 4 * half + l)] =
        make_uint4(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410),
                   __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
  }
}

// Codes and scales of a page's values.
template <int D>
__device__ __forceinline__ void store_values(const Kv8CacheParams& p, uint8_t* blk, int lane, uint32_t (&x)[Lane4<D>::kTokens][2]) {
  constexpr int kTokens = Lane4<D>::kTokens, kOwn = kTokens / 4;
  const int cg = Lane4<D>::cg(lane), t0 = Lane4<D>::t0(lane), l = lane & 3;
  // largest magnitudes of (token 2i, token 2i + 1), of a lane's channels, then of the 16 of four lanes
  uint32_t m[kTokens / 2], amax;
  auto maxima = [&] {
#pragma unroll
    for (int i = 0; i < kTokens / 2; ++i) {
      const uint32_t a = larger(x[2 * i][0], x[2 * i][1]), b = larger(x[2 * i + 1][0], x[2 * i + 1][1]);
      m[i] = larger(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    }
    return page_max(m, amax);
  };
  if (!maxima()) {
    report(p, OSCAR_DEVERR_NONFINITE);
    make_finite(x);
    maxima();
  }
  const PageScale g = page_scale(amax, reinterpret_cast<float*>(blk + Kv4Fmt<D>::kScales) + 1, lane);
#pragma unroll
  for (int i = 0; i < kTokens / 2; ++i) {
    m[i] = __vmaxu2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 1));
    m[i] = __vmaxu2(m[i], __shfl_xor_sync(0xffffffffu, m[i], 2));
  }
  // a lane finds the scales of kOwn tokens, l kOwn and on
  float own[kOwn];
  uint32_t scales = 0;
#pragma unroll
  for (int k = 0; k < kOwn; k += 2) {
    uint32_t pair = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (l == i) pair = m[(i * kOwn + k) / 2];
    scales |= block_scale(pair & 0xffffu, g, own[k]) << (8 * k);
    scales |= block_scale(pair >> 16, g, own[k + 1]) << (8 * k + 8);
  }
  uint8_t* at = blk + Kv4Fmt<D>::kValueScales + kv4_value_scale(t0 + l * kOwn, cg >> 2);
  if constexpr (kOwn == 4) *reinterpret_cast<uint32_t*>(at) = scales;
  else *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(scales);
  // four tokens of two channels a word: both words of a group of four tokens
  uint32_t w[kTokens / 4][2];
#pragma unroll
  for (int q = 0; q < kTokens / 4; ++q) {
    float r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = __shfl_sync(0xffffffffu, own[(4 * q + i) % kOwn], (lane & ~3) | ((4 * q + i) / kOwn));
    const uint64_t r01 = two(r[0], r[1]), r23 = two(r[2], r[3]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t a = __byte_perm(x[4 * q][j], x[4 * q + 1][j], 0x5410);       // channel 2j of tokens 0, 1
      const uint32_t b = __byte_perm(x[4 * q + 2][j], x[4 * q + 3][j], 0x5410);
      const uint32_t c = __byte_perm(x[4 * q][j], x[4 * q + 1][j], 0x7632);       // channel 2j + 1
      const uint32_t d = __byte_perm(x[4 * q + 2][j], x[4 * q + 3][j], 0x7632);
      w[q][j] = codes8(a, b, c, d, r01, r23, r01, r23);
    }
  }
  // with the lane of the channels 32 further: a chunk is 4 tokens of both lanes' channels
  const int high = (cg >> 3) & 1;
  uint4* out = reinterpret_cast<uint4*>(blk + Kv4Fmt<D>::kCodes) + (cg >> 4) * 32 + 4 * (cg & 7) + t0 / 4;
  constexpr int kHalf = kTokens / 8;   // chunks a lane stores
#pragma unroll
  for (int q = 0; q < kHalf; ++q) {
    uint32_t mine[2], got[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mine[j] = high ? w[kHalf + q][j] : w[q][j];
      got[j] = __shfl_xor_sync(0xffffffffu, high ? w[q][j] : w[kHalf + q][j], 8);
    }
    out[high * kHalf + q] = high ? make_uint4(got[0], got[1], mine[0], mine[1]) : make_uint4(mine[0], mine[1], got[0], got[1]);
  }
}

// blockIdx.x: (sequence, page of its rows), blockIdx.y: kCWarps (KV head, K/V) each.
// (8 CTAs an SM, 64 registers: the prompts 86 us; 5, 6 and 7: 104, 95 and 90.5; 9, with more spilled, 85.)
// The warp of a sequence's first page also writes the tail: the first page may
// take tokens from the tail that the last ones are about to overwrite.
template <int D>
__global__ void __launch_bounds__(32 * kCWarps, 8) kv4_place_kernel(const __grid_constant__ Kv8CacheParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, unit = blockIdx.y * kCWarps + (threadIdx.x >> 5);
  if (unit >= 2 * p.hkv) return;
  const int h = unit >> 1, kv = unit & 1;
  const int b = blockIdx.x / p.pages_per_seq, i = blockIdx.x - b * p.pages_per_seq;
  Span s;
  if (!span_of(p, b, s)) return;
  const int pg = s.t0 / kPage + i, whole = s.t1 / kPage;
  uint16_t* tail = nullptr;
  const bool reads_tail = i == 0 && pg < whole && s.t0 % kPage != 0;
  const bool writes_tail = i == 0 && s.t1 % kPage != 0;
  if (reads_tail || writes_tail) {
    tail = tail_area<D>(p, b, h, kv);
    if (!tail && pg >= whole) return;
  }
  if (pg < whole && !(reads_tail && !tail)) {
    const int64_t id = page_id(p, b, pg);
    if (id >= 0) {
      uint32_t x[Lane4<D>::kTokens][2];
      load_values<D>(p, s, h, kv, pg, tail, lane, x);
      uint8_t* blk = p.pool + (id * p.hkv + h) * Kv4Fmt<D>::kBlock;
      if (kv == 0) store_keys<D>(p, blk, lane, x);
      else store_values<D>(p, blk, lane, x);
    }
    __syncwarp();   // the tail has been read
  }
  if (writes_tail && tail) store_tail<D>(p, s, h, kv, max(s.t0, whole * kPage), tail, lane);
}

// Two codes times two scales times g, as bf16.
__device__ __forceinline__ uint32_t value_pair(uint32_t codes, uint32_t scales, float g) {
  const uint32_t x = hmul2_u32(codes, scales);
  return pack_bf162(__fmul_rn(half_lo(x), g), __fmul_rn(half_hi(x), g));
}

// Tokens [lo, hi) of a tail area (keys or values) to their rows.
template <int D>
__device__ __forceinline__ void tail_rows(const uint16_t* tail, int kv, int lo, int hi, int lane, uint16_t* out, int64_t stride) {
  uint32_t x[Lane<D>::kUnits][8];
#pragma unroll
  for (int u = 0; u < Lane<D>::kUnits; ++u) {
    int a0, a1;
    if (kv == 0) Lane<D>::key(lane, u, a0, a1);
    else Lane<D>::value(lane, u, a0, a1);
    const uint4* a = reinterpret_cast<const uint4*>(tail + (kv == 0 ? kv8_key_chunk(a0, a1) : kv8_value_chunk(a0, a1)) * 16);
    const uint4 q0 = a[0], q1 = a[1];
    x[u][0] = q0.x; x[u][1] = q0.y; x[u][2] = q0.z; x[u][3] = q0.w;
    x[u][4] = q1.x; x[u][5] = q1.y; x[u][6] = q1.z; x[u][7] = q1.w;
  }
#pragma unroll
  for (int u = 0; u < Lane<D>::kUnits; ++u) {
    int a0, a1;
    if (kv == 0) {
      Lane<D>::key(lane, u, a0, a1);
      if (a0 < lo || a0 >= hi) continue;
      uint4* dst = reinterpret_cast<uint4*>(out + a0 * stride + 16 * a1);
      dst[0] = make_uint4(x[u][0], x[u][1], x[u][2], x[u][3]);
      dst[1] = make_uint4(x[u][4], x[u][5], x[u][6], x[u][7]);
    } else {
      Lane<D>::value(lane, u, a0, a1);
      transpose4(x[u]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 4 * a0 + r;
        if (t >= lo && t < hi)
          *reinterpret_cast<uint2*>(out + t * stride + 4 * a1) = make_uint2(x[u][2 * r], x[u][2 * r + 1]);
      }
    }
  }
}

constexpr int kGatherCtas = 10;   // 48 registers a thread
// Codes back to bf16, rounded once from fl32(code s g); tail tokens as they are.  A warp does a page's keys and
// values of a KV head: every load of both is on its way before the first use (16 prefixes of 4097-8192 tokens 74 us; keys
// and values by warps of their own, 80).
template <int D>
__global__ void __launch_bounds__(32 * kCWarps, kGatherCtas) kv4_gather_kernel(const __grid_constant__ Kv8CacheParams p) {
  using F = Kv4Fmt<D>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, h = blockIdx.y * kCWarps + (threadIdx.x >> 5);
  if (h >= p.hkv) return;
  const int b = blockIdx.x / p.pages_per_seq, i = blockIdx.x - b * p.pages_per_seq;
  Span s;
  const int len = p.seq_lens[b];
  if (!span_of(p, b, s)) return;
  const int pg = s.t0 / kPage + i;
  // rows behind the stored tokens are left as they were
  if (s.t1 > len || len >= (static_cast<int64_t>(p.max_pages) + 1) * kPage) {
    report(p, OSCAR_DEVERR_SEQ_LEN);
    return;
  }
  if (pg > (s.t1 - 1) / kPage) return;
  const int lo = max(s.t0 - pg * kPage, 0), hi = min(s.t1 - pg * kPage, kPage);
  const int64_t first = ((s.r0 + (static_cast<int64_t>(pg) * kPage - s.t0)) * p.hkv + h) * D;
  const int64_t stride = static_cast<int64_t>(p.hkv) * D;
  if (pg >= len / kPage) {
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      const uint16_t* tail = tail_area<D>(p, b, h, kv);
      if (tail) tail_rows<D>(tail, kv, lo, hi, lane, (kv ? p.v_out : p.k_out) + first, stride);
    }
    return;
  }
  const int64_t id = page_id(p, b, pg);
  if (id < 0) return;
  const uint8_t* blk = p.pool + (id * p.hkv + h) * F::kBlock;
  const int gid = lane >> 2, tig = lane & 3;
  uint4 ck[D / 64], sk[D / 64], cv[D / 64];
  uint2 sv[D / 64];
  const float2 g = *reinterpret_cast<const float2*>(blk + F::kScales);
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    ck[j] = reinterpret_cast<const uint4*>(blk)[32 * j + lane];
    sk[j] = reinterpret_cast<const uint4*>(blk + F::kKeyScales)[4 * j + tig];
  }
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    cv[j] = reinterpret_cast<const uint4*>(blk + F::kCodes)[32 * j + lane];
    sv[j] = reinterpret_cast<const uint2*>(blk + F::kValueScales)[8 * j + 4 * (gid >> 2) + tig];
  }
  uint16_t* out = p.k_out + first;
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {   // two tokens, 16 channels
    const uint32_t w[4] = {ck[j].x, ck[j].y, ck[j].z, ck[j].w};
    uint32_t x[8];
    kv4_scales(sk[j].x, x[0], x[1]);
    kv4_scales(sk[j].y, x[2], x[3]);
    kv4_scales(sk[j].z, x[4], x[5]);
    kv4_scales(sk[j].w, x[6], x[7]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = 2 * gid + e;
      if (t < lo || t >= hi) continue;
      uint4* dst = reinterpret_cast<uint4*>(out + t * stride + 64 * j + 16 * tig);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t y[4];
        kv4_pairs(w[2 * e + half], y[0], y[1], y[2], y[3]);
        dst[half] = make_uint4(value_pair(y[0], x[4 * half], g.x), value_pair(y[1], x[4 * half + 1], g.x),
                               value_pair(y[2], x[4 * half + 2], g.x), value_pair(y[3], x[4 * half + 3], g.x));
      }
    }
  }
  out = p.v_out + first;
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {   // four tokens, 4 channels and the 4 that are 32 further
    const uint32_t w[4] = {cv[j].x, cv[j].y, cv[j].z, cv[j].w};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t s01, s23;
      kv4_scales(half ? sv[j].y : sv[j].x, s01, s23);
      uint32_t x[8];   // channel c: tokens 0..3 in x[2c], x[2c + 1]
      kv4_pairs(w[2 * half], x[0], x[1], x[2], x[3]);
      kv4_pairs(w[2 * half + 1], x[4], x[5], x[6], x[7]);
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = value_pair(x[k], k & 1 ? s23 : s01, g.y);
      transpose4(x);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 4 * tig + r;
        if (t >= lo && t < hi)
          *reinterpret_cast<uint2*>(out + t * stride + 64 * j + 32 * half + 4 * gid) = make_uint2(x[2 * r], x[2 * r + 1]);
      }
    }
  }
}

}  // namespace oscar

using namespace oscar;

extern "C" {

oscar_status oscar_kv4_place(const oscar_kv4_desc* desc, const void* k, const void* v,
                             int64_t k_stride, int64_t v_stride, const int32_t* lens_before,
                             const int32_t* row_starts, int32_t batch, int64_t total_rows,
                             int32_t max_new, void* stream) {
  oscar_kv8_desc c;
  oscar_status s = oscar_host::check_kv4(desc, &c);
  if (s != OSCAR_OK) return s;
  Kv8CacheParams p{};
  s = place_params(&c, k, v, k_stride, v_stride, lens_before, row_starts, batch, total_rows, max_new, &p);
  if (s != OSCAR_OK || p.batch == 0) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c.head_dim == 128 ? launch_cache(kv4_place_kernel<128>, p, st, 2 * p.hkv) : launch_cache(kv4_place_kernel<64>, p, st, 2 * p.hkv);
}

oscar_status oscar_kv4_gather(const oscar_kv4_desc* desc, const int32_t* seq_lens,
                              const int32_t* first, const int32_t* row_starts, int32_t batch,
                              int64_t total_rows, int32_t max_rows, void* k_out, void* v_out,
                              void* stream) {
  oscar_kv8_desc c;
  oscar_status s = oscar_host::check_kv4(desc, &c);
  if (s != OSCAR_OK) return s;
  Kv8CacheParams p{};
  s = gather_params(&c, seq_lens, first, row_starts, batch, total_rows, max_rows, k_out, v_out, &p);
  if (s != OSCAR_OK || p.batch == 0) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c.head_dim == 128 ? launch_cache(kv4_gather_kernel<128>, p, st, p.hkv) : launch_cache(kv4_gather_kernel<64>, p, st, p.hkv);
}

}  // extern "C"
