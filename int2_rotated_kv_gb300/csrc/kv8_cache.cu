// Placement into the 8-bit cache and reading back (kv8_layout.cuh).
//
//   a = max |x| over the 16 tokens and d channels of a block (finite values),
//   s = fl32(a / top), inv = fl32(top / a), code = round(fl32(x inv)).
// A block is written once, when its 16 tokens are there: its scale is final and
// every value is rounded once, whatever the sizes of the calls that brought the
// tokens.  Until then they lie in the sequence's bf16 tail block.
//
// One warp does one (page, KV head, keys or values): its 16 x d values are read
// once into registers (all loads in flight before the first use), reduced, coded
// and stored as 16-byte chunks.  Bound by HBM: 2 bytes read and 1 written per value
// (place), 1 read and 2 written (gather).  Measured, 32 prompts of 3001-4096 tokens, 8 KV
// heads, d = 128, e4m3: placing and reading back 1.39 GB in 216 us, 6450 GB/s.  What it takes
// is loads in flight: small CTAs, and 64 registers a thread for 32 warps an SM (CTAs of 8
// warps at 80 registers: 235 us; at 48 registers the calls of one token take longer, 10.3 us
// for 9.4).  One token a sequence: latency, a chain of lengths, tail and codes.
#include "kv8_spans.cuh"

namespace oscar {

// The 16 x D values of page pg (tokens before s.t0 from the tail, the others from
// the rows) in chunk order.
template <int D>
__device__ __forceinline__ void load_block(const Kv8CacheParams& p, const Span& s, int h, int kv,
                                           int pg, const uint16_t* tail, int lane,
                                           uint32_t (&x)[Lane<D>::kUnits][8]) {
  const uint16_t* src = kv ? p.v : p.k;
  const int64_t stride = kv ? p.v_stride : p.k_stride;
  // row of the page's token 0 (not read where the token comes from the tail)
  const uint16_t* base = src + (s.r0 + (static_cast<int64_t>(pg) * kPage - s.t0)) * stride + h * D;
  const int old = s.t0 - pg * kPage;   // tokens of the page that lie in the tail
#pragma unroll
  for (int u = 0; u < Lane<D>::kUnits; ++u) {
    if (kv == 0) {
      int t, cc;
      Lane<D>::key(lane, u, t, cc);
      const uint4* a = reinterpret_cast<const uint4*>(
          t < old ? tail + kv8_key_chunk(t, cc) * 16 : base + t * stride + 16 * cc);
      const uint4 lo = a[0], hi = a[1];
      x[u][0] = lo.x; x[u][1] = lo.y; x[u][2] = lo.z; x[u][3] = lo.w;
      x[u][4] = hi.x; x[u][5] = hi.y; x[u][6] = hi.z; x[u][7] = hi.w;
    } else {
      int tg, cg;
      Lane<D>::value(lane, u, tg, cg);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 4 * tg + r;
        if (t >= old) {
          const uint2 a = *reinterpret_cast<const uint2*>(base + t * stride + 4 * cg);
          x[u][2 * r] = a.x;
          x[u][2 * r + 1] = a.y;
        } else {
          const uint16_t* a = tail + kv8_value_chunk(tg, cg) * 16 + r;
          x[u][2 * r] = a[0] | (static_cast<uint32_t>(a[4]) << 16);
          x[u][2 * r + 1] = a[8] | (static_cast<uint32_t>(a[12]) << 16);
        }
      }
    }
  }
  if (kv) {
#pragma unroll
    for (int u = 0; u < Lane<D>::kUnits; ++u) transpose4(x[u]);
  }
}

// Codes and scale of a block in registers.
template <int D, bool kE4m3>
__device__ __forceinline__ void store_block(const Kv8CacheParams& p, int h, int kv, int64_t id,
                                            int lane, uint32_t (&x)[Lane<D>::kUnits][8]) {
  using F = Kv8Fmt<D>;
  constexpr int kUnits = Lane<D>::kUnits;
  // magnitudes of bf16 order as integers
  uint32_t top2 = 0;
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, x[u][i] & 0x7fff7fffu);
  uint32_t amax = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
  if (amax >= 0x7f80u) {   // NaN to 0, infinities left out of the range, then to +-top
    report(p, OSCAR_DEVERR_NONFINITE);
    top2 = 0;
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t w = x[u][i];
        if ((w & 0x7fffu) > 0x7f80u) w &= 0xffff0000u;
        if ((w & 0x7fff0000u) > 0x7f800000u) w &= 0xffffu;
        x[u][i] = w;
        const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
        top2 = max(top2, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
      }
    amax = __reduce_max_sync(0xffffffffu, top2);
    // an infinity takes the largest finite magnitude, which rounds to +-top
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t w = x[u][i];
        if ((w & 0x7fffu) == 0x7f80u) w = (w & 0xffff8000u) | amax;
        if ((w & 0x7fff0000u) == 0x7f800000u) w = (w & 0x8000ffffu) | (amax << 16);
        x[u][i] = w;
      }
  }
  const float a = __uint_as_float(amax << 16);
  const bool live = a >= kKv8Least;
  const float scale = live ? __fdiv_rn(a, kv8_top<kE4m3>()) : 0.f;
  const float inv = live ? __fdiv_rn(kv8_top<kE4m3>(), a) : 0.f;
  uint8_t* blk = p.pool + (id * p.hkv + h) * F::kBlock;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = kv8_codes4<kE4m3>(bf16_lo_value(x[u][2 * i]), bf16_hi_value(x[u][2 * i]),
                               bf16_lo_value(x[u][2 * i + 1]), bf16_hi_value(x[u][2 * i + 1]), inv);
    int a0, a1, chunk;
    if (kv == 0) {
      Lane<D>::key(lane, u, a0, a1);
      chunk = kv8_key_chunk(a0, a1);
    } else {
      Lane<D>::value(lane, u, a0, a1);
      chunk = kv8_value_chunk(a0, a1);
    }
    reinterpret_cast<uint4*>(blk + kv * F::kCodes)[chunk] = make_uint4(c[0], c[1], c[2], c[3]);
  }
  if (lane < 2) {   // the scale and one spare word
    float* w = reinterpret_cast<float*>(blk + F::kScales) + kv + 2 * lane;
    *w = lane == 0 ? scale : 0.f;
  }
}

// blockIdx.x: (sequence, page of its rows), blockIdx.y: kCWarps (KV head, K/V) each.
// The warp of a sequence's first page also writes the tail: the first page may
// take tokens from the tail that the last ones are about to overwrite.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(32 * kCWarps, 8) kv8_place_kernel(const __grid_constant__ Kv8CacheParams p) {
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
      uint32_t x[Lane<D>::kUnits][8];
      load_block<D>(p, s, h, kv, pg, tail, lane, x);
      store_block<D, kE4m3>(p, h, kv, id, lane, x);
    }
    __syncwarp();   // the tail has been read
  }
  if (writes_tail && tail) store_tail<D>(p, s, h, kv, max(s.t0, whole * kPage), tail, lane);
}

// The same units the other way: codes times scale, rounded to bf16; tail tokens as
// they are.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(32 * kCWarps) kv8_gather_kernel(const __grid_constant__ Kv8CacheParams p) {
  using F = Kv8Fmt<D>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, unit = blockIdx.y * kCWarps + (threadIdx.x >> 5);
  if (unit >= 2 * p.hkv) return;
  const int h = unit >> 1, kv = unit & 1;
  const int b = blockIdx.x / p.pages_per_seq, i = blockIdx.x - b * p.pages_per_seq;
  Span s;
  if (!span_of(p, b, s)) return;
  const int pg = s.t0 / kPage + i, len = p.seq_lens[b];
  // rows behind the stored tokens are left as they were
  if (s.t1 > len || len >= (static_cast<int64_t>(p.max_pages) + 1) * kPage) {
    report(p, OSCAR_DEVERR_SEQ_LEN);
    return;
  }
  if (pg > (s.t1 - 1) / kPage) return;
  const int lo = max(s.t0 - pg * kPage, 0), hi = min(s.t1 - pg * kPage, kPage);
  const uint8_t* blk = nullptr;
  const uint16_t* tail = nullptr;
  float scale = 1.f;
  if (pg < len / kPage) {
    const int64_t id = page_id(p, b, pg);
    if (id < 0) return;
    blk = p.pool + (id * p.hkv + h) * F::kBlock;
    scale = reinterpret_cast<const float*>(blk + F::kScales)[kv];
    blk += kv * F::kCodes;
  } else {
    tail = tail_area<D>(p, b, h, kv);
    if (!tail) return;
  }
  uint16_t* out = (kv ? p.v_out : p.k_out) +
      ((s.r0 + (static_cast<int64_t>(pg) * kPage - s.t0)) * p.hkv + h) * D;
  const int64_t stride = static_cast<int64_t>(p.hkv) * D;
  uint4 c[Lane<D>::kUnits];
#pragma unroll
  for (int u = 0; u < Lane<D>::kUnits; ++u) {
    int a0, a1;
    if (kv == 0) Lane<D>::key(lane, u, a0, a1);
    else Lane<D>::value(lane, u, a0, a1);
    const int chunk = kv == 0 ? kv8_key_chunk(a0, a1) : kv8_value_chunk(a0, a1);
    if (blk) c[u] = reinterpret_cast<const uint4*>(blk)[chunk];
  }
#pragma unroll
  for (int u = 0; u < Lane<D>::kUnits; ++u) {
    int a0, a1;
    if (kv == 0) Lane<D>::key(lane, u, a0, a1);
    else Lane<D>::value(lane, u, a0, a1);
    const int chunk = kv == 0 ? kv8_key_chunk(a0, a1) : kv8_value_chunk(a0, a1);
    uint32_t x[8];
    if (blk) {
      const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = pack_bf162(__fmul_rn(kv8_code_value<kE4m3>(w[k >> 1], 2 * (k & 1)), scale),
                          __fmul_rn(kv8_code_value<kE4m3>(w[k >> 1], 2 * (k & 1) + 1), scale));
    } else {
      const uint4* a = reinterpret_cast<const uint4*>(tail + chunk * 16);
      const uint4 q0 = a[0], q1 = a[1];
      x[0] = q0.x; x[1] = q0.y; x[2] = q0.z; x[3] = q0.w;
      x[4] = q1.x; x[5] = q1.y; x[6] = q1.z; x[7] = q1.w;
    }
    if (kv == 0) {
      if (a0 >= lo && a0 < hi) {
        uint4* dst = reinterpret_cast<uint4*>(out + a0 * stride + 16 * a1);
        dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
        dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
      }
    } else {
      transpose4(x);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = 4 * a0 + r;
        if (t >= lo && t < hi)
          *reinterpret_cast<uint2*>(out + t * stride + 4 * a1) = make_uint2(x[2 * r], x[2 * r + 1]);
      }
    }
  }
}

}  // namespace oscar

using namespace oscar;

extern "C" {

oscar_status oscar_kv8_place(const oscar_kv8_desc* desc, const void* k, const void* v,
                             int64_t k_stride, int64_t v_stride, const int32_t* lens_before,
                             const int32_t* row_starts, int32_t batch, int64_t total_rows,
                             int32_t max_new, void* stream) {
  oscar_status s = oscar_host::check_kv8(desc);
  if (s != OSCAR_OK) return s;
  Kv8CacheParams p{};
  s = place_params(desc, k, v, k_stride, v_stride, lens_before, row_starts, batch, total_rows, max_new, &p);
  if (s != OSCAR_OK || p.batch == 0) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = desc->format == OSCAR_KV8_E4M3;
  if (desc->head_dim == 128)
    return e4m3 ? launch_cache(kv8_place_kernel<128, true>, p, st, 2 * p.hkv)
                : launch_cache(kv8_place_kernel<128, false>, p, st, 2 * p.hkv);
  return e4m3 ? launch_cache(kv8_place_kernel<64, true>, p, st, 2 * p.hkv)
              : launch_cache(kv8_place_kernel<64, false>, p, st, 2 * p.hkv);
}

oscar_status oscar_kv8_gather(const oscar_kv8_desc* desc, const int32_t* seq_lens,
                              const int32_t* first, const int32_t* row_starts, int32_t batch,
                              int64_t total_rows, int32_t max_rows, void* k_out, void* v_out,
                              void* stream) {
  oscar_status s = oscar_host::check_kv8(desc);
  if (s != OSCAR_OK) return s;
  Kv8CacheParams p{};
  s = gather_params(desc, seq_lens, first, row_starts, batch, total_rows, max_rows, k_out, v_out, &p);
  if (s != OSCAR_OK || p.batch == 0) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = desc->format == OSCAR_KV8_E4M3;
  if (desc->head_dim == 128)
    return e4m3 ? launch_cache(kv8_gather_kernel<128, true>, p, st, 2 * p.hkv)
                : launch_cache(kv8_gather_kernel<128, false>, p, st, 2 * p.hkv);
  return e4m3 ? launch_cache(kv8_gather_kernel<64, true>, p, st, 2 * p.hkv)
              : launch_cache(kv8_gather_kernel<64, false>, p, st, 2 * p.hkv);
}

}  // extern "C"
