// Tokens of the calibrated cache (layout.cuh) read back as bf16 rows.
//
// A token t of a sequence of L tokens that is a sink (t < sink) or recent (t >= L - window) is in
// BF16 and comes back as it is.  The others are codes of x R: with y = code * s + z (fp32),
//   x[j] = sum_c y[c] R[j][c],
// what attention takes it for ("Technical Summary: OSCAR ...", section 2.2B: the rotation is undone
// when the history is used).
//
// The product runs on tcgen05 as bf16 pieces, y = y1 + y2 and R = R1 + R2 (each to 2^-17):
//   x = y2 R1^T + y1 R2^T + y1 R1^T,   fp32 accumulation in tensor memory.
// M = 128 tokens (8 pages of one sequence), N = K = d; R's pieces lie in shared memory (rows of R
// are the K-major rows of operand B as they are), y's pieces in tensor memory, where a thread writes
// its own token's row.  A CTA keeps the R of one (KV head, keys or values) and walks over tiles of
// tokens; two CTAs an SM, so that one's MMAs and stores run under the other's arithmetic.
//   warps 0-7  a token and half of its channels a thread: codes to y1, y2; then the product's row to
//              bf16 and out.  One lane of warp 0 issues the 3 d/16 MMAs of a tile.
//   warp 8     tiles ahead: finds the next tiles that hold rows (32 at a look), and copies the codes
//              of their pages into a ring of stages (bulk copies, one a page).
// Every wait is bounded; a CTA that gives up finishes its copies and MMAs first.
#include <algorithm>

#include "common.cuh"
#include "layout.cuh"
#include "tcgen05.cuh"

namespace oscar {

struct GatherParams {
  int hkv, max_pages, batch, tiles_per_seq, max_rows, sink, window, ctas_per_r;
  bool whole;        // outputs start at a multiple of 32 bytes
  int64_t n_coded, n_plain, total_rows;
  const uint8_t* coded;
  const uint8_t* plain;
  const int32_t* coded_table;
  const int32_t* plain_table;
  const float* r[2];
  uint16_t* out[2];
  const int32_t* seq_lens;
  const int32_t* first;
  const int32_t* row_starts;
  int32_t* status;
};

constexpr int kGTile = 128;                 // tokens of a tile
constexpr int kGPages = kGTile / kPage;
constexpr int kGStages = 4;
constexpr int kGWarps = 8;                  // that compute
constexpr int kGThreads = 32 * (kGWarps + 1);

// A tile as the computing warps need it: positions of its tokens are pos0 + row.
struct GatherTile {
  int64_t row0;      // output row of the token at pos0 (rows before lo are not written)
  int pos0, lo, hi;  // positions to be read back, [lo, hi)
  int c0, c1;        // of which [c0, c1) are codes
  int b;
  uint32_t pages;    // bit per page: its codes are there
  int stop;          // 1: there is no tile
};

template <int D, int P>
struct GatherSmem {
  using F = Fmt<D, P>;
  static constexpr int kPart = F::kInt2Block / 2;        // codes, scales and zeros of keys (values)
  static_assert(F::kVc == kPart, "keys and values have the same size");
  static constexpr int kPiece = D * D * 2;               // a piece of R
  static constexpr int kRing = 2 * kPiece;
  static constexpr int kTiles = kRing + kGStages * kGPages * kPart;
  static constexpr int kBars = kTiles + kGStages * static_cast<int>(sizeof(GatherTile));
  static constexpr int kMisc = kBars + (2 * kGStages + 2) * 8;
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kAlloc = kBytes + 1024;           // the base is rounded up to 1024 bytes
  static_assert(kTiles % 16 == 0 && sizeof(GatherTile) % 8 == 0, "alignment");
};

// Two codes in the low bits of the halves of x, times s plus z, as two bf16 pieces each.
__device__ __forceinline__ void split_pair(uint32_t x, uint64_t s, uint64_t z, uint32_t& hi, uint32_t& lo) {
  constexpr float kMagic = 8388608.f;   // 2^23: its low bits are the code
  const uint64_t c = add2(two(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7610)),
                              __uint_as_float(__byte_perm(x, 0x4B000000u, 0x7632))), two(-kMagic, -kMagic));
  const uint64_t y = fma2(c, s, z);
  hi = pack_bf162(first(y), second(y));
  const uint64_t rest = fma2(two(bf16_lo_value(hi), bf16_hi_value(hi)), two(-1.f, -1.f), y);
  lo = pack_bf162(first(rest), second(rest));
}

// A thread's channels [half * D/2, ...) of the coded token t of the page at blk (keys' or values' part), to its
// row of tensor memory: y1 from column a on, y2 from a + D/2 on, two channels a column.
template <int D, int P, bool kValue>
__device__ __forceinline__ void uncode(const uint8_t* blk, int t, int half, uint32_t a) {
  using F = Fmt<D, P>;
  constexpr int kOwn = F::kWords / 2;   // groups of 32 channels a thread has
  const int th = t >> 3;
  // words of a group: keys have channels 2q, 2q + 1 (and 8, 16, 24 further) of tokens t, t ^ 8 in word q, values
  // channel gid of tokens t, t ^ 1, t ^ 8, t ^ 9 in word gid
  uint32_t x[P][4][kOwn];
#pragma unroll
  for (int pl = 0; pl < P; ++pl)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint8_t* plane = blk + pl * F::kPlane + 4 * half * kOwn;
      uint32_t w[2][kOwn];
#pragma unroll
      for (int e = 0; e < (kValue ? 2 : 1); ++e) {
        const int lane = kValue ? 4 * (2 * q + e) + ((t >> 1) & 3) : 4 * (t & 7) + q;
        if constexpr (kOwn == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(plane + 4 * lane * F::kWords);
          w[e][0] = u.x;
          w[e][1] = u.y;
        } else {
          w[e][0] = *reinterpret_cast<const uint32_t*>(plane + 4 * lane * F::kWords);
        }
      }
      // the token's byte of an even channel in the lower half, of the odd one in the upper half
      const uint32_t sel = kValue ? 0x0400u + (2 * (t & 1) + th) * 0x0101u : 0x0200u + th * 0x0101u;
#pragma unroll
      for (int m = 0; m < kOwn; ++m) x[pl][q][m] = __byte_perm(w[0][m], kValue ? w[1][m] : 0u, sel);
    }
#pragma unroll
  for (int m = 0; m < kOwn; ++m) {
    const int g = half * kOwn + m;
    float s, z;
    if constexpr (kValue) {
      const __half* vs = reinterpret_cast<const __half*>(blk + F::kVs - F::kVc);
      const int at = vsz_index<D>(t, g);
      s = __half2float(vs[at]);
      z = __half2float(vs[(F::kVz - F::kVs) / 2 + at]);
    } else {
      const uint32_t w = reinterpret_cast<const uint32_t*>(blk + F::kKsz)[t * F::kNG + g];
      s = half_lo(w);
      z = half_hi(w);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t c = (x[0][q][m] >> (4 * h + 2 * i)) & 0x00030003u;
          if constexpr (P == 2) c = c * 4 + ((x[P - 1][q][m] >> (4 * h + 2 * i)) & 0x00030003u);
          split_pair(c, two(s, s), two(z, z), hi[4 * h + q], lo[4 * h + q]);
        }
      tc_st8(a + 16 * g + 8 * i, hi);
      tc_st8(a + D / 2 + 16 * g + 8 * i, lo);
    }
  }
}

// Whether any of the computing threads says so; a barrier among them.
__device__ __forceinline__ bool any_of(bool x) {
  uint32_t y;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 q, %1, 0;\n barrier.cta.red.or.pred p, 1, %2, q;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(y)
               : "r"(static_cast<uint32_t>(x)), "n"(32 * kGWarps)
               : "memory");
  return y != 0;
}

// 32 bytes, at once where every row starts at a multiple of 32.
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&x)[8], bool whole) {
  if (whole) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// A tile's BF16 tokens, a warp each, four channels a lane (two for d = 64); kFlight tokens at once.
template <int D, bool kValue>
__device__ __forceinline__ void plain_tokens(const GatherParams& p, const GatherTile& t, int h, int warp, int lane) {
  constexpr int kOwn = D / 32, kFlight = 4;
  const int before = t.c0 - t.lo, n = before + t.hi - t.c1;
#pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += kGWarps * kFlight) {
    int pos[kFlight], id[kFlight];
    uint32_t x[kFlight][kOwn / 2];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int i = i0 + k * kGWarps;
      pos[k] = i < before ? t.lo + i : t.c1 + i - before;
      id[k] = i < n ? p.plain_table[static_cast<size_t>(t.b) * p.max_pages + pos[k] / kPage] : -1;
      if (i < n && (id[k] < 0 || id[k] >= p.n_plain)) {
        if (p.status && lane == 0) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
        id[k] = -1;
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(
          p.plain + (static_cast<int64_t>(max(id[k], 0)) * p.hkv + h) * Fmt<D>::kBf16Block + (kValue ? Fmt<D>::kBf16V : 0));
#pragma unroll
      for (int c = 0; c < kOwn / 2; ++c) {
        const int j = kOwn * lane + 2 * c, tk = pos[k] % kPage;
        if (id[k] < 0) continue;
        x[k][c] = kValue ? src[bf16_value_elem(tk, j)] | (static_cast<uint32_t>(src[bf16_value_elem(tk, j + 1)]) << 16)
                         : *reinterpret_cast<const uint32_t*>(src + bf16_key_elem(tk, j));
      }
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (id[k] < 0) continue;
      uint16_t* dst = p.out[kValue] + ((t.row0 + pos[k] - t.pos0) * p.hkv + h) * D + kOwn * lane;
      if constexpr (kOwn == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(x[k][0], x[k][1]);
      else *reinterpret_cast<uint32_t*>(dst) = x[k][0];
    }
  }
}

template <int D, int P>
__global__ void __launch_bounds__(kGThreads, 2) gather_kernel(const __grid_constant__ GatherParams p) {
  using S = GatherSmem<D, P>;
  using F = Fmt<D, P>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  GatherTile* tiles = reinterpret_cast<GatherTile*>(smem + S::kTiles);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);
  uint64_t* empty = full + kGStages;
  uint64_t* done = empty + kGStages;       // the MMAs of a tile; then those in flight after a give-up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int which = blockIdx.x / p.ctas_per_r, number = blockIdx.x - which * p.ctas_per_r;
  const int h = which >> 1, kv = which & 1;

  if (tid == 0) {
    for (int i = 0; i < kGStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kGWarps);
    }
    mbar_init(done, 1);
    mbar_init(done + 1, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc_alloc(tmem_slot, 2 * D);
  // R as two bf16 pieces
  const float* r = p.r[kv] + static_cast<size_t>(h) * D * D;
  for (int i = tid; i < D * D / 8; i += kGThreads) {
    const int row = i / (D / 8), k = 8 * (i % (D / 8));
    const float4 a = reinterpret_cast<const float4*>(r + row * D + k)[0];
    const float4 b = reinterpret_cast<const float4*>(r + row * D + k)[1];
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      hi[x] = pack_bf162(v[2 * x], v[2 * x + 1]);
      lo[x] = pack_bf162(v[2 * x] - bf16_lo_value(hi[x]), v[2 * x + 1] - bf16_hi_value(hi[x]));
    }
    const uint32_t at = tc_sw128_offset(row, k, D);
    *reinterpret_cast<uint4*>(smem + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(smem + S::kPiece + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  fence_proxy_async();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == kGWarps) {
    // ------------------------------------------------------------- tiles ahead
    uint32_t n = 0;   // tiles published
    bool ok = true;
    const int64_t total = static_cast<int64_t>(p.batch) * p.tiles_per_seq;
    auto slot_free = [&](uint32_t k) {
      const bool got = mbar_wait(empty + k % kGStages, ((k / kGStages) & 1) ^ 1, p.status);
      return __all_sync(0xffffffffu, got && !*abort_flag);
    };
    for (int64_t base = number; base < total && ok; base += static_cast<int64_t>(32) * p.ctas_per_r) {
      // a tile a lane
      const int64_t tile = base + static_cast<int64_t>(lane) * p.ctas_per_r;
      GatherTile t{};
      bool some = false;
      if (tile < total) {
        t.b = static_cast<int>(tile / p.tiles_per_seq);
        const int i = static_cast<int>(tile - static_cast<int64_t>(t.b) * p.tiles_per_seq);
        const int64_t r0 = p.row_starts[t.b], rows = p.row_starts[t.b + 1] - r0;
        const int t0 = p.first[t.b], len = p.seq_lens[t.b];
        if (rows != 0) {
          if (rows < 0 || rows > p.max_rows || r0 < 0 || r0 + rows > p.total_rows || t0 < 0 || t0 + rows > len ||
              len > static_cast<int64_t>(p.max_pages) * kPage) {
            if (p.status) atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
          } else {
            const int64_t pos0 = (t0 / kPage + static_cast<int64_t>(kGPages) * i) * kPage;
            if (pos0 < t0 + rows) {
              some = true;
              t.pos0 = static_cast<int>(pos0);
              t.lo = max(t0, t.pos0);
              t.hi = static_cast<int>(min(t0 + rows, pos0 + kGTile));
              t.row0 = r0 + pos0 - t0;
              t.c0 = min(max(t.lo, p.sink), t.hi);
              t.c1 = max(t.c0, min(t.hi, max(len - p.window, 0)));
            }
          }
        }
      }
      for (uint32_t todo = __ballot_sync(0xffffffffu, some); todo && ok; todo &= todo - 1) {
        const int src = __ffs(todo) - 1;
        GatherTile u{};
        u.b = __shfl_sync(0xffffffffu, t.b, src);
        u.pos0 = __shfl_sync(0xffffffffu, t.pos0, src);
        u.lo = __shfl_sync(0xffffffffu, t.lo, src);
        u.hi = __shfl_sync(0xffffffffu, t.hi, src);
        u.c0 = __shfl_sync(0xffffffffu, t.c0, src);
        u.c1 = __shfl_sync(0xffffffffu, t.c1, src);
        u.row0 = __shfl_sync(0xffffffffu, t.row0, src);
        // the codes of a page a lane
        const int at = u.pos0 + kPage * lane;
        const bool coded = lane < kGPages && max(at, u.c0) < min(at + kPage, u.c1);
        int id = -1;
        if (coded) id = p.coded_table[static_cast<size_t>(u.b) * p.max_pages + at / kPage];
        const bool there = coded && id >= 0 && id < p.n_coded;
        if (coded && !there && p.status) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
        u.pages = __ballot_sync(0xffffffffu, there);
        if (!(ok = slot_free(n))) break;
        const int st = n % kGStages;
        if (lane == 0) {
          tiles[st] = u;
          mbar_arrive_expect_tx(full + st, __popc(u.pages) * S::kPart);
        }
        __syncwarp();
        if (there)
          bulk_g2s(smem + S::kRing + (st * kGPages + lane) * S::kPart,
                   p.coded + (static_cast<int64_t>(id) * p.hkv + h) * F::kInt2Block + kv * S::kPart, S::kPart, full + st);
        ++n;
      }
    }
    uint32_t k = n > kGStages ? n - kGStages : 0;
    if (ok && slot_free(n)) {
      if (n >= kGStages) k = n - kGStages + 1;   // (the slot's last tile has been used)
      if (lane == 0) {
        tiles[n % kGStages].stop = 1;
        mbar_arrive_expect_tx(full + n % kGStages, 0);
      }
    }
    // no copy is in flight when the CTA ends, whatever becomes of the others
    for (; k < n; ++k) mbar_wait(full + k % kGStages, (k / kGStages) & 1, p.status);
  } else {
    // ------------------------------------------------------- codes to rows
    constexpr uint32_t idesc = tc_idesc_bf16(kGTile, D);
    constexpr int kAtom = D * 128;   // 64 channels of R's rows
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const bool leader = warp == 0 && tc_elect();
    const uint32_t r1 = smem_u32(smem), r2 = r1 + S::kPiece;
    const int64_t stride = static_cast<int64_t>(p.hkv) * D;
    uint32_t n = 0;
    for (;; ++n) {
      const int st = n % kGStages;
      const bool came = __all_sync(0xffffffffu, mbar_wait(full + st, (n / kGStages) & 1, p.status));
      if (!came) *abort_flag = 1;
      const GatherTile t = tiles[st];
      const bool end = !came || t.stop;
      const int pos = t.pos0 + row, slot = row / kPage;
      if (!end) {
        const uint8_t* blk = smem + S::kRing + (st * kGPages + slot) * S::kPart;
        if (kv) uncode<D, P, true>(blk, row % kPage, half, lanes + D);
        else uncode<D, P, false>(blk, row % kPage, half, lanes + D);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) tc_arrive(empty + st);
      }
      if (any_of(end || *abort_flag)) break;   // (all warps together)
      if (leader) {
        tc_fence_after();
#pragma unroll
        for (int piece = 0; piece < 3; ++piece) {   // y2 R1, y1 R2, y1 R1
          const uint32_t a = tmem + D + (piece == 0 ? D / 2 : 0), b = piece == 1 ? r2 : r1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma_ts(tmem, a + 8 * kk, tc_desc_sw128(b + (kk >> 2) * kAtom + (kk & 3) * 32), idesc, piece != 0 || kk != 0);
        }
        tc_commit(done);
      }
      __syncwarp();
      uint16_t* dst = p.out[kv] + ((t.row0 + row) * p.hkv + h) * D + half * (D / 2);
      if (t.c0 > t.lo || t.c1 < t.hi) {
        if (kv) plain_tokens<D, true>(p, t, h, warp, lane);
        else plain_tokens<D, false>(p, t, h, warp, lane);
        __syncwarp();
      }
      const bool got = __all_sync(0xffffffffu, mbar_wait(done, n & 1, p.status));
      if (!got) *abort_flag = 1;
      tc_fence_after();
      const bool mine = got && pos >= t.c0 && pos < t.c1 && ((t.pages >> slot) & 1u);
#pragma unroll
      for (int j = 0; j < D / 2; j += 32) {
        uint32_t y[32];
        tc_request32(lanes + half * (D / 2) + j, y);
        tc_wait_ld(y);
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = pack_bf162(__uint_as_float(y[k + 2 * i]), __uint_as_float(y[k + 2 * i + 1]));
          if (mine) store32(dst + j + k, x, p.whole);
        }
      }
      tc_fence_before();
    }
    if (*abort_flag && leader) {   // MMAs in flight finish before the CTA ends
      tc_commit(done + 1);
      mbar_wait(done + 1, 0, p.status);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tc_dealloc(tmem, 2 * D);
  }
}

template <int D, int P>
oscar_status launch_gather(const GatherParams& p, cudaStream_t st) {
  using S = GatherSmem<D, P>;
  const auto kernel = gather_kernel<D, P>;
  if (!oscar_host::allow_smem(reinterpret_cast<const void*>(kernel), S::kAlloc)) return OSCAR_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.hkv * p.ctas_per_r));
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = S::kAlloc;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // namespace oscar

using namespace oscar;

extern "C" {

oscar_status oscar_gather(const oscar_cache_desc* desc, const int32_t* seq_lens, const int32_t* first,
                          const int32_t* row_starts, int32_t batch, int64_t total_rows,
                          int32_t max_rows, void* k_out, void* v_out, void* stream) {
  oscar_status s = oscar_host::check_desc(desc, true, true);
  if (s != OSCAR_OK) return s;
  if (batch < 0 || total_rows < 0 || max_rows < 0) return OSCAR_ERR_INVALID_ARG;
  if (batch == 0 || total_rows == 0 || max_rows == 0) return OSCAR_OK;
  if (!seq_lens || !first || !row_starts || !k_out || !v_out ||
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15))
    return OSCAR_ERR_INVALID_ARG;
  if (total_rows > 0x7fffffff) return OSCAR_ERR_UNSUPPORTED;   // row_starts are int32
  // tiles that max_rows consecutive positions can touch
  const int64_t pages = (static_cast<int64_t>(max_rows) + kPage - 2) / kPage + 1;
  const int64_t tiles = (pages + kGPages - 1) / kGPages;
  if (pages * batch > 0x7fffffff || desc->num_kv_heads > 32767) return OSCAR_ERR_UNSUPPORTED;
  GatherParams p{};
  p.hkv = desc->num_kv_heads;
  p.max_pages = desc->max_pages_per_seq;
  p.batch = batch;
  p.tiles_per_seq = static_cast<int>(tiles);
  // two CTAs an SM, and no more for a rotation than there are tiles
  p.ctas_per_r = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(oscar_host::sm_count() / p.hkv, tiles * batch)));
  p.max_rows = max_rows;
  p.sink = desc->sink;
  p.window = desc->window;
  p.n_coded = desc->num_int2_pages;
  p.n_plain = desc->num_bf16_pages;
  p.total_rows = total_rows;
  p.coded = static_cast<const uint8_t*>(desc->int2_pool);
  p.plain = static_cast<const uint8_t*>(desc->bf16_pool);
  p.coded_table = desc->int2_page_table;
  p.plain_table = desc->bf16_page_table;
  p.r[0] = desc->r_k;
  p.r[1] = desc->r_v;
  p.out[0] = static_cast<uint16_t*>(k_out);
  p.out[1] = static_cast<uint16_t*>(v_out);
  p.whole = !((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31);
  p.seq_lens = seq_lens;
  p.first = first;
  p.row_starts = row_starts;
  p.status = desc->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool four = oscar_host::code_planes(desc) == 2;
  if (desc->head_dim == 128) return four ? launch_gather<128, 2>(p, st) : launch_gather<128, 1>(p, st);
  return four ? launch_gather<64, 2>(p, st) : launch_gather<64, 1>(p, st);
}

}  // extern "C"
