// Attention over the 8-bit cache for many query columns of a KV head (a chunk of
// prefill, a long verification): tiles of 128 (row, query head) columns on tcgen05.
//
// Same mathematics, unit division and partial results as kv8_attention.cu.  Per tile
// of 128 tokens (8 pages):
//   S = Q K^T   M = 128 columns of queries, N = 128 tokens, K = d   (Q, K in shared memory)
//   w = 2^(s_K fac S + log2 s_V - m)                                (a thread per query)
//   O += w V    M = 128, N = d, K = 128 tokens      (w in tensor memory, V in shared memory)
// Here the bound is arithmetic, so the codes are turned into fp16 operands once per
// tile and CTA (exact: integers up to 127, or e4m3 values) and the MMAs run from
// shared and tensor memory.  The value scale of a page rides in the exponent: w is
// p s_V, rounded once to fp16, and the sum of p is that of w / s_V.
//
// One CTA per SM, 14 warps:
//   0-3, 4-7  softmax of even and odd tiles ("streams", each with its own S, w, O in
//             tensor memory, own maxima and sums, merged at the unit's end): reads S
//             twice, for the maximum and for w, which overwrites S;
//   8-11      raw pages -> fp16 K and V tiles, 128-byte swizzled, two of each; the
//             queries of a unit;
//   12        page ids and bulk copies, a ring of 7 x 4 pages (keys and values apart);
//   13        MMAs from one lane.
// Every wait is bounded; a CTA that gives up finishes its copies and MMAs first.
// Tensor memory: S0, S1 (128 columns each), O0, O1 (d each); w in the first half of S.
// What bounds it: shared memory, 1536 cycles a tile at d = 128 (fp16 tiles written once
// and read by the MMAs, Q read per tile), above the 1024 cycles of the MMAs.
#include <algorithm>

#include "kv8_units.cuh"
#include "tcgen05.cuh"

namespace oscar {

constexpr int kRWarps = 14;
constexpr int kRThreads = 32 * kRWarps;
constexpr int kRTile = 128;        // tokens of a tile
constexpr int kREntries = 7;       // raw ring: 4 pages of keys or of values each
constexpr int kRHidden = 0x7fff0000;   // position of a page slot that holds no page

template <int D>
struct RowsSmem {
  using F = Kv8Fmt<D>;
  static constexpr int kTile16 = kRTile * D * 2;           // fp16 K or V tile, or Q
  static constexpr int kEntry = 4 * F::kCodes + 64;        // codes, and 4 x 16 bytes of scales
  static constexpr int kK = 0;
  static constexpr int kV = 2 * kTile16;
  static constexpr int kQ = 4 * kTile16;
  static constexpr int kRaw = 5 * kTile16;
  static constexpr int kMeta = kRaw + kREntries * kEntry;  // float4 [4][8]: s_K, log2 s_V, 1/s_V, position
  static constexpr int kFac = kMeta + 512;                 // float [2][128]
  static constexpr int kMl = kFac + 1024;                  // float2 [2][2][128]
  static constexpr int kValid = kMl + 4096;                // int [kREntries], then int bad[4]
  static constexpr int kBars = kValid + 64;
  static constexpr int kMisc = kBars + 40 * 8;
  static constexpr int kBytes = kMisc + 64;
  static constexpr int kAlloc = kBytes + 1024;             // the base is rounded up to 1024 bytes
  static_assert(kMeta % 16 == 0, "metadata is read by 16 bytes");
};

struct RowsBars {
  uint64_t rawfull[kREntries], rawempty[kREntries];
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];   // fp16 tiles, by tile number
  uint64_t sfull[2], pfull[2], wdone[2];               // S ready, w ready, w used, by stream
  uint64_t qfull[2], oempty[2];                        // by unit: queries ready, O read
  uint64_t qempty, odone, mlfull;
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
    tiles = tail ? n8 / 8 + 1 + (n8 % 8 == 7 ? 1 : 0) : (n8 + 7) / 8;
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
    unit0 += t.pages;
    if (++h == p.hkv) {
      h = 0;
      t = entry_of<kRowsNT>(p, ++e);
    }
    p0 = 0;
    set();
    return true;
  }
  // Page slots of tile i: pages in slots 0 .. n - 1, the tail's two slots from `tail_slot`
  // (-1: none; it does not cross the border of four slots), slots in use.
  __device__ __forceinline__ void slots(int i, int& n, int& tail_slot, int& used) const {
    n = max(0, min(8, n8 - 8 * i));
    tail_slot = tail && i == tiles - 1 ? ((n & 3) == 3 ? n + 1 : n) : -1;
    used = tail_slot >= 0 ? tail_slot + 2 : n;
  }
};

// Sixteen codes as fp16 pairs in order, exact.
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

// Power of two that brings a bf16 magnitude (bits) to [2^7, 2^8), as its exponent.
__device__ __forceinline__ int scale_up(uint32_t amax) {
  return amax ? max(-96, min(100, 134 - static_cast<int>(amax >> 7))) : 0;
}
__device__ __forceinline__ float power_of_two(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
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

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kRThreads, 1)
kv8_rows_kernel(const __grid_constant__ Kv8Params p, int min_share) {
  using S = RowsSmem<D>;
  using F = Kv8Fmt<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t scratch[kRWarps];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  RowsBars* bar = reinterpret_cast<RowsBars*>(smem + S::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  volatile int* n_copies = reinterpret_cast<volatile int*>(smem + S::kMisc + 8);
  float4* meta = reinterpret_cast<float4*>(smem + S::kMeta);
  float* facs = reinterpret_cast<float*>(smem + S::kFac);
  float2* mls = reinterpret_cast<float2*>(smem + S::kMl);
  volatile int* valid = reinterpret_cast<volatile int*>(smem + S::kValid);
  volatile int* bad_tail = valid + kREntries;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kREntries; ++i) {
      mbar_init(&bar->rawfull[i], 1);
      mbar_init(&bar->rawempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar->kfull[i], 4);
      mbar_init(&bar->kempty[i], 1);
      mbar_init(&bar->vfull[i], 4);
      mbar_init(&bar->vempty[i], 1);
      mbar_init(&bar->sfull[i], 1);
      mbar_init(&bar->pfull[i], 4);
      mbar_init(&bar->wdone[i], 1);
      mbar_init(&bar->qfull[i], 4);
      mbar_init(&bar->oempty[i], 8);
    }
    mbar_init(&bar->qempty, 1);
    mbar_init(&bar->odone, 1);
    mbar_init(&bar->mlfull, 8);
    *abort_flag = 0;
    *n_copies = 0;
    fence_mbar_init();
  }
  if (warp == 13) tc_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  Share sh;
  const bool any = find_share<kRowsNT, kRWarps>(p, min_share, scratch, sh);
  if (!any && tid == 0) p.info[blockIdx.x] = make_int4(0, 0, 0, 0);
  Walk u;
  if (any) u.start(sh);
  // A wait of one thread, or of a warp together (one answer for all lanes); false: give up.
  // No barrier completes a second phase before all that wait for the first have passed.
  auto wait1 = [&](uint64_t* b, uint32_t parity) -> bool {
    const bool ok = mbar_wait(b, parity & 1u, p.status) && !*abort_flag;
    if (!ok) *abort_flag = 1;
    return ok;
  };
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(b, parity & 1u, p.status) && !*abort_flag);
    if (!ok) *abort_flag = 1;
    return ok;
  };
  auto arrive = [&](uint64_t* b) {
    __syncwarp();
    if (lane == 0) tc_arrive(b);
  };

  if (any && warp == 12) {
    // ---------------------------------------------------------------- copies
    uint32_t r = 0;
    for (bool go = true; go; go = u.next(p)) {
      if (u.tiles == 0) continue;
      const int32_t* row = p.page_table + static_cast<size_t>(u.t.b) * p.max_pages + u.p0;
      // ids of 32 pages from 32 * window, and of the 32 after them
      auto ids_of = [&](int window) { const int i = 32 * window + lane; return i < u.n8 ? row[i] : -1; };
      int window = 0, ids0 = ids_of(0), ids1 = ids_of(1);
      const int64_t tail_id = p.tail_ids ? p.tail_ids[u.t.b] : u.t.b;
      const bool tail_ok = tail_id >= 0 && tail_id < p.n_tails;
      const uint8_t* tail = p.tail + ((tail_ok ? tail_id : 0) * p.hkv + u.h) * F::kTailBytes;
      bool ok = true;
      // keys of tile i + 1, then values of tile i
      for (int step = 0; step < 2 * u.tiles && ok; ++step) {
        const bool keys = step == 0 || (step & 1 && step < 2 * u.tiles - 1);
        const int i = keys ? (step + 1) / 2 : (step == 2 * u.tiles - 1 ? u.tiles - 1 : step / 2 - 1);
        int n, tail_slot, used;
        u.slots(i, n, tail_slot, used);
        for (; !keys && i / 4 > window; ++window) {
          ids0 = ids1;
          ids1 = ids_of(window + 2);
        }
        for (int half = 0; half < (used + 3) / 4; ++half, ++r) {
          const int en = r % kREntries;
          if (!(ok = wait(&bar->rawempty[en], r / kREntries + 1))) break;
          // lanes 0-3: codes of slots 4 half + lane; lanes 4-7: their scales
          const int slot = 4 * half + (lane & 3);
          const int id = __shfl_sync(0xffffffffu, i / 4 == window ? ids0 : ids1, (8 * i + slot) & 31);
          const bool page = slot < n, ends = slot == tail_slot;
          const bool good = page ? id >= 0 && id < p.n_pages : ends && tail_ok;
          const uint32_t mask = __ballot_sync(0xffffffffu, lane < 4 && good);
          if (lane < 4 && (page || ends) && !good && keys && p.status)
            atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
          const int pages = __popc(__ballot_sync(0xffffffffu, lane < 4 && page));
          const int tails = __popc(__ballot_sync(0xffffffffu, lane < 4 && ends));
          if (lane == 0) {
            valid[en] = static_cast<int>(mask);
            mbar_arrive_expect_tx(&bar->rawfull[en],
                                  pages * (F::kCodes + (keys ? 16 : 0)) + tails * 2 * F::kCodes);
            *n_copies = static_cast<int>(r) + 1;
          }
          __syncwarp();
          uint8_t* dst = smem + S::kRaw + en * S::kEntry;
          const uint8_t* blk = p.pool + (static_cast<int64_t>(page && good ? id : 0) * p.hkv + u.h) * F::kBlock;
          if (lane < 4) {
            if (page) bulk_g2s(dst + lane * F::kCodes, blk + (keys ? 0 : F::kCodes), F::kCodes, &bar->rawfull[en]);
            else if (ends) bulk_g2s(dst + lane * F::kCodes, tail + (keys ? 0 : 2 * F::kCodes), 2 * F::kCodes, &bar->rawfull[en]);
          } else if (lane < 8 && keys && page) {
            bulk_g2s(dst + 4 * F::kCodes + 16 * (lane & 3), blk + F::kScales, 16, &bar->rawfull[en]);
          }
        }
      }
      if (!ok) break;
    }
  } else if (any && warp == 13) {
    // ------------------------------------------------------------------ MMAs
    if (lane == 0) {
      constexpr uint32_t id_s = tc_idesc_f16(kRTile, kRTile), id_o = tc_idesc_f16(kRTile, D);
      constexpr int kAtom = kRTile * 128;   // 64 channels of K or Q
      constexpr int kAtomV = D * 128;       // 64 tokens of V
      uint32_t g0 = 0, seg = 0;             // tiles before this unit, units with tiles
      uint32_t count[2] = {0, 0};           // tiles of each stream whose O has been issued
      bool ok = true;
      for (bool go = true; go && ok; go = u.next(p)) {
        if (u.tiles == 0) continue;
        if (!(ok = wait1(&bar->qfull[seg & 1], seg >> 1))) break;
        for (int i = 0; i <= u.tiles && ok; ++i) {
          if (i < u.tiles) {   // S of tile i, once w of the stream's tile before has been used
            const uint32_t g = g0 + i, buf = g & 1, st = i & 1;
            ok = wait1(&bar->kfull[buf], g >> 1);
            if (ok && count[st]) ok = wait1(&bar->wdone[st], count[st] - 1);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a0 = sb + S::kQ, b0 = sb + S::kK + buf * S::kTile16;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * kAtom + (kk & 3) * 32;
              tc_mma(tmem + st * kRTile, tc_desc_sw128(a0 + off), tc_desc_sw128(b0 + off), id_s, kk != 0);
            }
            tc_commit(&bar->sfull[st]);
            tc_commit(&bar->kempty[buf]);
            if (i == u.tiles - 1) tc_commit(&bar->qempty);
          }
          if (i > 0) {         // O of tile i - 1
            const uint32_t g = g0 + i - 1, buf = g & 1, st = (i - 1) & 1;
            ok = wait1(&bar->pfull[st], count[st]) && wait1(&bar->vfull[buf], g >> 1);
            if (ok && i <= 2 && seg > 0)   // the unit before has been read
              ok = wait1(&bar->oempty[(seg - 1) & 1], (seg - 1) >> 1);
            if (!ok) break;
            ++count[st];
            tc_fence_after();
            const uint32_t b0 = sb + S::kV + buf * S::kTile16;
#pragma unroll
            for (int kk = 0; kk < kRTile / 16; ++kk)
              tc_mma_ts(tmem + 2 * kRTile + st * D, tmem + st * kRTile + 8 * kk,
                        tc_desc_sw128(b0 + (kk >> 2) * kAtomV + (kk & 3) * 32), id_o, i > 2 || kk != 0);
            tc_commit(&bar->vempty[buf]);
            tc_commit(&bar->wdone[st]);
          }
        }
        if (!ok) break;
        tc_commit(&bar->odone);
        g0 += u.tiles;
        ++seg;
      }
      if (!ok) {   // MMAs in flight finish before the CTA ends: the phase after odone's next
        tc_commit(&bar->odone);
        mbar_wait(&bar->odone, seg & 1u, p.status);
      }
    }
  } else if (any && warp >= 8) {
    // -------------------------------------------------------- fp16 operands
    const int w = warp - 8;
    uint32_t r = 0, g0 = 0, seg = 0;
    for (bool go = true; go; go = u.next(p)) {
      if (u.tiles == 0) continue;
      if (!wait(&bar->qempty, seg + 1)) break;
      // and the unit before the last has been read (what is kept by unit comes round again)
      if (seg > 1 && !wait(&bar->oempty[seg & 1], (seg - 2) >> 1)) break;
      {   // a query column per thread: fp16 scaled by a power of two
        const int rr = 32 * w + lane;
        const uint16_t* src = column(p, u.t, u.h, u.t.tile * 128 + rr, D);
        uint4 q[D / 8];
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          q[c] = src ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0, 0, 0, 0);
          const uint32_t x[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t lo = x[j] & 0x7fffu, hi = (x[j] >> 16) & 0x7fffu;
            top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
          }
        }
        const int up = scale_up(top);
        const float mul = power_of_two(up);
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(smem + S::kQ + tc_sw128_offset(rr, 8 * c, kRTile)) =
              make_uint4(half_pair(q[c].x, mul), half_pair(q[c].y, mul), half_pair(q[c].z, mul),
                         half_pair(q[c].w, mul));
        facs[(seg & 1) * 128 + rr] = p.scale_log2 * power_of_two(-up);
        fence_proxy_async();
        arrive(&bar->qfull[seg & 1]);
      }
      const int n_tail = u.t.len % kPage;
      const int64_t tail_id = p.tail_ids ? p.tail_ids[u.t.b] : u.t.b;
      const bool tail_ok = tail_id >= 0 && tail_id < p.n_tails;
      const uint16_t* tail = reinterpret_cast<const uint16_t*>(
          p.tail + ((tail_ok ? tail_id : 0) * p.hkv + u.h) * F::kTailBytes);
      int up_v = 0;
      bool ok = true;
      for (int step = 0; step < 2 * u.tiles && ok; ++step) {   // in the order of the copies
        const bool keys = step == 0 || (step & 1 && step < 2 * u.tiles - 1);
        const int i = keys ? (step + 1) / 2 : (step == 2 * u.tiles - 1 ? u.tiles - 1 : step / 2 - 1);
        const uint32_t g = g0 + i, buf = g & 1;
        int n, tail_slot, used;
        u.slots(i, n, tail_slot, used);
        uint8_t* dst = smem + (keys ? S::kK : S::kV) + buf * S::kTile16;
        if (!(ok = wait(keys ? &bar->kempty[buf] : &bar->vempty[buf], (g >> 1) + 1))) break;
        for (int half = 0; half < 2; ++half) {
          const int slot = 4 * half + w;
          const bool page = slot < n, ends = slot == tail_slot;
          const bool copies = half < (used + 3) / 4;
          const int en = r % kREntries;
          if (copies && !(ok = wait(&bar->rawfull[en], r / kREntries))) break;
          const uint8_t* raw = smem + S::kRaw + en * S::kEntry + w * F::kCodes;
          const bool good = copies && ((valid[en] >> w) & 1);
          if (keys) {
            float4 m = make_float4(0.f, 0.f, 0.f, __int_as_float(kRHidden));
            if (page) {
              const uint4* chunks = reinterpret_cast<const uint4*>(raw);
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                const uint4 x = chunks[32 * c + lane];
                uint32_t o[8];
                code_pairs<kE4m3>(x.x, o[0], o[1]);
                code_pairs<kE4m3>(x.y, o[2], o[3]);
                code_pairs<kE4m3>(x.z, o[4], o[5]);
                code_pairs<kE4m3>(x.w, o[6], o[7]);
                const int row = 16 * slot + 2 * (lane >> 2) + (c & 1);
                const int ch = 64 * (c >> 1) + 16 * (lane & 3);
                // lanes of odd pairs of rows store their halves in the other order: no bank conflicts
                const int first = (lane >> 2) & 1;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int part = k ^ first;
                  *reinterpret_cast<uint4*>(dst + tc_sw128_offset(row, ch + 8 * part, kRTile)) =
                      part ? make_uint4(o[4], o[5], o[6], o[7]) : make_uint4(o[0], o[1], o[2], o[3]);
                }
              }
              const float2 sc = *reinterpret_cast<const float2*>(
                  smem + S::kRaw + en * S::kEntry + 4 * F::kCodes + 16 * w);
              // a page of zeros (scale 0) still counts its tokens: weight 1, values 0
              const bool live = sc.y > 0.f;
              m = make_float4(sc.x, live ? log2f(sc.y) : 0.f, live ? 1.f / sc.y : 1.f,
                              __int_as_float(good ? (u.p0 + 8 * i + slot) * kPage : kRHidden));
            } else if (ends) {
              bool odd;
              const int up = scale_up(tail_magnitude<D>(tail, 0, n_tail, lane, odd));
              const uint32_t top = tail_magnitude<D>(tail + F::kTailHalf, 1, n_tail, lane, odd);
              up_v = scale_up(top);
              if (lane == 0) bad_tail[seg & 3] = odd && tail_ok;
              const float mul = power_of_two(up);
              const uint4* chunks = reinterpret_cast<const uint4*>(raw);
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                const int row = 16 * slot + 2 * (lane >> 2) + (c & 1);
                const int ch = 64 * (c >> 1) + 16 * (lane & 3);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                  const uint4 x = chunks[2 * (32 * c + lane) + part];
                  *reinterpret_cast<uint4*>(dst + tc_sw128_offset(row, ch + 8 * part, kRTile)) =
                      make_uint4(half_pair(x.x, mul), half_pair(x.y, mul), half_pair(x.z, mul),
                                 half_pair(x.w, mul));
                }
              }
              m = make_float4(power_of_two(-up), static_cast<float>(-up_v), power_of_two(up_v),
                              __int_as_float(good ? u.t.len / kPage * kPage : kRHidden));
            }
            if (lane == 0) meta[(g & 3) * 8 + slot] = m;
          } else {
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {   // 4 channels x 8 tokens
              const int pair = 32 * c + lane, cg = pair >> 1, tg = pair & 1;
              uint32_t o[4][4];
              if (page) {
                const uint4* chunks = reinterpret_cast<const uint4*>(raw) + 2 * pair;
                const uint4 x = chunks[0], y = chunks[1];
                const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  code_pairs<kE4m3>(a[k], o[k][0], o[k][1]);
                  code_pairs<kE4m3>(b[k], o[k][2], o[k][3]);
                }
              } else if (ends) {
                // what is not finite, or not a token, becomes 0 (the epilogue adds the former)
                up_v = __shfl_sync(0xffffffffu, up_v, 0);
                const float mul = power_of_two(up_v);
                const uint4* chunks = reinterpret_cast<const uint4*>(raw) + 4 * pair;
#pragma unroll
                for (int half4 = 0; half4 < 2; ++half4) {
                  const uint4 x = chunks[2 * half4], y = chunks[2 * half4 + 1];
                  const uint32_t a[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const int t0 = 8 * tg + 4 * half4 + 2 * (k & 1);
                    uint32_t v = a[k];
                    if (t0 >= n_tail || (v & 0x7fffu) >= 0x7f80u) v &= 0xffff0000u;
                    if (t0 + 1 >= n_tail || ((v >> 16) & 0x7fffu) >= 0x7f80u) v &= 0xffffu;
                    o[k >> 1][2 * half4 + (k & 1)] = half_pair(v, mul);
                  }
                }
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0u;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(dst + tc_sw128_offset(4 * cg + k, 16 * slot + 8 * tg, D)) =
                    make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
            }
          }
          if (copies) {
            arrive(&bar->rawempty[en]);
            ++r;
          }
        }
        if (!ok) break;
        fence_proxy_async();
        arrive(keys ? &bar->kfull[buf] : &bar->vfull[buf]);
      }
      if (!ok) break;
      g0 += u.tiles;
      ++seg;
    }
  } else if (any) {
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
      int vis = 0;
      if (gcol < p.cols) vis = p.q_pos ? row_limit(p, u.t.b, row, u.t.len) : u.t.len;
      if (u.p0 == 0 && u.h == 0 && p.status && st == 0) {
        const int len = p.seq_lens[u.t.b];
        if (u.t.tile == 0 && rr == 0 && (len < 0 || len > p.max_len))
          atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
        if (p.q_pos && gcol < p.cols && p.q_pos[static_cast<size_t>(u.t.b) * p.m_rows + row] >= u.t.len)
          atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
      }
      float m = kLowest, l = 0.f, top = kLowest, a0 = 0.f, a1 = 0.f;
      if (u.tiles > 0) {
        if (!wait(&bar->qfull[seg & 1], seg >> 1)) break;
        const float fac = facs[(seg & 1) * 128 + rr];
        bool ok = true;
        for (int i = st; i < u.tiles; i += 2) {
          if (!(ok = wait(&bar->sfull[st], count))) break;
          ++count;
          tc_fence_after();
          const float4* mt = meta + ((g0 + i) & 3) * 8;
          bool hides = false;
#pragma unroll
          for (int j = 0; j < 8; ++j) hides |= __float_as_int(mt[j].w) + kPage > vis;
          const bool masked = __any_sync(0xffffffffu, hides);
          // the largest exponent of this tile
          float big = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float s[32];
            tc_ld32(ts + 32 * c, s);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 pm = mt[2 * c + j];
              float x = -INFINITY;
              if (masked) {
                const int seen = vis - __float_as_int(pm.w);
#pragma unroll
                for (int k = 0; k < 16; ++k) x = fmaxf(x, k < seen ? s[16 * j + k] : -INFINITY);
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) x = fmaxf(x, s[16 * j + k]);
              }
              // (a hidden page's -inf times a scale of 0 would be NaN)
              big = fmaxf(big, x == -INFINITY ? x : fmaf(x, pm.x * fac, pm.y));
            }
          }
          const bool over = big > m + kLag;
          if (__any_sync(0xffffffffu, over)) {
            const float up = over ? big : m;
            const float a = over ? fast_exp2(m - up) : 1.f;
            m = up;
            l *= a;
            if (i > 1) {   // the stream's O so far (its last MMA finished before this S began)
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tc_ld16(to + 16 * c, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * a);
                tc_st16(to + 16 * c, o);
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float s[32];
            tc_ld32(ts + 32 * c, s);
            uint32_t out[16];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float4 pm = mt[2 * c + j];
              const float f = pm.x * fac, off = pm.y - m;
              const int seen = masked ? vis - __float_as_int(pm.w) : kPage;
              float sum = 0.f;
#pragma unroll
              for (int k = 0; k < 16; k += 2) {
                float x0 = fast_exp2(fmaf(s[16 * j + k], f, off));
                float x1 = fast_exp2(fmaf(s[16 * j + k + 1], f, off));
                if (masked) {
                  x0 = k < seen ? x0 : 0.f;
                  x1 = k + 1 < seen ? x1 : 0.f;
                }
                sum += x0 + x1;
                out[8 * j + k / 2] = pack_half2(x0, x1);
              }
              if (!masked || seen > 0) l = fmaf(sum, pm.z, l);
            }
            tc_st16(ts + 16 * c, out);   // columns of S that have been read
          }
          tc_wait_st();
          tc_fence_before();
          arrive(&bar->pfull[st]);
        }
        if (!ok) break;
        // the other stream's maximum and sum
        float2* ml = mls + (seg & 1) * 256;
        ml[128 * st + rr] = make_float2(m, l);
        arrive(&bar->mlfull);
        if (!wait(&bar->mlfull, seg) || !wait(&bar->odone, seg)) break;
        tc_fence_after();
        const float2 other = ml[128 * (1 - st) + rr];
        top = fmaxf(m, other.x);
        const float mine = fast_exp2(m - top), theirs = fast_exp2(other.x - top);
        l = l * mine + other.y * theirs;
        a0 = st ? theirs : mine;
        a1 = st ? mine : theirs;
      }
      // channels [st * D/2, (st + 1) * D/2) of this column
      const bool complete = u.p0 == 0 && u.p1 == u.t.pages;
      float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (u.p0 == 0 ? 1 : 0)) * kv8_slot<D, kRowsNT>();
      const int tail0 = u.t.len / kPage * kPage;
      const bool odd = u.tail && u.tiles > 0 && bad_tail[seg & 3];
      const int64_t tail_id = p.tail_ids ? p.tail_ids[u.t.b] : u.t.b;
      const uint16_t* tail = reinterpret_cast<const uint16_t*>(p.tail + (tail_id * p.hkv + u.h) * F::kTailBytes) +
          F::kTailHalf;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {   // 16 channels
        const int ch = st * (D / 2) + 16 * c;
        float o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = 0.f;
        if (u.tiles > 0) {
          uint32_t x[16];
          tc_ld16(lanes + 2 * kRTile + ch, x);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __uint_as_float(x[k]) * a0;
        }
        if (u.tiles > 1) {
          uint32_t x[16];
          tc_ld16(lanes + 2 * kRTile + D + ch, x);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = fmaf(__uint_as_float(x[k]), a1, o[k]);
        }
        if (odd) {   // values of the tail that are not finite, to the rows that see them
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
                  make_uint4(pack_bf162(o[k] * inv, o[k + 1] * inv), pack_bf162(o[k + 2] * inv, o[k + 3] * inv),
                             pack_bf162(o[k + 4] * inv, o[k + 5] * inv), pack_bf162(o[k + 6] * inv, o[k + 7] * inv));
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4*>(slot + rr * D + ch + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
            if (ch == 0) *reinterpret_cast<float2*>(slot + 128 * D + 2 * rr) = make_float2(top, l);
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

  // ---- after a give-up, copies in flight land before the CTA ends (the MMAs' own thread
  // has waited for them)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && tid == 0) {
    const int n = *n_copies;
    for (int r = max(0, n - kREntries); r < n; ++r)
      mbar_wait(&bar->rawfull[r % kREntries], static_cast<uint32_t>(r / kREntries) & 1u, p.status);
  }
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
}

template <int D, bool kE4m3>
oscar_status launch_rows(const Kv8Params& p, int64_t ctas, int min_share, cudaStream_t st) {
  const auto kernel = kv8_rows_kernel<D, kE4m3>;
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

oscar_status run_kv8_rows(const Kv8Params& p, int head_dim, bool e4m3, int64_t ctas, int min_share,
                          cudaStream_t st) {
  if (head_dim == 128)
    return e4m3 ? launch_rows<128, true>(p, ctas, min_share, st) : launch_rows<128, false>(p, ctas, min_share, st);
  return e4m3 ? launch_rows<64, true>(p, ctas, min_share, st) : launch_rows<64, false>(p, ctas, min_share, st);
}

}  // namespace oscar
