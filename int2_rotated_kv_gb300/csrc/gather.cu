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
// its own token's row.  A CTA, one an SM, keeps the R of one (KV head, keys or values) and walks over
// tiles of tokens, which pass through its roles:
//   warp 24       finds the next tiles that hold rows (of 32 sequences at a look), and copies the codes of their
//                 pages into a ring of stages (bulk copies, one a page);
//   warps 8-15,   codes to y1, y2 of even and odd tiles (each with its own columns of tensor memory),
//   16-23         a token and half of its channels a thread;
//   warp 25       the 3 d/16 MMAs of a tile, into one of two accumulators;
//   warps 0-3,    R's pieces, while the first codes come; then the rows of even and odd tiles to bf16 and
//   4-7           out, a token a thread;
//   warps 26, 27  the tiles' BF16 tokens, as soon as a tile is found (2000 tokens of INT2 4.7 us, by the warps that store
//                 rows 5.1, when it was measured).
// Every wait is bounded; a CTA that gives up finishes its copies and MMAs first.
//
// What bounds it: the chain of a group of uncoding warps.  INT4, 16 sequences of 2048-4096 tokens, 8 KV heads of 128: 59.3
// us, 3.8 TB/s and 1130 TFLOP/s of bf16 products (a tile's 24 MMAs take 1536 cycles), with the ALU 60%, the tensor cores
// 58% and shared memory 64% busy; bytes and products by themselves would take 34 and 34 us.  A group takes 3650 cycles for its
// every second tile, 1090 of them for codes from shared memory, and waits for 340; 10000 pass before the first products.
// Fewer instructions there (the larger piece by splitting in fp32, 64.9 us; codes by one operation less, 64.1) and the
// next words uncoded while the last are stored (65.0) changed nothing (63.8 at the time); more warps would have 56
// registers.  INT2, as many tokens of other lengths 63.8 us for INT4's 65.9.  2000 tokens of INT2, 4 heads of 64: 4.85 us.
// BF16 tokens are far from it: two warps a CTA copy them, a page each at a time, at 0.6 us a page.  With a window of 1024
// tokens those 16 sequences take 115 us (46 by their bytes), of BF16 alone 214 (60); 256 sequences of 130 tokens 177 (40).
// The same in its steps: without tensor cores 1156 us; a CTA that does one thing after another 124; rows stored by 32 bytes
// 111 (two CTAs of 8 warps an SM no faster); roles and two accumulators 74; a tile's channels in two steps, so
// that MMAs start on the first half, and keys' codes read without bank conflicts 67; R turned into pieces beside
// the first tiles 63.8; tiles with BF16 tokens shared out by themselves 59.3.
#include <algorithm>

#include "common.cuh"
#include "layout.cuh"
#include "tcgen05.cuh"

namespace oscar {

struct GatherParams {
  int hkv, max_pages, batch, max_rows, sink, window, ctas_per_r, turn;
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
constexpr int kGStages = 8;
constexpr int kGWarps = 8;                  // of a role that computes
constexpr int kGPlain = 2;                  // and of the BF16 tokens
constexpr int kGThreads = 32 * (3 * kGWarps + 2 + kGPlain);

// A tile as the computing warps need it: positions of its tokens are pos0 + row.
struct GatherTile {
  int64_t row0;      // output row of the token at pos0 (rows before lo are not written)
  int pos0, lo, hi;  // positions to be read back, [lo, hi)
  int c0, c1;        // of which [c0, c1) are codes
  int b;
  uint32_t pages;    // bit per page: its codes are there
  int stop;          // 1: there is no tile
  int plain[kGPages];   // id of a page with BF16 tokens, -1: refused
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
  static constexpr int kSteps = D / 64;                  // a tile's channels pass from role to role in so many steps
  static constexpr int kMisc = kBars + (2 * kGStages + 4 * kSteps + 4) * 8;
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

// The words of codes that a thread needs for its half of a token's channels, of the page at blk (keys' or
// values' part): x[plane][q][m] has, of group half * kOwn + m, channels 2q, 2q + 1 in its two halves (and 8, 16, 24
// further: bits 4h + 2i of the lower byte for channel 2q + 8h + 16i).
template <int D, int P, bool kValue>
__device__ __forceinline__ void load_codes(const uint8_t* blk, int t, int half, uint32_t (&x)[P][4][D / 64]) {
  using F = Fmt<D, P>;
  constexpr int kOwn = D / 64;
  const int th = t >> 3;
  // in memory, a word holds channels 2q, 2q + 1 of tokens t, t ^ 8 (keys: its bytes th and 2 + th are this
  // token's), or one channel of tokens t, t ^ 1, t ^ 8, t ^ 9 (values: two words' byte 2 (t & 1) + th)
  const uint32_t sel = kValue ? 0x0400u + (2 * (t & 1) + th) * 0x0101u : 0x0200u + th * 0x0101u;
  // eight tokens' keys lie 64 bytes apart: each two of them begin at another q, for the banks
  const int turn = kValue ? 0 : (t >> 1) & 3;
#pragma unroll
  for (int pl = 0; pl < P; ++pl) {
    const uint8_t* plane = blk + pl * F::kPlane + 4 * half * kOwn;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[2][kOwn] = {};
#pragma unroll
      for (int e = 0; e < (kValue ? 2 : 1); ++e) {
        const int lane = kValue ? 4 * (2 * q + e) + ((t >> 1) & 3) : 4 * (t & 7) + ((q + turn) & 3);
        if constexpr (kOwn == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(plane + 4 * lane * F::kWords);
          w[e][0] = u.x;
          w[e][1] = u.y;
        } else {
          w[e][0] = *reinterpret_cast<const uint32_t*>(plane + 4 * lane * F::kWords);
        }
      }
#pragma unroll
      for (int m = 0; m < kOwn; ++m) x[pl][q][m] = __byte_perm(w[0][m], w[1][m], sel);
    }
    if constexpr (!kValue) {   // back in order
#pragma unroll
      for (int m = 0; m < kOwn; ++m) {
        uint32_t y[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = turn & 1 ? x[pl][(q + 3) & 3][m] : x[pl][q][m];
#pragma unroll
        for (int q = 0; q < 4; ++q) x[pl][q][m] = turn & 2 ? y[(q + 2) & 3] : y[q];
      }
    }
  }
}

// Group half * kOwn + m of the token's channels to its row of tensor memory: y1 from column a on, y2 from a + D/2 on,
// two channels a column.
template <int D, int P, bool kValue>
__device__ __forceinline__ void uncode(const uint8_t* blk, int t, int half, int m, const uint32_t (&x)[P][4][D / 64],
                                       uint32_t a) {
  using F = Fmt<D, P>;
  const int g = half * (D / 64) + m;
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
    for (int q = 0; q < 4; ++q) {
      uint32_t c = x[0][q][m] >> (2 * i);
      if constexpr (P == 2) {   // both planes' bits of a code side by side
        const uint32_t up = i ? x[0][q][m] : x[0][q][m] << 2, down = x[P - 1][q][m] >> (2 * i);
        c = (up & 0xccccccccu) | (down & 0x33333333u);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        split_pair((c >> (4 * h)) & (P == 2 ? 0x000f000fu : 0x00030003u), two(s, s), two(z, z), hi[4 * h + q], lo[4 * h + q]);
    }
    tc_st8(a + 16 * g + 8 * i, hi);
    tc_st8(a + D / 2 + 16 * g + 8 * i, lo);
  }
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

// The BF16 tokens of page slot i of a tile, by a warp: 16 bytes a lane are channels 16 m + 2 tig, + 1, + 8, + 9 of two
// tokens (keys), or the same transposed in 8x8 blocks (values).
template <int D, bool kValue>
__device__ __forceinline__ void plain_page(const GatherParams& p, const GatherTile& t, int h, int i, int lane) {
  const int gid = lane >> 2, tig = lane & 3, id = t.plain[i];
  if (id < 0) return;
  const uint4* src = reinterpret_cast<const uint4*>(
      p.plain + (static_cast<int64_t>(id) * p.hkv + h) * Fmt<D>::kBf16Block + (kValue ? Fmt<D>::kBf16V : 0)) + lane;
  uint4 x[D / 16];
#pragma unroll
  for (int m = 0; m < D / 16; ++m) x[m] = src[32 * m];
  if constexpr (kValue) {
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {   // then as keys: tokens gid and gid + 8, channels 2 tig and 2 tig + 8
      const uint32_t up = movmatrix_trans(x[m].y), down = movmatrix_trans(x[m].z);
      x[m].x = movmatrix_trans(x[m].x);
      x[m].w = movmatrix_trans(x[m].w);
      x[m].y = down;
      x[m].z = up;
    }
  }
  uint16_t* dst = p.out[kValue] + (t.row0 * p.hkv + h) * D + 2 * tig;
#pragma unroll
  for (int th = 0; th < 2; ++th) {
    const int row = kPage * i + 8 * th + gid, pos = t.pos0 + row;
    if (pos < t.lo || pos >= t.hi || (pos >= t.c0 && pos < t.c1)) continue;
    uint16_t* out = dst + static_cast<int64_t>(row) * p.hkv * D;
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
      *reinterpret_cast<uint32_t*>(out + 16 * m) = th ? x[m].y : x[m].x;
      *reinterpret_cast<uint32_t*>(out + 16 * m + 8) = th ? x[m].w : x[m].z;
    }
  }
}

// The rest of a wait that did not end at once: false when it takes too long, or the CTA has given up.
static __device__ __noinline__ bool wait_or_give_up(uint64_t* bar, uint32_t parity, int32_t* status, volatile int* abort_flag) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort_flag) return false;
    if (global_timer_ns() - t0 > 2000000000ull) {
      *abort_flag = 1;
      if (status) atomicOr(status, OSCAR_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

template <int D, int P>
__global__ void __launch_bounds__(kGThreads, 1) gather_kernel(const __grid_constant__ GatherParams p) {
  using S = GatherSmem<D, P>;
  using F = Fmt<D, P>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  GatherTile* tiles = reinterpret_cast<GatherTile*>(smem + S::kTiles);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBars);   // a tile's codes are there
  uint64_t* empty = full + kGStages;       // and may be overwritten
  constexpr int kSteps = S::kSteps;
  uint64_t* yfull = empty + kGStages;      // y of an even (odd) tile is there, [kSteps] each
  uint64_t* done = yfull + 2 * kSteps;     // its MMAs are done, likewise
  uint64_t* xempty = done + 2 * kSteps;    // its product has been read
  uint64_t* rfull = xempty + 2;            // R's pieces are there
  uint64_t* last = rfull + 1;              // MMAs in flight after a give-up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int which = blockIdx.x / p.ctas_per_r, number = blockIdx.x - which * p.ctas_per_r;
  const int h = which >> 1, kv = which & 1;

  if (tid == 0) {
    for (int i = 0; i < kGStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, kGWarps + kGWarps / 2 + kGPlain);
    }
    for (int i = 0; i < 2 * kSteps; ++i) {
      mbar_init(yfull + i, kGWarps);
      mbar_init(done + i, 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(xempty + i, kGWarps / 2);
    mbar_init(rfull, kGWarps);
    mbar_init(last, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tc_alloc(tmem_slot, 4 * D);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;   // products of even and odd tiles (d columns each), then their y
  pdl_wait();
  pdl_trigger();

  // A wait of a warp together; false: give up.
  auto wait = [&](uint64_t* b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, mbar_try_wait(b, parity & 1u) || wait_or_give_up(b, parity & 1u, p.status, abort_flag));
  };
  auto arrive = [&](uint64_t* b) {
    __syncwarp();
    if (lane == 0) tc_arrive(b);
  };

  if (warp == 3 * kGWarps) {
    // ------------------------------------------------------------- tiles ahead
    // The tiles that hold rows go round the rotation's CTAs: the fast ones, of codes alone, in order; the slow ones, with BF16
    // tokens (2 us for one page, 4.7 for eight, where codes take 1.5; less between fast ones), by themselves, each round
    // turned against the one before.  (Handed out by number of sequence and announced rows, one-tile sequences beside a
    // longer one fell to one CTA: 255 of 100 tokens and one of 1130, 8 heads of 128, 1071 us for 136.  All in one order,
    // the slow tiles of sequences of as many tiles as there are CTAs do: 64 of 1132 tokens 298 us for 121, 1024 of 300 1262
    // for 969.)
    uint32_t n = 0;   // tiles published
    bool ok = true;
    // lanes with a sequence, up to a power of two
    const int among = p.batch < 32 ? 1 << (32 - __clz(p.batch - 1)) : 32;
    const int ctas = p.ctas_per_r;
    // of a look's fast tiles this CTA's first; of its slow ones the first of the present round (or one before the look's), and
    // this CTA's place in it
    int next_fast = ctas - 1 - number, round0 = 0, place = number;
    const auto slow_of = [&](int round) {   // this CTA's in the round that is so many on
      const int x = (place - p.turn * round) % ctas;
      return round0 + round * ctas + (x < 0 ? x + ctas : x);
    };
    // the lane (of those with a sequence) that holds number x of what `upto` counts
    const auto holder = [&](int upto, int x) {
      int of = 0;
#pragma unroll 1
      for (int o = among >> 1; o > 0; o >>= 1)
        if (__shfl_sync(0xffffffffu, upto, of + o - 1) <= x) of += o;
      return of;
    };
    for (int64_t b0 = 0; b0 < p.batch && ok; b0 += 32) {
      // a sequence a lane
      const int b = static_cast<int>(b0) + lane;
      int t0 = 0, end = 0, len = 0;
      int r0 = 0, before = 0, slow = 0, fast = 0;   // its tiles: the fast ones come after `before` of the slow ones
      if (b0 + lane < p.batch) {
        r0 = p.row_starts[b];
        const int64_t rows = static_cast<int64_t>(p.row_starts[b + 1]) - r0;
        t0 = p.first[b];
        len = p.seq_lens[b];
        if (rows != 0) {
          if (rows < 0 || rows > p.max_rows || r0 < 0 || r0 + rows > p.total_rows || t0 < 0 || t0 + rows > len ||
              len > static_cast<int64_t>(p.max_pages) * kPage) {
            if (p.status) atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
          } else {
            end = t0 + static_cast<int>(rows);
            const int count = static_cast<int>((t0 % kPage + rows + kGTile - 1) / kGTile), page0 = t0 / kPage;
            const int recent = min(max(max(len - p.window, 0) / kPage - page0, 0) / kGPages, count);   // the window's first
            before = min(t0 < p.sink ? ((p.sink - 1) / kPage - page0) / kGPages + 1 : 0, recent);
            fast = recent - before;
            slow = count - fast;
          }
        }
      }
      int upto_slow = slow, upto_fast = fast;   // up to and with the lane's sequence
#pragma unroll 1
      for (int o = 1; o < among; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, upto_slow, o), v = __shfl_up_sync(0xffffffffu, upto_fast, o);
        if (lane >= o) {
          upto_slow += u;
          upto_fast += v;
        }
      }
      const int all_slow = __shfl_sync(0xffffffffu, upto_slow, among - 1);
      const int all_fast = __shfl_sync(0xffffffffu, upto_fast, among - 1);
      // no more tiles than CTAs: one each, found with fewer steps (2000 tokens of INT2 4.85 us, like the others 5.3)
      const bool few = p.batch <= 32 && all_slow + all_fast <= ctas;
      int slows = 0, fasts = few && number < all_slow + all_fast, skip = 0;   // this CTA's; skip: had in the look before
      if (!few) {
        if (all_fast > next_fast) fasts = (all_fast - next_fast + ctas - 1) / ctas;
        const int rounds = (all_slow - round0 + ctas - 1) / ctas;
        skip = slow_of(0) < 0;
        if (rounds > skip) slows = rounds - skip - (slow_of(rounds - 1) >= all_slow);
      }
      // the slow ones are spread among the fast ones: of the first q tiles, q slows / all are slow (in 32 bits: a CTA
      // has far fewer than 2^26 tiles)
      const uint32_t all = slows + fasts;
      uint32_t had = 0, rest = 0;   // of the first `base`; what the division has left
      for (uint32_t base = 0; base < all && ok; base += 32) {
        // a tile a lane: its number among the slow or the fast ones, its sequence's lane and its number there
        const bool some = base + lane < all;
        int of, i;
        if (__builtin_expect(few, 1)) {
          of = holder(upto_slow + upto_fast, number);
          i = number - __shfl_sync(0xffffffffu, upto_slow + upto_fast - slow - fast, of);
        } else {
          const uint32_t v = rest + lane * slows, q = v / all, before_it = had + q;
          const bool is_slow = v - q * all + slows >= all;
          const int slow_at = slow_of(skip + before_it), fast_at = next_fast + static_cast<int>(base + lane - before_it) * ctas;
          const int of_slow = holder(upto_slow, slow_at), of_fast = holder(upto_fast, fast_at);
          of = is_slow ? of_slow : of_fast;
          const int x = slow_at - __shfl_sync(0xffffffffu, upto_slow - slow, of_slow);
          const int y = fast_at - __shfl_sync(0xffffffffu, upto_fast - fast, of_fast);
          const int head = __shfl_sync(0xffffffffu, before, of), its_fast = __shfl_sync(0xffffffffu, fast, of);
          i = !is_slow ? head + y : x < head ? x : x + its_fast;
          had += (rest + 32 * slows) / all;
          rest = (rest + 32 * slows) % all;
        }
        for (uint32_t todo = __ballot_sync(0xffffffffu, some); todo && ok;) {
          // the next four of them, eight lanes each (one at a time, the look-ups of page ids bound the walk)
          uint32_t left = todo;
          for (int k = 0; k < (lane >> 3); ++k) left &= left - 1;
          const int src = left ? __ffs(left) - 1 : 0;
          const int from_lane = __shfl_sync(0xffffffffu, of, src);
          const int from = __shfl_sync(0xffffffffu, t0, from_lane), to = __shfl_sync(0xffffffffu, end, from_lane);
          GatherTile u{};
          u.b = static_cast<int>(b0) + from_lane;
          u.pos0 = (from / kPage + kGPages * __shfl_sync(0xffffffffu, i, src)) * kPage;
          u.lo = max(from, u.pos0);
          u.hi = u.pos0 + min(to - u.pos0, kGTile);
          u.row0 = static_cast<int64_t>(__shfl_sync(0xffffffffu, r0, from_lane)) + u.pos0 - from;
          u.c0 = min(max(u.lo, p.sink), u.hi);
          u.c1 = max(u.c0, min(u.hi, max(__shfl_sync(0xffffffffu, len, from_lane) - p.window, 0)));
          // a page a lane: its codes, and the id of its BF16 tokens
          const int pg = lane & 7, at = u.pos0 + kPage * pg;
          const bool coded = left && max(at, u.c0) < min(at + kPage, u.c1);
          const bool plain = left && (max(at, u.lo) < min(at + kPage, u.c0) || max(at, u.c1) < min(at + kPage, u.hi));
          const size_t entry = static_cast<size_t>(u.b) * p.max_pages + at / kPage;
          int id = -1, id16 = -1;
          if (coded) id = p.coded_table[entry];
          if (plain) id16 = p.plain_table[entry];
          const bool there = coded && id >= 0 && id < p.n_coded, there16 = plain && id16 >= 0 && id16 < p.n_plain;
          if (((coded && !there) || (plain && !there16)) && p.status) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
          const uint32_t pages = __ballot_sync(0xffffffffu, there);
          for (int g = 0; g < 4 && todo; ++g, todo &= todo - 1, ++n) {
            const int st = n % kGStages;
            if (!(ok = wait(empty + st, (n / kGStages) + 1))) break;
            if (lane == 8 * g) {
              u.pages = (pages >> (8 * g)) & 0xffu;
              tiles[st] = u;
            }
            __syncwarp();
            if (lane >> 3 == g) tiles[st].plain[pg] = there16 ? id16 : -1;
            __syncwarp();
            if (lane == 8 * g) mbar_arrive_expect_tx(full + st, __popc(u.pages) * S::kPart);
            __syncwarp();
            if (lane >> 3 == g && there)
              bulk_g2s(smem + S::kRing + (st * kGPages + pg) * S::kPart,
                       p.coded + (static_cast<int64_t>(id) * p.hkv + h) * F::kInt2Block + kv * S::kPart, S::kPart, full + st);
          }
        }
      }
      next_fast += fasts * ctas - all_fast;
      const int whole = (all_slow - round0) / ctas;
      place = slow_of(whole) - round0 - whole * ctas;
      round0 += whole * ctas - all_slow;
    }
    // the end, for the warps of even and of odd tiles
    uint32_t k = n > kGStages ? n - kGStages : 0;
    for (int e = 0; e < 2 && ok; ++e) {
      const uint32_t m = n + e;
      if (!(ok = wait(empty + m % kGStages, (m / kGStages) + 1))) break;
      if (m >= kGStages) k = m - kGStages + 1;   // (the slot's last tile has been used)
      if (lane == 0) {
        tiles[m % kGStages].stop = 1;
        mbar_arrive_expect_tx(full + m % kGStages, 0);
      }
      __syncwarp();
    }
    // no copy is in flight when the CTA ends, whatever becomes of the others
    for (; k < n; ++k) mbar_wait(full + k % kGStages, (k / kGStages) & 1, p.status);
  } else if (warp == 3 * kGWarps + 1) {
    // ------------------------------------------------------------------ MMAs
    constexpr uint32_t idesc = tc_idesc_bf16(kGTile, D);
    constexpr int kAtom = D * 128;   // 64 channels of R's rows
    const bool leader = tc_elect();
    const uint32_t r1 = smem_u32(smem), r2 = r1 + S::kPiece;
    bool ok = wait(rfull, 0);
    for (uint32_t n = 0; ok; ++n) {
      const uint32_t e = n & 1;
      if (!(ok = wait(full + n % kGStages, n / kGStages))) break;
      if (tiles[n % kGStages].stop) break;
      if (!(ok = wait(xempty + e, (n >> 1) + 1))) break;
      const uint32_t x = tmem + e * D, y = tmem + 2 * D + e * D;
#pragma unroll
      for (int m = 0; m < kSteps; ++m) {   // groups m and kSteps + m of 32 channels
        if (!(ok = wait(yfull + e * kSteps + m, n >> 1))) break;
        if (leader) {
          tc_fence_after();
#pragma unroll
          for (int piece = 0; piece < 3; ++piece) {   // y2 R1, y1 R2, y1 R1
            const uint32_t a = y + (piece == 0 ? D / 2 : 0), b = piece == 1 ? r2 : r1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int kk = 2 * (m + (k >> 1) * kSteps) + (k & 1);
              tc_mma_ts(x, a + 8 * kk, tc_desc_sw128(b + (kk >> 2) * kAtom + (kk & 3) * 32), idesc,
                        m != 0 || piece != 0 || k != 0);
            }
          }
          tc_commit(done + e * kSteps + m);
        }
        __syncwarp();
      }
    }
    if (!ok && leader) {   // MMAs in flight finish before the CTA ends
      tc_commit(last);
      mbar_wait(last, 0, p.status);
    }
  } else if (warp > 3 * kGWarps + 1) {
    // ------------------------------------------------------------ BF16 tokens
    for (uint32_t n = 0;; ++n) {
      const int st = n % kGStages;
      if (!wait(full + st, n / kGStages)) break;
      const GatherTile& t = tiles[st];
      if (t.stop) break;
      if (t.c0 > t.lo || t.c1 < t.hi) {
#pragma unroll 1
        for (int i = warp & 1; i < kGPages; i += kGPlain) {
          if (kv) plain_page<D, true>(p, t, h, i, lane);
          else plain_page<D, false>(p, t, h, i, lane);
          __syncwarp();
        }
      }
      arrive(empty + st);
    }
  } else if (warp >= kGWarps) {
    // ------------------------------------------------------------- codes to y
    const int row = 32 * (warp & 3) + lane, half = (warp >> 2) & 1, odd = (warp - kGWarps) / kGWarps;
    const uint32_t y = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 2 * D + odd * D;
    for (uint32_t n = odd;; n += 2) {
      const int st = n % kGStages;
      if (!wait(full + st, n / kGStages) || tiles[st].stop) break;
      const uint8_t* blk = smem + S::kRing + (st * kGPages + row / kPage) * S::kPart;
      uint32_t x[P][4][kSteps];
      if (kv) load_codes<D, P, true>(blk, row % kPage, half, x);
      else load_codes<D, P, false>(blk, row % kPage, half, x);
      bool ok = true;
#pragma unroll
      for (int m = 0; m < kSteps; ++m) {
        // y of the tile before has been used
        if (!(ok = wait(done + odd * kSteps + m, (n >> 1) + 1))) break;
        tc_fence_after();
        if (kv) uncode<D, P, true>(blk, row % kPage, half, m, x, y);
        else uncode<D, P, false>(blk, row % kPage, half, m, x, y);
        tc_wait_st();
        tc_fence_before();
        arrive(yfull + odd * kSteps + m);
      }
      if (!ok) break;
      if (lane == 0) tc_arrive(empty + st);
    }
  } else {
    // ----------------------------------------------------------- rows to bf16
    // R as two bf16 pieces
    const float* r = p.r[kv] + static_cast<size_t>(h) * D * D;
#pragma unroll
    for (int j = 0; j < D * D / 8 / (32 * kGWarps); ++j) {
      const int i = tid + 32 * kGWarps * j, at_row = i / (D / 8), k = 8 * (i % (D / 8));
      const float4 a = reinterpret_cast<const float4*>(r + at_row * D + k)[0];
      const float4 b = reinterpret_cast<const float4*>(r + at_row * D + k)[1];
      const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        hi[c] = pack_bf162(v[2 * c], v[2 * c + 1]);
        lo[c] = pack_bf162(v[2 * c] - bf16_lo_value(hi[c]), v[2 * c + 1] - bf16_hi_value(hi[c]));
      }
      const uint32_t at = tc_sw128_offset(at_row, k, D);
      *reinterpret_cast<uint4*>(smem + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(smem + S::kPiece + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    fence_proxy_async();
    arrive(rfull);
    const int row = 32 * (warp & 3) + lane, odd = warp >> 2;
    const uint32_t x = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + odd * D;
    for (uint32_t n = odd;; n += 2) {
      const int st = n % kGStages;
      if (!wait(full + st, n / kGStages)) break;
      const GatherTile& t = tiles[st];
      if (t.stop || !wait(done + odd * kSteps + kSteps - 1, n >> 1)) break;
      tc_fence_after();
      const int pos = t.pos0 + row;
      uint16_t* dst = p.out[kv] + ((t.row0 + row) * p.hkv + h) * D;
      const bool mine = pos >= t.c0 && pos < t.c1 && ((t.pages >> (row / kPage)) & 1u);
#pragma unroll
      for (int j = 0; j < D; j += 32) {
        uint32_t y[32];
        tc_request32(x + j, y);
        tc_wait_ld(y);
        if (j + 32 == D) {
          tc_fence_before();
          arrive(xempty + odd);
        }
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack_bf162(__uint_as_float(y[k + 2 * i]), __uint_as_float(y[k + 2 * i + 1]));
          if (mine) store32(dst + j + k, w, p.whole);
        }
      }
      arrive(empty + st);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tc_dealloc(tmem, 4 * D);
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
  oscar_status s = oscar_host::check_desc(desc, true, true, false);
  if (s != OSCAR_OK) return s;
  if (batch < 0 || total_rows < 0 || max_rows < 0) return OSCAR_ERR_INVALID_ARG;
  if (batch == 0 || total_rows == 0 || max_rows == 0) return OSCAR_OK;
  if (!seq_lens || !first || !row_starts || !k_out || !v_out ||
      ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 15))
    return OSCAR_ERR_INVALID_ARG;
  if (total_rows > 0x7fffffff) return OSCAR_ERR_UNSUPPORTED;   // row_starts are int32
  // pages that so many consecutive positions can touch, and tiles of them
  const auto pages = [](int64_t rows) { return (rows + kPage - 2) / kPage + 1; };
  if (pages(max_rows) * batch > 0x7fffffff || desc->num_kv_heads > 32767) return OSCAR_ERR_UNSUPPORTED;
  const int64_t tiles = (pages(std::min<int64_t>(max_rows, total_rows)) + kGPages - 1) / kGPages;   // (no sequence has more)
  GatherParams p{};
  p.hkv = desc->num_kv_heads;
  p.max_pages = desc->max_pages_per_seq;
  p.batch = batch;
  // a CTA an SM, and no more for a rotation than there are tiles
  p.ctas_per_r = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(oscar_host::sm_count() / (2 * p.hkv), tiles * batch)));
  p.turn = std::max(1, p.ctas_per_r * 5 / 8);   // (near the golden section, so that turns come back to a CTA late)
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
