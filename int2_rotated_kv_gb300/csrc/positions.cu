// What a serving step derives from request lengths and positions: page tables and
// per-token lists, and the rotary embedding of queries and keys.
//
// oscar_extend_pages.  A table holds pages for the tokens t < n - hold_back of a
// sequence of n tokens: pages(n) = max(0, ceil((n - hold_back) / 16)).  One CTA forms
// both exclusive prefix sums over the batch (rows, new pages) and advances the
// lengths and the free-list cursor; the rows and the new table entries follow in
// the same CTA when the row lists are short, else in a grid of their own that finds each row's
// sequence by bisection of the prefix sums.  Bound by latency (a chain of a scan and
// two dependent loads) for a decode step, by the 16 bytes written per row for a
// large prefill.  Measured: 256 sequences, a token each 4.6 us; 0.8 million rows
// 7.4 us, 1750 GB/s of lists that stay in L2.
//
// oscar_rope.  For a rotated pair (a, b) at position m with frequency f turns per
// token: a' = A (a cos 2 pi m f - b sin 2 pi m f), b' = A (b cos + a sin).  f is held
// as a 64-bit fraction, so m f modulo one turn is the low 64 bits of an integer
// product: no rounding at all whatever the position; the upper 32 bits of it go to
// sincospif.  cos and sin are formed once per (token, pair) in shared memory and
// shared by all heads.  Bound by HBM: 2 bytes read and 2 written per value.  Measured,
// 16411 tokens, 32 + 8 heads of 128: 336 MB in 56.3 us, 5970 GB/s; one token 2.4 us.
#include <algorithm>
#include <cmath>

#include "common.cuh"

namespace oscar {

inline cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                     cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// ------------------------------------------------------------------ page tables

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
// Prefix sums that a filling CTA bisects in shared memory (0.8 million rows of 256 sequences: 7.4 us
// against 8.6 from L1).
constexpr int kSharedStarts = 2048;
// Rows that the scan's CTA writes itself, with the table entries of the step.  Itself against a grid of its own: 256 rows 4.7 us
// against 5.6, 2048 rows 4.6 against 5.5, 4096 rows 5.4 against 5.3, 8192 rows 7.6 against 5.7.
constexpr int64_t kInlineRows = 4096;

struct PagesParams {
  int batch, max_pages, hold;
  int64_t n_free, max_rows;
  int32_t* table;
  const int32_t* lens;
  const int32_t* new_tokens;
  const int32_t* free_pages;
  const int32_t* cursor;
  int32_t* lens_after;
  int32_t* page_starts;
  int32_t* row_starts;
  int32_t* seq_ids;
  int32_t* positions;
  int64_t* slots;
  int32_t* status;
  int fill;   // the scan's CTA also writes rows and table entries
  int wide;   // the row lists take 16-byte stores
};

__device__ __forceinline__ int pages_held(int n, int hold) {
  return n > hold ? (n - hold - 1) / kPage + 1 : 0;
}

// Index of the sequence, `lo` or one behind it, whose [starts[b], starts[b + 1]) holds i (starts
// ascend).
__device__ __forceinline__ int sequence_of(const int32_t* starts, int batch, int i, int lo = 0) {
  int hi = batch;   // starts[lo] <= i < starts[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Page of logical index `pg` that the step gives to sequence b, from the free list.
__device__ __forceinline__ int fresh_page(const PagesParams& p, int first, int pg, int held_before) {
  const int64_t at = static_cast<int64_t>(first) + pg - held_before;
  return at < p.n_free ? p.free_pages[at] : -1;
}

// Many new table entries by the scan's CTA, as it has them when the caller takes few row lists of
// many new tokens, or none: a warp takes runs of 32 * kRun, a lane every 32nd of them, with its loads in
// flight together and a bisection only where a sequence ends.  256 prompts of 4096 tokens, 65280
// entries: 18 us, where an entry at a time takes 56.  (Out of line, and not for the few of a decode
// step or for a grid, which it makes slower: 4.6 us to 5.0, 7.4 to 8.9.)
constexpr int kManyEntries = 8192;
static __device__ __noinline__ void fill_entries(const PagesParams& p, int first, int fresh) {
  constexpr int kRun = 8;
  const int32_t* free_pages = p.free_pages + first;   // (not read where there are none)
  const int here = static_cast<int>(max(static_cast<int64_t>(0), min(p.n_free - first, static_cast<int64_t>(fresh))));
  for (int64_t j = 32 * kRun * (threadIdx.x >> 5) + (threadIdx.x & 31); j < fresh; j += kScanThreads * kRun) {
    const int j0 = static_cast<int>(j), left = (fresh - j0 - 1) / 32 + 1;   // entries of this lane
    int b = 0, end = j0, last = 0;   // entries [.., end) are sequence b's, of which [.., last) have a column
    int32_t* row = nullptr;
    int32_t* dst[kRun];
    int id[kRun];
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      dst[k] = nullptr;
      if (k < left) {
        const int at = j0 + 32 * k;
        if (at >= end) {
          b = sequence_of(p.page_starts, p.batch, first + at, b);
          const int begin = p.page_starts[b] - first;
          end = p.page_starts[b + 1] - first;
          const int held = pages_held(p.lens_after[b] - (p.row_starts[b + 1] - p.row_starts[b]), p.hold);
          row = p.table + static_cast<int64_t>(b) * p.max_pages + held - begin;
          last = p.max_pages - held + begin;
        }
        if (at < last) dst[k] = row + at;
        id[k] = at < here ? free_pages[at] : -1;
      }
    }
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (dst[k]) *dst[k] = id[k];
  }
}

// Rows and new table entries, `i` of `n` workers.  A worker writes runs of four rows:
// one bisection, then the next sequence where its rows end.  row_starts, page_starts: the
// step's, or a copy of them in shared memory.  kScan: by the scan's CTA.
template <bool kScan>
__device__ __forceinline__ void fill_rows(const PagesParams& p, const int32_t* row_starts,
                                          const int32_t* page_starts, int64_t i, int64_t n) {
  const int64_t rows = row_starts[p.batch];
  for (int64_t r0 = 4 * i; r0 < p.max_rows; r0 += 4 * n) {
    int b = -1, end = -1, start = 0, before = 0, held = 0, holds = 0;   // of the run's current sequence
    int ids[4], pos[4];
    int64_t slot[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = r0 + j;
      ids[j] = pos[j] = -1;
      slot[j] = -1;
      if (r >= rows || r >= p.max_rows) continue;
      if (r >= end) {
        if (b < 0) b = sequence_of(row_starts, p.batch, static_cast<int>(r));
        else while (row_starts[b + 1] <= r) ++b;
        start = row_starts[b];
        end = row_starts[b + 1];
        const int after = p.lens_after[b];
        before = after - (end - start);
        held = pages_held(before, p.hold);
        holds = min(pages_held(after, p.hold), p.max_pages);
      }
      ids[j] = b;
      pos[j] = before + static_cast<int>(r) - start;
      const int pg = pos[j] / kPage;
      if (p.slots && pg < holds) {
        const int id = pg >= held ? fresh_page(p, page_starts[b], pg, held)
                                  : p.table[static_cast<size_t>(b) * p.max_pages + pg];
        if (id >= 0) slot[j] = static_cast<int64_t>(id) * kPage + pos[j] % kPage;
      }
    }
    if (p.wide && r0 + 4 <= p.max_rows) {
      *reinterpret_cast<int4*>(p.seq_ids + r0) = make_int4(ids[0], ids[1], ids[2], ids[3]);
      *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.slots) {
        reinterpret_cast<longlong2*>(p.slots + r0)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(p.slots + r0)[1] = make_longlong2(slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r0 + j >= p.max_rows) break;
        p.seq_ids[r0 + j] = ids[j];
        p.positions[r0 + j] = pos[j];
        if (p.slots) p.slots[r0 + j] = slot[j];
      }
    }
  }
  const int first = page_starts[0];
  const int64_t fresh = static_cast<int64_t>(page_starts[p.batch]) - first;
  if (kScan && fresh > kManyEntries) {
    fill_entries(p, first, static_cast<int>(fresh));
    return;
  }
  for (int64_t j = i; j < fresh; j += n) {
    const int at = first + static_cast<int>(j);
    const int b = sequence_of(page_starts, p.batch, at);
    const int after = p.lens_after[b];
    const int held = pages_held(after - (row_starts[b + 1] - row_starts[b]), p.hold);
    const int pg = held + at - page_starts[b];
    if (pg < p.max_pages)
      p.table[static_cast<size_t>(b) * p.max_pages + pg] = at < p.n_free ? p.free_pages[at] : -1;
  }
}

__global__ void __launch_bounds__(kScanThreads) extend_scan_kernel(const __grid_constant__ PagesParams p) {
  __shared__ int64_t sums[2][kScanThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t cursor = *p.cursor;   // read before page_starts, which may hold it, is written
  // totals before this turn; a cursor that cannot be used, or has run past the list, gives no page
  int64_t rows = 0, pages = cursor < 0 ? p.n_free : min(cursor, p.n_free);
  bool refused = cursor < 0;
  for (int b0 = 0; b0 < p.batch; b0 += kScanThreads) {
    const int b = b0 + tid;
    int n = 0, need = 0, before = 0;
    if (b < p.batch) {
      before = p.lens[b];
      n = p.new_tokens[b];
      // a sequence with an impossible length or more tokens than its table holds gets nothing
      const int64_t after = static_cast<int64_t>(before) + n;
      if (before < 0 || n < 0 || after > 0x7fffffff ||
          after - p.hold > static_cast<int64_t>(p.max_pages) * kPage) {
        n = 0;
        refused = true;
      }
      need = pages_held(before + n, p.hold) - pages_held(before, p.hold);
    }
    int64_t r = n, g = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, r, o), w = __shfl_up_sync(0xffffffffu, g, o);
      if (lane >= o) { r += u; g += w; }
    }
    if (lane == 31) { sums[0][warp] = r; sums[1][warp] = g; }
    __syncthreads();
    if (warp == 0) {
      int64_t u = sums[0][lane], w = sums[1][lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, u, o), y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) { u += x; w += y; }
      }
      sums[0][lane] = u;
      sums[1][lane] = w;
    }
    __syncthreads();
    const int64_t r0 = rows + r - n + (warp ? sums[0][warp - 1] : 0);
    const int64_t g0 = pages + g - need + (warp ? sums[1][warp - 1] : 0);
    if (b < p.batch) {
      // totals beyond int32 are cut here and reported; rows stop at max_rows anyway
      p.row_starts[b] = static_cast<int>(min(r0, static_cast<int64_t>(0x7fffffff)));
      p.page_starts[b] = static_cast<int>(min(g0, static_cast<int64_t>(0x7fffffff)));
      p.lens_after[b] = before + n;
    }
    rows += sums[0][kScanThreads / 32 - 1];
    pages += sums[1][kScanThreads / 32 - 1];
    __syncthreads();
  }
  if (tid == 0) {
    p.row_starts[p.batch] = static_cast<int>(min(rows, static_cast<int64_t>(0x7fffffff)));
    p.page_starts[p.batch] = static_cast<int>(min(pages, static_cast<int64_t>(0x7fffffff)));
  }
  if (p.status) {
    int bits = 0;
    if (refused || (tid == 0 && rows > p.max_rows)) bits |= OSCAR_DEVERR_SEQ_LEN;
    if (tid == 0 && pages > p.n_free) bits |= OSCAR_DEVERR_NO_PAGES;
    if (bits) atomicOr(p.status, bits);
  }
  if (p.fill) {
    __syncthreads();   // this CTA's global writes above are read back
    fill_rows<true>(p, p.row_starts, p.page_starts, tid, kScanThreads);
  }
}

__global__ void __launch_bounds__(kFillThreads) extend_fill_kernel(const __grid_constant__ PagesParams p) {
  __shared__ int32_t starts[2][kSharedStarts];
  pdl_wait();
  pdl_trigger();
  const bool few = p.batch < kSharedStarts;
  if (few) {
    for (int b = threadIdx.x; b <= p.batch; b += kFillThreads) {
      starts[0][b] = p.row_starts[b];
      starts[1][b] = p.page_starts[b];
    }
    __syncthreads();
  }
  fill_rows<false>(p, few ? starts[0] : p.row_starts, few ? starts[1] : p.page_starts,
                   static_cast<int64_t>(blockIdx.x) * kFillThreads + threadIdx.x,
                   static_cast<int64_t>(gridDim.x) * kFillThreads);
}

// ----------------------------------------------------------------------- rotary

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;   // per CTA, at most

struct RopeParams {
  int hq, hkv, d, half, tokens;   // half: rotated pairs per head; tokens per CTA
  int64_t n, q_stride, k_stride, q_out_stride, k_out_stride;
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  const int32_t* positions;
  const uint64_t* phases;
  float amplitude, sign;
  int copy;   // the output is not the input: unrotated channels are copied
};

// Two pairs (low and high halves of a and b); r: cos, sin of the first, of the second.
__device__ __forceinline__ void rotate2(uint32_t a, uint32_t b, float4 r, uint32_t& x, uint32_t& y) {
  const float a0 = bf16_lo_value(a), a1 = bf16_hi_value(a);
  const float b0 = bf16_lo_value(b), b1 = bf16_hi_value(b);
  x = pack_bf162(a0 * r.x - b0 * r.y, a1 * r.z - b1 * r.w);
  y = pack_bf162(b0 * r.x + a0 * r.y, b1 * r.z + a1 * r.w);
}

// One item of a head vector: a run of rotated pairs (it < pairs), else of channels that
// are copied.  kInter: pairs (2i, 2i + 1), else (i, i + half).  kVec: 16-byte accesses
// (the rotated part in runs of 8 channels, pointers and strides 16-byte aligned), else
// one pair, or one channel, at a time.  Loading and storing are apart so that a thread
// has the loads of two items in flight.
template <bool kInter, bool kVec>
struct RopeItem {
  uint4 a, b;
  uint16_t* dst;
  const float2* c;

  __device__ __forceinline__ void load(const RopeParams& p, const float2* cs, int64_t row, int t, int h,
                                       int it, int pairs) {
    const uint16_t* src;
    if (h < p.hq) {
      src = p.q + row * p.q_stride + h * p.d;
      dst = p.q_out + row * p.q_out_stride + h * p.d;
    } else {
      src = p.k + row * p.k_stride + (h - p.hq) * p.d;
      dst = p.k_out + row * p.k_out_stride + (h - p.hq) * p.d;
    }
    c = cs + t * p.half;
    constexpr int kRun = kVec ? 8 : 1;
    if (it >= pairs) {
      const int ch = 2 * p.half + (it - pairs) * kRun;
      dst += ch;
      if constexpr (kVec) a = *reinterpret_cast<const uint4*>(src + ch);
      else a.x = src[ch];
    } else if constexpr (kVec) {
      dst += 8 * it;
      c += (kInter ? 4 : 8) * it;
      a = *reinterpret_cast<const uint4*>(src + 8 * it);
      if constexpr (!kInter) b = *reinterpret_cast<const uint4*>(src + p.half + 8 * it);
    } else {
      const int at = kInter ? 2 * it : it;
      dst += at;
      c += it;
      a.x = src[at];
      b.x = src[at + (kInter ? 1 : p.half)];
    }
  }

  __device__ __forceinline__ void store(const RopeParams& p, int it, int pairs) const {
    if (it >= pairs) {
      if constexpr (kVec) *reinterpret_cast<uint4*>(dst) = a;
      else *dst = static_cast<uint16_t>(a.x);
    } else if constexpr (!kVec) {
      const float x = bf16_to_float(static_cast<uint16_t>(a.x));
      const float y = bf16_to_float(static_cast<uint16_t>(b.x));
      dst[0] = __bfloat16_as_ushort(__float2bfloat16_rn(x * c->x - y * c->y));
      dst[kInter ? 1 : p.half] = __bfloat16_as_ushort(__float2bfloat16_rn(y * c->x + x * c->y));
    } else if constexpr (kInter) {
      const float4* r = reinterpret_cast<const float4*>(c);   // two pairs each
      const float4 r0 = r[0], r1 = r[1];
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(turn(a.x, r0.x, r0.y), turn(a.y, r0.z, r0.w), turn(a.z, r1.x, r1.y),
                     turn(a.w, r1.z, r1.w));
    } else {
      const float4* r = reinterpret_cast<const float4*>(c);
      uint4 x, y;
      rotate2(a.x, b.x, r[0], x.x, y.x);
      rotate2(a.y, b.y, r[1], x.y, y.y);
      rotate2(a.z, b.z, r[2], x.z, y.z);
      rotate2(a.w, b.w, r[3], x.w, y.w);
      *reinterpret_cast<uint4*>(dst) = x;
      *reinterpret_cast<uint4*>(dst + p.half) = y;
    }
  }

  static __device__ __forceinline__ uint32_t turn(uint32_t w, float c, float s) {
    const float x = bf16_lo_value(w), y = bf16_hi_value(w);
    return pack_bf162(x * c - y * s, y * c + x * s);
  }
};

// cos and sin of a CTA's tokens, and their positions, in shared memory.
__device__ __forceinline__ void rope_angles(const RopeParams& p, int64_t t0, int nt, float2* cs, int* pos) {
  if (threadIdx.x < nt) pos[threadIdx.x] = p.positions[t0 + threadIdx.x];
  for (int i = threadIdx.x; i < nt * p.half; i += kRopeThreads) {
    const int t = i / p.half, j = i - t * p.half;
    const int m = p.positions[t0 + t];
    // m * phase modulo 2^64: the position in the turn; its upper half as a signed fraction
    const uint64_t turn = p.phases[j] * static_cast<uint64_t>(static_cast<uint32_t>(m));
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * (1.f / 2147483648.f), &s, &c);
    cs[i] = make_float2(p.amplitude * c, p.amplitude * p.sign * s);
  }
  __syncthreads();
}

template <bool kInter, bool kVec>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float2 cs[];   // [tokens][half]: A cos, A sin
  __shared__ int pos[kRopeTokens];
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.n - t0));
  rope_angles(p, t0, nt, cs, pos);
  const int heads = p.hq + p.hkv;
  constexpr int kRun = kVec ? 8 : 1;
  // items of a head: rotated pairs in runs, then the unrotated channels in runs
  const int pairs = kVec ? (kInter ? p.half / 4 : p.half / 8) : p.half;
  const int items = pairs + (p.copy ? (p.d - 2 * p.half) / kRun : 0);
  // A thread keeps its item and steps over heads and tokens: one division in all.
  // Items beyond the threads go round again; threads left over do nothing.
  const int step = max(1, kRopeThreads / items);
  const int first = threadIdx.x / items;
  if (first >= step) return;
  for (int it = threadIdx.x - first * items; it < items; it += kRopeThreads) {
    int t = 0, h = first;
    auto settle = [&] {   // on to the next head that exists, in a row that is not padding
      while (true) {
        for (; h >= heads && t < nt; h -= heads) ++t;
        if (t >= nt || pos[t] >= 0) return;
        h += step;
      }
    };
    settle();
    while (t < nt) {
      RopeItem<kInter, kVec> x, y;
      x.load(p, cs, t0 + t, t, h, it, pairs);
      h += step;
      settle();
      const bool two = t < nt;
      if (two) {
        y.load(p, cs, t0 + t, t, h, it, pairs);
        h += step;
        settle();
      }
      x.store(p, it, pairs);
      if (two) y.store(p, it, pairs);
    }
  }
}

// Runs of 8 channels (16-byte accesses) where the rotated part is not made of such runs:
// a run's partners may lie across two others, so the head vectors of a round pass through
// shared memory.  A round: as many head vectors as the CTA has threads for.
template <bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_runs_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float2 cs[];   // [tokens][half]: A cos, A sin
  __shared__ __align__(16) uint16_t rows[8 * kRopeThreads];
  __shared__ int pos[kRopeTokens];
  pdl_wait();
  pdl_trigger();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.n - t0));
  rope_angles(p, t0, nt, cs, pos);
  const int heads = p.hq + p.hkv, items = p.d / 8, step = kRopeThreads / items;
  const int vec = threadIdx.x / items, c0 = 8 * (threadIdx.x - vec * items);
  int t = 0, h = vec;
  for (int r = 0; r < nt * heads; r += step) {
    for (; h >= heads && t < nt; h -= heads) ++t;
    const bool mine = vec < step && t < nt && pos[t] >= 0;
    const int64_t row = t0 + t;
    const bool is_q = h < p.hq;
    if (mine)
      *reinterpret_cast<uint4*>(rows + vec * p.d + c0) = *reinterpret_cast<const uint4*>(
          (is_q ? p.q + row * p.q_stride + h * p.d : p.k + row * p.k_stride + (h - p.hq) * p.d) + c0);
    __syncthreads();
    if (mine) {
      const uint16_t* x = rows + vec * p.d;
      const float2* w = cs + t * p.half;
      uint32_t out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = c0 + 2 * k + e;
          const bool first = kInter ? e == 0 : c < p.half;
          const int pair = kInter ? c >> 1 : first ? c : c - p.half;
          y[e] = bf16_to_float(x[c]);
          if (c < 2 * p.half) {
            const float other = bf16_to_float(x[kInter ? c ^ 1 : first ? c + p.half : c - p.half]);
            const float2 a = w[pair];
            y[e] = first ? y[e] * a.x - other * a.y : y[e] * a.x + other * a.y;
          }
        }
        out[k] = pack_bf162(y[0], y[1]);
      }
      *reinterpret_cast<uint4*>((is_q ? p.q_out + row * p.q_out_stride + h * p.d
                                      : p.k_out + row * p.k_out_stride + (h - p.hq) * p.d) + c0) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncthreads();
    h += step;
  }
}

}  // namespace oscar

using namespace oscar;

extern "C" {

oscar_status oscar_extend_pages(int32_t* page_table, int32_t max_pages_per_seq, const int32_t* lens,
                                const int32_t* new_tokens, int32_t batch, int32_t hold_back,
                                const int32_t* free_pages, int64_t num_free, const int32_t* cursor,
                                int32_t* lens_after, int32_t* page_starts, int32_t* row_starts,
                                int32_t* seq_ids, int32_t* positions, int64_t* slots,
                                int64_t max_rows, int32_t* status, void* stream) {
  if (batch < 0 || max_pages_per_seq < 1 || hold_back < 0 || num_free < 0 || max_rows < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (batch == 0) return OSCAR_OK;
  if (!page_table || !lens || !new_tokens || !cursor || !lens_after || !page_starts || !row_starts ||
      (num_free > 0 && !free_pages) || (max_rows > 0 && (!seq_ids || !positions)))
    return OSCAR_ERR_INVALID_ARG;
  if (num_free > 0x7fffffff || max_rows > 0x7fffffff || batch == 0x7fffffff)
    return OSCAR_ERR_UNSUPPORTED;
  PagesParams p{};
  p.batch = batch;
  p.max_pages = max_pages_per_seq;
  p.hold = hold_back;
  p.n_free = num_free;
  p.max_rows = max_rows;
  p.table = page_table;
  p.lens = lens;
  p.new_tokens = new_tokens;
  p.free_pages = free_pages;
  p.cursor = cursor;
  p.lens_after = lens_after;
  p.page_starts = page_starts;
  p.row_starts = row_starts;
  p.seq_ids = seq_ids;
  p.positions = positions;
  p.slots = slots;
  p.status = status;
  p.fill = max_rows <= kInlineRows ? 1 : 0;
  p.wide = ((reinterpret_cast<uintptr_t>(seq_ids) | reinterpret_cast<uintptr_t>(positions) |
             reinterpret_cast<uintptr_t>(slots)) & 15) == 0;
  cudaLaunchAttribute attr;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg = pdl_config(dim3(1), dim3(kScanThreads), 0, st, &attr);
  if (cudaLaunchKernelEx(&cfg, extend_scan_kernel, p) != cudaSuccess) return OSCAR_ERR_CUDA;
  if (!p.fill) {
    const int64_t want = (max_rows + 4 * kFillThreads - 1) / (4 * kFillThreads);
    const int64_t most = static_cast<int64_t>(oscar_host::sm_count()) * 8;
    cfg = pdl_config(dim3(static_cast<unsigned>(std::min(want, most))), dim3(kFillThreads), 0, st, &attr);
    if (cudaLaunchKernelEx(&cfg, extend_fill_kernel, p) != cudaSuccess) return OSCAR_ERR_CUDA;
  }
  return OSCAR_OK;
}

oscar_status oscar_rope_phases(double base, int32_t rotary_dim, double factor, int32_t original_len,
                               double low_turns, double high_turns, uint64_t* phases_out) {
  if (!(base > 1.0) || !std::isfinite(base) || rotary_dim < 2 || rotary_dim % 2 || !phases_out ||
      !(factor >= 1.0) || !std::isfinite(factor) || original_len < 0)
    return OSCAR_ERR_INVALID_ARG;
  if (original_len > 0 && !(std::isfinite(low_turns) && std::isfinite(high_turns) && low_turns < high_turns))
    return OSCAR_ERR_INVALID_ARG;
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    // turns per token; every value is below 1 / (2 pi)
    double f = std::pow(base, -2.0 * i / rotary_dim) / 6.283185307179586;
    if (original_len > 0) {
      const double keep = std::min(1.0, std::max(0.0, (f * original_len - low_turns) /
                                                          (high_turns - low_turns)));
      f = (1.0 - keep) * f / factor + keep * f;
    } else {
      f /= factor;
    }
    phases_out[i] = static_cast<uint64_t>(std::nearbyint(std::ldexp(f, 64)));
  }
  return OSCAR_OK;
}

oscar_status oscar_rope(const void* q, const void* k, const int32_t* positions,
                        const uint64_t* phases, int64_t n, int32_t num_q_heads,
                        int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim,
                        int32_t interleaved, float amplitude, int32_t inverse, int64_t q_stride,
                        int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride, void* q_out,
                        void* k_out, void* stream) {
  if (n < 0 || num_q_heads < 0 || num_kv_heads < 0 || num_q_heads + static_cast<int64_t>(num_kv_heads) < 1 ||
      head_dim < 2 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim ||
      !std::isfinite(amplitude) || (interleaved & ~1) || (inverse & ~1))
    return OSCAR_ERR_INVALID_ARG;
  if (n == 0) return OSCAR_OK;
  if (!positions || !phases || (num_q_heads && (!q || !q_out)) || (num_kv_heads && (!k || !k_out)))
    return OSCAR_ERR_INVALID_ARG;
  const int64_t heads = static_cast<int64_t>(num_q_heads) + num_kv_heads;
  if (head_dim > 1024 || heads > 65536) return OSCAR_ERR_UNSUPPORTED;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim;
  const int64_t kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if ((num_q_heads && (q_stride < qw || q_out_stride < qw)) ||
      (num_kv_heads && (k_stride < kw || k_out_stride < kw)))
    return OSCAR_ERR_INVALID_ARG;
  if ((num_q_heads && q_out == q && q_out_stride != q_stride) ||
      (num_kv_heads && k_out == k && k_out_stride != k_stride))
    return OSCAR_ERR_INVALID_ARG;   // in place: row by row
  RopeParams p{};
  p.hq = num_q_heads;
  p.hkv = num_kv_heads;
  p.d = head_dim;
  p.half = rotary_dim / 2;
  p.n = n;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.q_stride = num_q_heads ? q_stride : 0;
  p.k_stride = num_kv_heads ? k_stride : 0;
  p.q_out_stride = num_q_heads ? q_out_stride : 0;
  p.k_out_stride = num_kv_heads ? k_out_stride : 0;
  p.positions = positions;
  p.phases = phases;
  p.amplitude = amplitude;
  p.sign = inverse ? -1.f : 1.f;
  p.copy = (num_q_heads && q_out != q) || (num_kv_heads && k_out != k);
  const bool aligned = ((reinterpret_cast<uintptr_t>(num_q_heads ? q : nullptr) |
                         reinterpret_cast<uintptr_t>(num_kv_heads ? k : nullptr) |
                         reinterpret_cast<uintptr_t>(num_q_heads ? q_out : nullptr) |
                         reinterpret_cast<uintptr_t>(num_kv_heads ? k_out : nullptr)) & 15) == 0;
  const bool vec = p.half % (interleaved ? 4 : 8) == 0 && head_dim % 8 == 0 &&
      ((p.q_stride | p.k_stride | p.q_out_stride | p.k_out_stride) & 7) == 0 && aligned;
  const bool runs = !vec && head_dim % 8 == 0 && head_dim <= 8 * kRopeThreads &&
      ((p.q_stride | p.k_stride | p.q_out_stride | p.k_out_stride) & 7) == 0 && aligned;
  // About four items a thread: fewer leave the angles' cost bare, more make the last,
  // partly filled wave of CTAs long (72 heads x 16 items, 5003 tokens: 4 tokens a CTA
  // 55.9 us, one token a CTA 31.5 us).
  const int64_t items = heads * (runs  ? head_dim / 8
                                 : vec ? p.half / (interleaved ? 4 : 8) + (p.copy ? (head_dim - rotary_dim) / 8 : 0)
                                       : p.half + (p.copy ? head_dim - rotary_dim : 0));
  p.tokens = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kRopeTokens, 4 * kRopeThreads / items)));
  const int64_t ctas = (n + p.tokens - 1) / p.tokens;
  if (ctas > 0x7fffffff) return OSCAR_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(p.tokens) * p.half * sizeof(float2);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(ctas)), dim3(kRopeThreads),
                                            smem, static_cast<cudaStream_t>(stream), &attr);
  const auto kernel = runs  ? (interleaved ? rope_runs_kernel<true> : rope_runs_kernel<false>)
                      : vec ? (interleaved ? rope_kernel<true, true> : rope_kernel<false, true>)
                            : (interleaved ? rope_kernel<true, false> : rope_kernel<false, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
}

}  // extern "C"
