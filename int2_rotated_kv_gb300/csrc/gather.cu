// Tokens of the calibrated cache (layout.cuh) read back as bf16 rows.
//
// A token t of a sequence of L tokens that is a sink (t < sink) or recent (t >= L - window) is in
// BF16 and comes back as it is.  The others are codes of x R: with y = code * s + z (fp32),
//   x[j] = sum_c y[c] R[j][c],
// what attention takes it for ("Technical Summary: OSCAR ...", section 2.2B: the rotation is undone
// when the history is used).
#include "common.cuh"
#include "layout.cuh"

namespace oscar {

struct GatherParams {
  int hkv, max_pages, batch, pages_per_seq, max_rows, sink, window;
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

// The value of a coded token's channel j, kv: 0 key, 1 value.
template <int D, int P>
__device__ __forceinline__ float coded_value(const uint8_t* blk, int kv, int t, int j) {
  using F = Fmt<D, P>;
  const int m = j >> 5, i = (j >> 4) & 1, h = (j >> 3) & 1;
  const int at = kv ? value_byte<D>(t, j & 7, m) : key_byte<D>(t, (j >> 1) & 3, m, j & 1);
  const uint8_t* codes = blk + (kv ? F::kVc : F::kKc) + at;
  int code = 0;
#pragma unroll
  for (int q = 0; q < P; ++q) code = 4 * code + ((codes[q * F::kPlane] >> (4 * h + 2 * i)) & 3);
  __half s, z;
  if (kv) {
    const int g = vsz_index<D>(t, m);
    s = reinterpret_cast<const __half*>(blk + F::kVs)[g];
    z = reinterpret_cast<const __half*>(blk + F::kVz)[g];
  } else {
    const __half2 w = reinterpret_cast<const __half2*>(blk + F::kKsz)[t * F::kNG + m];
    s = __low2half(w);
    z = __high2half(w);
  }
  return fmaf(static_cast<float>(code), __half2float(s), __half2float(z));
}

// blockIdx.x: (sequence, page of its rows), blockIdx.y: (KV head, keys or values); a thread per channel.
template <int D, int P>
__global__ void __launch_bounds__(D) gather_kernel(const __grid_constant__ GatherParams p) {
  __shared__ float y[kPage][D];
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y >> 1, kv = blockIdx.y & 1, j = threadIdx.x;
  const int b = blockIdx.x / p.pages_per_seq, i = blockIdx.x - b * p.pages_per_seq;
  const int64_t r0 = p.row_starts[b], n = p.row_starts[b + 1] - r0;
  const int t0 = p.first[b], len = p.seq_lens[b];
  if (n == 0) return;
  if (n < 0 || n > p.max_rows || r0 < 0 || r0 + n > p.total_rows || t0 < 0 || t0 + n > len ||
      len > static_cast<int64_t>(p.max_pages) * kPage) {
    if (p.status && j == 0) atomicOr(p.status, OSCAR_DEVERR_SEQ_LEN);
    return;
  }
  const int pg = t0 / kPage + i, t1 = t0 + static_cast<int>(n);
  if (pg * kPage >= t1) return;
  const int lo = max(t0 - pg * kPage, 0), hi = min(t1 - pg * kPage, kPage);
  // tokens [lo, c0) and [c1, hi) of the page are in BF16
  const int c0 = min(max(p.sink - pg * kPage, lo), hi), c1 = max(min(max(len - p.window, 0) - pg * kPage, hi), c0);
  uint16_t* out = p.out[kv] + ((r0 + (static_cast<int64_t>(pg) * kPage - t0)) * p.hkv + h) * D + j;
  const int64_t stride = static_cast<int64_t>(p.hkv) * D;
  const size_t entry = static_cast<size_t>(b) * p.max_pages + pg;
  if (c0 > lo || c1 < hi) {
    const int id = p.plain_table[entry];
    if (id < 0 || id >= p.n_plain) {
      if (p.status && j == 0) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
    } else {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(
          p.plain + (static_cast<int64_t>(id) * p.hkv + h) * Fmt<D>::kBf16Block + kv * Fmt<D>::kBf16V);
      for (int t = lo; t < hi; ++t)
        if (t < c0 || t >= c1) out[t * stride] = src[kv ? bf16_value_elem(t, j) : bf16_key_elem(t, j)];
    }
  }
  if (c0 >= c1) return;
  const int id = p.coded_table[entry];
  if (id < 0 || id >= p.n_coded) {
    if (p.status && j == 0) atomicOr(p.status, OSCAR_DEVERR_PAGE_ID);
    return;
  }
  const uint8_t* blk = p.coded + (static_cast<int64_t>(id) * p.hkv + h) * Fmt<D, P>::kInt2Block;
  for (int t = c0; t < c1; ++t) y[t][j] = coded_value<D, P>(blk, kv, t, j);
  __syncthreads();
  const float4* r = reinterpret_cast<const float4*>(p.r[kv] + (static_cast<size_t>(h) * D + j) * D);
  float acc[kPage] = {};
  for (int c = 0; c < D / 4; ++c) {
    const float4 w = r[c];
#pragma unroll
    for (int t = 0; t < kPage; ++t)
      if (t >= c0 && t < c1) {
        const float4 x = *reinterpret_cast<const float4*>(&y[t][4 * c]);
        acc[t] = fmaf(x.x, w.x, fmaf(x.y, w.y, fmaf(x.z, w.z, fmaf(x.w, w.w, acc[t]))));
      }
  }
#pragma unroll
  for (int t = 0; t < kPage; ++t)
    if (t >= c0 && t < c1) out[t * stride] = static_cast<uint16_t>(pack_bf162(acc[t], 0.f));
}

template <int D, int P>
oscar_status launch_gather(const GatherParams& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * static_cast<unsigned>(p.pages_per_seq),
                     static_cast<unsigned>(2 * p.hkv));
  cfg.blockDim = dim3(D);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gather_kernel<D, P>, p) == cudaSuccess ? OSCAR_OK : OSCAR_ERR_CUDA;
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
  const int64_t pages = (static_cast<int64_t>(max_rows) + kPage - 2) / kPage + 1;
  if (pages * batch > 0x7fffffff || desc->num_kv_heads > 32767) return OSCAR_ERR_UNSUPPORTED;
  GatherParams p{};
  p.hkv = desc->num_kv_heads;
  p.max_pages = desc->max_pages_per_seq;
  p.batch = batch;
  p.pages_per_seq = static_cast<int>(pages);
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
