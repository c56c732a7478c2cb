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
#include "kv8_tiles.cuh"

namespace oscar {

// (The kernel for d = 128 stands for all: every cluster kernel fills an SM.)
static ClusterSizes count_clusters() {
  using C = Kv8Cfg<128, kCluster>;
  const auto kernel = kv8_attention_kernel<128, kCodeInt8, kCluster>;
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
  if (oscar_host::check_kv8(desc) != OSCAR_OK) return 0;
  return workspace_of(desc, batch, m_rows, max_seq_len);
}

oscar_status oscar_kv8_attention(const oscar_kv8_desc* desc, const void* q, const int32_t* seq_lens,
                                 const int32_t* q_pos, int32_t batch, int32_t m_rows,
                                 int32_t max_seq_len, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const oscar_status s = oscar_host::check_kv8(desc);
  if (s != OSCAR_OK) return s;
  return desc->format == OSCAR_KV8_E4M3
             ? attend<kCodeE4m3>(desc, q, seq_lens, q_pos, batch, m_rows, max_seq_len, out, workspace,
                                 workspace_bytes, stream)
             : attend<kCodeInt8>(desc, q, seq_lens, q_pos, batch, m_rows, max_seq_len, out, workspace,
                                 workspace_bytes, stream);
}

}  // extern "C"
