// Attention over the 4-bit cache (kv4_layout.cuh): decode and several query rows per sequence,
// split over the context.
//
//   out[b][m][hq] = sum_t softmax_t(q . k_t / sqrt(d)) v_t,  t <= position of row m,
// with k_t = code s(channel) g_K(page, head), v_t = code s(token, 16 channels) g_V(page, head) for
// tokens in whole pages and bf16 keys and values for the tokens of the tail.
//
// The forms, the division of work and the arithmetic are those of the 8-bit cache
// (kv8_attention.cu), with code * s, exact in fp16, where that one has codes, and g for its scale: the
// only roundings are q (exact down to 2^-21 of a column's largest), p g_V (11 bits, unbiased) and
// the output.
#include "kv8_tiles.cuh"

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
  if (oscar_host::check_kv4(desc, &c) != OSCAR_OK) return 0;
  return workspace_of<kCodeE2m1>(&c, batch, m_rows, max_seq_len);
}

oscar_status oscar_kv4_attention(const oscar_kv4_desc* desc, const void* q, const int32_t* seq_lens,
                                 const int32_t* q_pos, int32_t batch, int32_t m_rows,
                                 int32_t max_seq_len, void* out, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  oscar_kv8_desc c;
  const oscar_status s = oscar_host::check_kv4(desc, &c);
  if (s != OSCAR_OK) return s;
  return attend<kCodeE2m1>(&c, q, seq_lens, q_pos, batch, m_rows, max_seq_len, out, workspace,
                           workspace_bytes, stream);
}

}  // extern "C"
