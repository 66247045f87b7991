// pa_prefill_fp4 (4-bit pools).
#include "pa_prefill_quant.cuh"

extern "C" int pa_prefill_fp4(const void* q, const void* k_cache, const void* v_cache,
                   const int32_t* block_tables, int32_t table_stride, const int32_t* seq_lens,
                              const int32_t* query_start, int32_t num_seqs, int64_t total_q,
                              int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t block_size, int64_t num_blocks, int32_t q_dtype, float scale,
                              float k_scale, float v_scale, int32_t window, void* out, void* workspace,
                              size_t workspace_bytes, int32_t* err_word, pa_stream stream) {
  return pa::prefill_quant<true>(q, k_cache, v_cache, block_tables, table_stride, seq_lens,
                                         query_start, num_seqs, total_q, num_q_heads, num_kv_heads, head_dim,
                                         block_size, num_blocks, q_dtype, scale, k_scale, v_scale, window,
                                         out, workspace, workspace_bytes, err_word, stream);
}
