// Causal attention of whole prompts over their own keys and values: dispatch.
#include "sv_prompt.cuh"

namespace sv {

sv_status prompt_attention(const sv_prompt_attention_desc& d, const void* q, const void* k, const void* v,
                           const int32_t* new_start, void* out, float* lse, int32_t* row_status, cudaStream_t stream) {
  start_phases(stream);
  if (row_status && cudaMemsetAsync(row_status, 0, static_cast<size_t>(d.batch) * sizeof(int32_t), stream) != cudaSuccess) return SV_ERR_CUDA;
  const PromptView a{q, k, v, out, lse, d.q_row_stride, d.q_head_stride, d.k_row_stride, d.k_head_stride, d.v_row_stride, d.v_head_stride,
               d.out_row_stride, d.out_head_stride, new_start, row_status, d.batch, d.max_new, d.total_new, d.heads, d.kv_heads,
               d.heads / d.kv_heads, d.head_dim, d.window, d.sinks, d.scale};
  return prompt_takes_tiles(a, d.dtype) ? prompt_tiles(a, stream) : prompt_split(a, d.dtype, stream);
}

}  // namespace sv
