// What the kernels of prompt attention share.
#pragma once

#include "sv_kv.cuh"

namespace sv {

struct PromptView {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  float* lse;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
  const int32_t* new_start;
  int32_t* status;  // [batch], cleared before the launch, or NULL
  int batch, max_new, total_new, heads, kv_heads, group, dim, window, sinks;
  float scale;
};

// Sequence b's rows; false: they are not rows of the call.
struct PromptSpan {
  int row0, n;
  bool ok;
};

__device__ __forceinline__ PromptSpan prompt_span(const PromptView& a, int b) {
  if (!a.new_start) return PromptSpan{b * a.max_new, a.max_new, true};
  const int row0 = __ldg(a.new_start + b);
  const int64_t n = static_cast<int64_t>(__ldg(a.new_start + b + 1)) - row0;
  const bool ok = row0 >= 0 && n >= 0 && n <= a.max_new && row0 + n <= a.total_new;
  return PromptSpan{row0, ok ? static_cast<int>(n) : 0, ok};
}

__device__ __forceinline__ void prompt_flag(const PromptView& a, int b, int bit) {
  if (a.status) atomicOr(a.status + b, bit);
}

// bf16 rows that tensor copies can read, on the tensor cores (sv_prompt_tiles.cu).
bool prompt_takes_tiles(const PromptView& a, sv_dtype dtype);
sv_status prompt_tiles(const PromptView& a, cudaStream_t stream);
// Any others, on the tensor cores, too (sv_prompt_split.cu).
sv_status prompt_split(const PromptView& a, sv_dtype dtype, cudaStream_t stream);

}  // namespace sv
