// Causal attention of whole prompts over their own keys and values.
#include "sv_prompt.cuh"

namespace sv {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float value_of(const float* p) { return __ldg(p); }
__device__ __forceinline__ float value_of(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(floats_to_bf16x2(v, 0.0f)); }

// A warp a query row and head; a lane has every 32nd dim.  One pass over the
// keys with the running maximum and sum of a softmax.
template <typename E>
__global__ void __launch_bounds__(32 * kWarps) prompt_rows_kernel(PromptView a) {
  const int b = blockIdx.z, head = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const PromptSpan s = prompt_span(a, b);
  if (!s.ok && blockIdx.x == 0 && head == 0 && threadIdx.x == 0) prompt_flag(a, b, SV_ROW_BAD_LENGTH);
  if (i >= s.n || !sv_in(s.row0 + i, a.total_new)) return;
  constexpr int N = SV_MAX_HEAD_DIM / 32;
  const int h = head / a.group, dim = a.dim;
  const E* q = static_cast<const E*>(a.q) + (s.row0 + i) * a.q_row + head * a.q_head;
  const E* k = static_cast<const E*>(a.k) + s.row0 * a.k_row + h * a.k_head;
  const E* v = static_cast<const E*>(a.v) + s.row0 * a.v_row + h * a.v_head;
  float mine[N], o[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    mine[n] = lane + 32 * n < dim ? value_of(q + lane + 32 * n) * a.scale : 0.0f;
    o[n] = 0.0f;
  }
  float m = -CUDART_INF_F, l = 0.0f;
  const int64_t from = a.window ? max(int64_t{0}, i - a.window + 1) : 0;
  for (int64_t j = 0; j <= i; ++j) {
    if (j < from && j >= a.sinks) j = from;
    float x = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (lane + 32 * n < dim) x = fmaf(mine[n], value_of(k + j * a.k_row + lane + 32 * n), x);
    x = warp_sum(x);
    const float top = fmaxf(m, x);
    const float fix = m == -CUDART_INF_F ? 0.0f : __expf(m - top), e = x == -CUDART_INF_F ? 0.0f : __expf(x - top);
    l = l * fix + e;
    m = top;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (lane + 32 * n < dim) o[n] = fmaf(e, value_of(v + j * a.v_row + lane + 32 * n), o[n] * fix);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  E* out = static_cast<E*>(a.out) + (s.row0 + i) * a.out_row + head * a.out_head;
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (lane + 32 * n < dim) put(out + lane + 32 * n, o[n] * inv);
  if (a.lse && lane == 0) a.lse[(s.row0 + i) * a.heads + head] = m + logf(l);
}

}  // namespace

size_t prompt_attention_workspace_bytes(const sv_prompt_attention_desc&) { return 256; }

sv_status prompt_attention(const sv_prompt_attention_desc& d, const void* q, const void* k, const void* v,
                           const int32_t* new_start, void* out, float* lse, int32_t* row_status, void*, cudaStream_t stream) {
  start_phases(stream);
  if (row_status && cudaMemsetAsync(row_status, 0, static_cast<size_t>(d.batch) * sizeof(int32_t), stream) != cudaSuccess) return SV_ERR_CUDA;
  const PromptView a{q, k, v, out, lse, d.q_row_stride, d.q_head_stride, d.k_row_stride, d.k_head_stride, d.v_row_stride, d.v_head_stride,
               d.out_row_stride, d.out_head_stride, new_start, row_status, d.batch, d.max_new, d.total_new, d.heads, d.kv_heads,
               d.heads / d.kv_heads, d.head_dim, d.window, d.sinks, d.scale};
  if (prompt_takes_tiles(a, d.dtype)) return prompt_tiles(a, stream);
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(d.max_new) + kWarps - 1) / kWarps + (d.max_new == 0)), d.heads, d.batch);
  if (d.dtype == SV_BF16)
    prompt_rows_kernel<uint16_t><<<grid, 32 * kWarps, 0, stream>>>(a);
  else
    prompt_rows_kernel<float><<<grid, 32 * kWarps, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
