// Attention of the new tokens over the 8-bit cache.
#include "sv_kv.cuh"

namespace sv {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttentionParams {
  KvView w;
  const void* q;
  void* out;
  float* lse;
  const int32_t* parents;
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  int heads, group, window, sinks;
  float scale_log2;  // scale * log2(e)
};

// Parent of node i of a sequence whose rows start at `parents`, -1 for a root.
__device__ __forceinline__ int tree_parent(const int32_t* parents, int i) {
  const int p = __ldg(parents + i);
  return p >= 0 && p < i ? p : -1;
}

// One block per (query, head): a tile of THREADS tokens at a time, one score
// a thread, then the tile's values with one or two dims a thread.
template <typename E, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_attention_simple_kernel(AttentionParams a) {
  __shared__ float s_q[SV_MAX_HEAD_DIM];
  __shared__ float s_p[THREADS], scratch[32];
  __shared__ int s_page[THREADS];
  const KvView& w = a.w;
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const KvSpan s = kv_span(w, b);
  const bool first = i == 0 && h == 0 && threadIdx.x == 0;
  if (!s.ok && first) kv_flag(w, b, SV_ROW_BAD_LENGTH);
  if (i >= s.n) return;
  const int64_t row = s.row0 + i;
  const int32_t* parents = a.parents ? a.parents + s.row0 : nullptr;
  if (parents && s.ok && first)
    for (int t = 0; t < s.n; ++t)
      if (__ldg(parents + t) != (t == 0 ? -1 : tree_parent(parents, t)) || (t > 0 && tree_parent(parents, t) < 0))
        kv_flag(w, b, SV_ROW_BAD_PARENT);
  int depth = i;
  if (parents) {
    depth = 0;
    for (int t = tree_parent(parents, i); t >= 0; t = tree_parent(parents, t)) ++depth;
  }
  const int pos = s.ok ? s.ctx + depth : 0;
  const E* q = static_cast<const E*>(a.q) + row * a.q_row_stride + h * a.q_head_stride;
  for (int d = threadIdx.x; d < w.dim; d += THREADS) s_q[d] = Elem<E>::load(q + d);
  const int kvh = h / a.group;
  float m = -CUDART_INF_F, l = 0.0f, o[2] = {0.0f, 0.0f};
  const int end = s.ok ? s.ctx + i + 1 : 0;
  for (int t0 = 0; t0 < end; t0 += THREADS) {
    __syncthreads();
    const int j = t0 + threadIdx.x;
    bool seen = j < end;
    int at = j;
    if (seen && parents && j >= s.ctx) {
      int t = i, back = 0;
      while (t > j - s.ctx) t = tree_parent(parents, t), ++back;
      seen = t == j - s.ctx;
      at = pos - back;
    }
    seen = seen && (a.window == 0 || pos - at < a.window || at < a.sinks);
    const int page = seen ? kv_page(w, b, j >> w.page_shift) : -1;
    float x = -CUDART_INF_F;
    if (page >= 0) {
      const uint8_t* k = w.c.k + kv_offset(w, page, kvh, j & ((1 << w.page_shift) - 1));
      float dot = 0.0f;
      for (int d = 0; d < w.dim; d += 4) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(k + d);
        const float2 u = f16x2_to_float2(e4m3x2_to_f16x2(c & 0xffffu)), v = f16x2_to_float2(e4m3x2_to_f16x2(c >> 16));
        dot = fmaf(s_q[d], u.x, fmaf(s_q[d + 1], u.y, fmaf(s_q[d + 2], v.x, fmaf(s_q[d + 3], v.y, dot))));
      }
      x = dot * __ldg(w.c.k_scale + static_cast<int64_t>(page) * w.kv_heads + kvh) * a.scale_log2;
    }
    const float top = fmaxf(m, block_max<THREADS>(x, scratch));
    const float base = top == -CUDART_INF_F ? 0.0f : top;
    const float p = page >= 0 ? exp2f(x - base) : 0.0f;
    const float fix = exp2f(m - base);
    l = l * fix + block_sum<THREADS>(p, scratch);
    m = top;
    s_p[threadIdx.x] = page >= 0 ? p * __ldg(w.c.v_scale + static_cast<int64_t>(page) * w.kv_heads + kvh) : 0.0f;
    s_page[threadIdx.x] = page;
    __syncthreads();
    o[0] *= fix;
    o[1] *= fix;
    const int n = min(THREADS, end - t0);
    for (int t = 0; t < n; ++t) {
      if (s_page[t] < 0) continue;
      const uint8_t* v = w.c.v + kv_offset(w, s_page[t], kvh, (t0 + t) & ((1 << w.page_shift) - 1));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int d = threadIdx.x + k * THREADS;
        if (d < w.dim) o[k] = fmaf(s_p[t], f16x2_to_float2(e4m3x2_to_f16x2(v[d])).x, o[k]);
      }
    }
  }
  E* out = static_cast<E*>(a.out) + row * a.out_row_stride + h * a.out_head_stride;
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = threadIdx.x + k * THREADS;
    if (d >= w.dim) continue;
    if (sizeof(E) == 2)
      reinterpret_cast<uint16_t*>(out)[d] = static_cast<uint16_t>(floats_to_bf16x2(o[k] * inv, 0.0f));
    else
      reinterpret_cast<float*>(out)[d] = o[k] * inv;
  }
  if (a.lse && threadIdx.x == 0) a.lse[row * a.heads + h] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * kLn2;
}

}  // namespace

size_t kv_attention_workspace_bytes(const sv_kv_attention_desc&) { return 256; }

sv_status kv_attention(const sv_kv_attention_desc& d, const void* q, const KvCache& c, const int32_t* ctx_lens,
                       const int32_t* new_start, const int32_t* parents, void* out, float* lse, int32_t* row_status,
                       void* workspace, cudaStream_t stream) {
  (void)workspace;
  start_phases(stream);
  if (row_status && cudaMemsetAsync(row_status, 0, static_cast<size_t>(d.kv.batch) * 4, stream) != cudaSuccess)
    return SV_ERR_CUDA;
  if (d.max_new == 0 || d.total_new == 0) return SV_OK;
  const AttentionParams a{kv_view(d.kv, c, ctx_lens, new_start, d.max_new, d.total_new, row_status), q, out, lse, parents,
                          d.q_row_stride, d.q_head_stride, d.out_row_stride, d.out_head_stride, d.heads,
                          d.heads / d.kv.kv_heads, d.window, d.sinks, d.scale * kLog2e};
  const dim3 grid(d.max_new, d.heads, d.kv.batch);
  if (d.dtype == SV_BF16)
    kv_attention_simple_kernel<uint16_t, 128><<<grid, 128, 0, stream>>>(a);
  else
    kv_attention_simple_kernel<float, 128><<<grid, 128, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
