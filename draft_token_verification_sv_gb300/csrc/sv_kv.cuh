// Device view of the 8-bit cache and of a call's new tokens, shared by the
// cache kernels (sv_kv.cu) and the attention kernels.
#pragma once

#include "sv_internal.h"

#include <type_traits>

namespace sv {

struct KvView {
  KvCache c;
  int64_t page_stride, head_stride, token_stride, table_stride;
  int num_pages, max_pages, page_shift;  // page_size = 1 << page_shift
  int batch, kv_heads, dim;
  const int32_t* ctx_lens;
  const int32_t* new_start;
  int max_new, total_new;
  int32_t* status;  // [batch], cleared before the launch, or NULL
};

inline KvView kv_view(const sv_kv_desc& d, const KvCache& c, const int32_t* ctx_lens, const int32_t* new_start,
                      int max_new, int total_new, int32_t* status) {
  int shift = 4;
  while ((1 << shift) < d.page_size) ++shift;
  return KvView{c, d.page_stride, d.head_stride, d.token_stride, d.table_stride, d.num_pages, d.max_pages, shift,
                d.batch, d.kv_heads, d.head_dim, ctx_lens, new_start, max_new, total_new, status};
}

// Sequence b's cached and new tokens.  n < 0: its rows are not known.
struct KvSpan {
  int ctx, n, row0;
  bool ok;  // false: the sequence is left out (n is then the rows to clear, or -1)
};

__device__ __forceinline__ KvSpan kv_span(const KvView& w, int b) {
  KvSpan s;
  s.ctx = __ldg(w.ctx_lens + b);
  bool rows = true;
  if (w.new_start) {
    s.row0 = __ldg(w.new_start + b);
    const int64_t n = static_cast<int64_t>(__ldg(w.new_start + b + 1)) - s.row0;
    rows = s.row0 >= 0 && n >= 0 && n <= w.max_new && s.row0 + n <= w.total_new;
    s.n = rows ? static_cast<int>(n) : -1;
  } else {
    s.row0 = b * w.max_new;
    s.n = w.max_new;
  }
  s.ok = rows && s.ctx >= 0 && static_cast<int64_t>(s.ctx) + s.n <= (static_cast<int64_t>(w.max_pages) << w.page_shift);
  return s;
}

__device__ __forceinline__ void kv_flag(const KvView& w, int b, int bit) {
  if (w.status) atomicOr(w.status + b, bit);
}

// Flags bad lengths, for calls without a new token.
sv_status kv_check_lengths(const KvView& w, cudaStream_t stream);

// For the debug build's checks: is this a row of new tokens, a slot of a page (the first of `span`)?
__device__ __forceinline__ bool kv_row_in(const KvView& w, long long row) { return sv_in(row, w.total_new); }
__device__ __forceinline__ bool kv_slot_in(const KvView& w, int slot, int span = 1) { return sv_in(slot, (1 << w.page_shift) - span + 1); }

// Page id of column `col` of sequence b, or -1 (flagged) outside the pool.
__device__ __forceinline__ int kv_page(const KvView& w, int b, int col) {
  if (!sv_in(col, w.max_pages)) return -1;
  const int p = __ldg(w.c.page_table + b * w.table_stride + col);
  if (p >= 0 && p < w.num_pages) return p;
  kv_flag(w, b, SV_ROW_BAD_PAGE);
  return -1;
}

__device__ __forceinline__ int64_t kv_offset(const KvView& w, int page, int head, int slot) {
  return page * w.page_stride + head * w.head_stride + slot * w.token_stride;
}

// Two e4m3 codes (low byte first) as two halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }" : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// Two floats rounded to e4m3 (nearest even, clamped to +-448); a in the low byte.
__device__ __forceinline__ uint32_t floats_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}

__device__ __forceinline__ uint32_t floats_to_bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// The smallest power of two s >= 2^-100 with a <= 448 s, a >= 0 finite:
// 448 = 1.75 * 2^8, so with a = m * 2^e it is 2^(e - 8) for m <= 1.75 and
// 2^(e - 7) above.
__device__ __forceinline__ float kv_scale_for(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // biased exponent of s
  return __uint_as_float(static_cast<uint32_t>(max(e, 27)) << 23);
}

// Launches a kernel whose blocks may take their places while the launch
// before it in the stream ends; wait_for_stream() comes before anything in
// it that reads or writes memory.
template <typename... Args>
cudaError_t launch_early(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                         const std::remove_cv_t<Args>&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace sv
