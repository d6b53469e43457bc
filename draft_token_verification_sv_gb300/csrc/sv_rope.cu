// Rotary positions of queries and keys, with one position or several (time,
// height, width) for a token.  Bound by HBM: every value is read and written once.
#include "sv_kv.cuh"

namespace sv {

namespace {

struct RopeSide {
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;
};

struct RopeView {
  RopeSide side[2];  // queries, keys
  int heads[2];
  int rows, dim, half, axes, adjacent;  // half: pairs of a head
  int64_t position_stride;
  const int32_t* positions;
  const float* inv_freq;
  uint8_t axis[SV_MAX_HEAD_DIM / 2];
};

// Radians a position as turns in units of 2^-64, modulo whole turns: a
// position's multiple of it wraps around where the angle does, so the angle
// of a far position loses nothing to its size.  1 / (2 pi) is the sum of two
// doubles and the products are exact to 2^-64 turns, 2^-33 after 2^31 positions.
__device__ __forceinline__ unsigned long long turns(float inv_freq) {
  const double f = inv_freq, high = f * 0.15915494309189535;
  const double low = fma(f, -9.839338337591243e-18, fma(f, 0.15915494309189535, -high));
  return static_cast<unsigned long long>(__double2ll_rn((high - rint(high)) * 0x1p64)) + static_cast<unsigned long long>(__double2ll_rn(low * 0x1p64));
}

// Cosine and sine of an angle in units of 2^-64 turns: the nearest quarter
// turn, and Taylor's polynomials on the rest, which is at most pi / 4 (the
// first term left out is 2^-29 of a sine, 2^-32 of a cosine).
__device__ __forceinline__ float2 cos_sin(unsigned long long angle) {
  const uint32_t a = static_cast<uint32_t>(angle >> 32);
  const uint32_t quarter = (a + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int32_t>(a - (quarter << 30))) * 1.46291807926715968105e-9f;  // 2 pi / 2^32
  const float z = x * x;
  const float s = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 2.755731922e-6f, -1.984126984e-4f), 8.333333333e-3f), -1.666666667e-1f), x);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.755731922e-7f, 2.480158730e-5f), -1.388888889e-3f), 4.166666667e-2f), -0.5f), 1.0f);
  const float u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
  return make_float2(quarter + 1 & 2 ? -u : u, quarter & 2 ? -v : v);
}

__device__ __forceinline__ float value_of(const float* p) { return *p; }
__device__ __forceinline__ float value_of(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(floats_to_bf16x2(v, 0.0f)); }

// A block a token, a thread a pair (or one of the dims that stay).
constexpr int kThreads = 128;

template <typename E>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeView w) {
  const int row = blockIdx.x;
  if (!sv_in(row, w.rows)) return;
  for (int u = threadIdx.x; u < w.dim - w.half; u += kThreads) {
    const bool pair = u < w.half;
    const int i = !pair ? u + w.half : w.adjacent ? 2 * u : u, j = w.adjacent ? 2 * u + 1 : u + w.half;
    float2 t = make_float2(1.0f, 0.0f);
    if (pair) {
      const long long position = __ldg(w.positions + w.axis[u] * w.position_stride + row);
      t = cos_sin(static_cast<unsigned long long>(position) * turns(__ldg(w.inv_freq + u)));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const E* x = static_cast<const E*>(w.side[s].x) + row * w.side[s].x_row;
      E* y = static_cast<E*>(w.side[s].y) + row * w.side[s].y_row;
      for (int h = 0; h < w.heads[s]; ++h, x += w.side[s].x_head, y += w.side[s].y_head) {
        if (!pair) {
          y[i] = x[i];
          continue;
        }
        const float a = value_of(x + i), b = value_of(x + j);
        put(y + i, a * t.x - b * t.y);
        put(y + j, a * t.y + b * t.x);
      }
    }
  }
}

}  // namespace

sv_status rope(const sv_rope_desc& d, const void* q, const void* k, const int32_t* positions, const float* inv_freq,
               void* q_out, void* k_out, cudaStream_t stream) {
  start_phases(stream);
  RopeView w{};
  w.side[0] = RopeSide{q, q_out, d.q_row_stride, d.q_head_stride, d.q_out_row_stride, d.q_out_head_stride};
  w.side[1] = RopeSide{k, k_out, d.k_row_stride, d.k_head_stride, d.k_out_row_stride, d.k_out_head_stride};
  w.heads[0] = d.heads;
  w.heads[1] = d.kv_heads;
  w.rows = d.rows;
  w.dim = d.head_dim;
  w.half = d.rotary_dim / 2;
  w.axes = d.axes;
  w.adjacent = d.adjacent;
  w.position_stride = d.position_stride;
  w.positions = positions;
  w.inv_freq = inv_freq;
  for (int i = 0; i < w.half; ++i) w.axis[i] = d.axis[i];
  if (d.dtype == SV_BF16)
    rope_kernel<uint16_t><<<d.rows, kThreads, 0, stream>>>(w);
  else
    rope_kernel<float><<<d.rows, kThreads, 0, stream>>>(w);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
