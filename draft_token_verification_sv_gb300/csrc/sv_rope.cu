// Rotary positions of queries and keys, with one position or several (time,
// height, width) for a token: pair (a, b) becomes (a cos t - b sin t, a sin t +
// b cos t).
//
// Bound by HBM: every value is read and written once, and a thread's sines and
// cosines serve all the heads that it takes of a token.  52,000 tokens of 32 + 8
// heads of 128 bf16 dims take 165 us, 96% of the measured copy bandwidth; 12,700
// of 28 + 4 heads with three positions each 39 us, 80% (a launch's start and end
// and eight angles a thread for 32 heads are a larger part).  Few tokens take
// 4 us, a launch and the way to memory and back.
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
// of a far position loses nothing to its size.  A float is m 2^e, so this is
// m times the bits of 1 / (2 pi), moved by e: off by 2^-64 turns, 2^-33 after
// 2^31 positions.  (Doubles would do, but eight of them for each thread took
// longer than the rest of 12,700 tokens of 32 heads: 72 us, now 39.)
__device__ __forceinline__ unsigned long long turns(float inv_freq) {
  constexpr unsigned long long kHigh = 0x28be60db9391054aull, kLow = 0x7f09d5f47d4d3770ull;  // 2^128 / (2 pi)
  const uint32_t u = __float_as_uint(inv_freq), raised = u >> 23 & 0xffu;
  const uint32_t m = (u & 0x7fffffu) | (raised ? 0x800000u : 0u);
  const int down = 64 + 150 - static_cast<int>(raised ? raised : 1u);  // bits that the product moves down by
  const unsigned __int128 low = static_cast<unsigned __int128>(m) * kLow;
  const unsigned __int128 high = static_cast<unsigned __int128>(m) * kHigh + static_cast<unsigned long long>(low >> 64);
  unsigned long long t = 0;
  if (down >= 64)
    t = down < 192 ? static_cast<unsigned long long>(high >> (down - 64)) : 0ull;
  else if (down > 0)
    t = static_cast<unsigned long long>(high) << (64 - down) | static_cast<unsigned long long>(low) >> down;
  return u >> 31 ? 0ull - t : t;
}

// Is it one that turns() takes?
__device__ __forceinline__ bool is_frequency(float inv_freq) { return fabsf(inv_freq) < 0x1p60f; }

// Cosine and sine of an angle in units of 2^-64 turns: the nearest quarter
// turn, and Taylor's polynomials on the rest, which is at most pi / 4 (the
// first term left out is 2^-29 of a sine, 2^-32 of a cosine).  The rest is
// taken in two halves of 32 bits with signs, so that a small one keeps float's
// bits, and with it the sine of a small angle: 2^-21 of its value.
__device__ __forceinline__ float2 cos_sin(unsigned long long angle) {
  constexpr float kUnit = 1.46291807926715968105e-9f;  // 2 pi / 2^32
  const uint32_t quarter = static_cast<uint32_t>((angle + (1ull << 61)) >> 62);
  const unsigned long long rest = angle - (static_cast<unsigned long long>(quarter) << 62);
  const int32_t low = static_cast<int32_t>(static_cast<uint32_t>(rest)), high = static_cast<int32_t>(static_cast<uint32_t>(rest + 0x80000000ull >> 32));
  const float x = fmaf(static_cast<float>(high), kUnit, static_cast<float>(low) * (kUnit * 0x1p-32f));
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

__device__ __forceinline__ int64_t angle_position(const RopeView& w, int pair, int row) {
  return __ldg(w.positions + w.axis[pair] * w.position_stride + row);
}

// Rows on any boundary, and parts of a head that are no multiple of 16 dims: a block a token, a thread a pair (or one of the
// dims that stay).
constexpr int kPairThreads = 128;

template <typename E>
__global__ void __launch_bounds__(kPairThreads) rope_pairs_kernel(const __grid_constant__ RopeView w) {
  const int row = blockIdx.x;
  wait_for_stream();
  if (!sv_in(row, w.rows)) return;
  for (int u = threadIdx.x; u < w.dim - w.half; u += kPairThreads) {
    const bool pair = u < w.half;
    const int i = !pair ? u + w.half : w.adjacent ? 2 * u : u, j = w.adjacent ? 2 * u + 1 : u + w.half;
    float2 t = make_float2(1.0f, 0.0f);
    if (pair) {
      const float f = __ldg(w.inv_freq + u);
      t = is_frequency(f) ? cos_sin(static_cast<unsigned long long>(angle_position(w, u, row)) * turns(f)) : make_float2(CUDART_NAN_F, CUDART_NAN_F);
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

// ---- rows on 16-byte boundaries ----

// (not by the read-only path: a call may work in place)
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}

template <typename E> __device__ __forceinline__ uint4 pack(const float* x);
template <> __device__ __forceinline__ uint4 pack<float>(const float* x) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
template <> __device__ __forceinline__ uint4 pack<uint16_t>(const float* x) {
  return make_uint4(floats_to_bf16x2(x[0], x[1]), floats_to_bf16x2(x[2], x[3]), floats_to_bf16x2(x[4], x[5]), floats_to_bf16x2(x[6], x[7]));
}

constexpr int kThreads = 256, kWarps = kThreads / 32;

// A thread has eight pairs of a head, whose sines and cosines it uses for every head that it takes of a token: the units of 16
// values of a head lie side by side in a warp, and as many heads as fit.  `split` warps share a token.
template <typename E, bool ADJACENT>
__global__ void __launch_bounds__(kThreads) rope_units_kernel(const __grid_constant__ RopeView w, int split) {
  constexpr int kVec = Elem<E>::kPerVec, kVecs = 16 / kVec, kHeads = sizeof(E) == 2 ? 4 : 2;  // heads under way
  const int units = w.dim >> 4, per = 32 / units;
  const int lane = threadIdx.x & 31, unit = lane % units, sub = lane / units;
  const int warp = threadIdx.x >> 5, part = warp % split, first = warp / split;
  const bool turned = unit < w.half >> 3, busy = sub < per;
  wait_for_stream();
  unsigned long long by[8];
  uint32_t axes = 0, none = 0;  // two bits a pair: its axis; a bit: it has no frequency
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    by[i] = 0;
    if (turned) {
      const float f = __ldg(w.inv_freq + 8 * unit + i);
      by[i] = turns(f);
      none |= is_frequency(f) ? 0u : 1u << i;
      axes |= static_cast<uint32_t>(w.axis[8 * unit + i]) << (2 * i);
    }
  }
  // where the thread's vectors lie in a head
  int at[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v)
    at[v] = ADJACENT || !turned ? 16 * unit + v * kVec : 8 * unit + (v % (kVecs / 2)) * kVec + (v >= kVecs / 2 ? w.half : 0);
  const int all = w.heads[0] + w.heads[1], step = split * per;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kWarps / split) + first; row < w.rows; row += static_cast<int64_t>(gridDim.x) * (kWarps / split)) {
    if (!sv_in(row, w.rows)) break;
    float2 t[8];
    const int32_t* p = w.positions + row;
    if (w.axes == 1) {
      const long long position = __ldg(p);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = cos_sin(static_cast<unsigned long long>(position) * by[i]);
    } else {
      int position[SV_MAX_ROPE_AXES];
#pragma unroll
      for (int n = 0; n < SV_MAX_ROPE_AXES; ++n) position[n] = n < w.axes ? __ldg(p + n * w.position_stride) : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t n = axes >> (2 * i) & 3u;
        const long long mine = n & 2 ? (n & 1 ? position[3] : position[2]) : (n & 1 ? position[1] : position[0]);
        t[i] = cos_sin(static_cast<unsigned long long>(mine) * by[i]);
      }
    }
    if (none != 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (none >> i & 1u) t[i] = make_float2(CUDART_NAN_F, CUDART_NAN_F);
    }
    if (!busy) continue;
    for (int h0 = part * per + sub; h0 < all; h0 += kHeads * step) {
      uint4 raw[kHeads][kVecs];
#pragma unroll
      for (int n = 0; n < kHeads; ++n) {
        const int h = h0 + n * step;
        if (h >= all) break;
        const int s = h >= w.heads[0];
        const E* x = static_cast<const E*>(w.side[s].x) + row * w.side[s].x_row + (h - (s ? w.heads[0] : 0)) * w.side[s].x_head;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) raw[n][v] = load16(x + at[v]);
      }
#pragma unroll
      for (int n = 0; n < kHeads; ++n) {
        const int h = h0 + n * step;
        if (h >= all) break;
        const int s = h >= w.heads[0];
        E* y = static_cast<E*>(w.side[s].y) + row * w.side[s].y_row + (h - (s ? w.heads[0] : 0)) * w.side[s].y_head;
        if (turned) {
          float x[16];
#pragma unroll
          for (int v = 0; v < kVecs; ++v) unpack<E>(raw[n][v], x + v * kVec);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float& a = x[ADJACENT ? 2 * i : i];
            float& b = x[ADJACENT ? 2 * i + 1 : i + 8];
            const float u = a * t[i].x - b * t[i].y, z = a * t[i].y + b * t[i].x;
            a = u;
            b = z;
          }
#pragma unroll
          for (int v = 0; v < kVecs; ++v) raw[n][v] = pack<E>(x + v * kVec);
        }
#pragma unroll
        for (int v = 0; v < kVecs; ++v) *reinterpret_cast<uint4*>(y + at[v]) = raw[n][v];
      }
    }
  }
}

template <typename E>
bool whole_vectors(const RopeView& w) {
  if (w.half % 8) return false;
  uintptr_t all = 0;
  for (int s = 0; s < (w.heads[1] ? 2 : 1); ++s) {
    const RopeSide& r = w.side[s];
    all |= reinterpret_cast<uintptr_t>(r.x) | reinterpret_cast<uintptr_t>(r.y) | static_cast<uintptr_t>(r.x_row | r.x_head | r.y_row | r.y_head) * sizeof(E);
  }
  return all % 16 == 0;
}

template <typename E>
cudaError_t launch(const RopeView& w, cudaStream_t stream) {
  if (!whole_vectors<E>(w)) return launch_early(rope_pairs_kernel<E>, dim3(w.rows), dim3(kPairThreads), 0, stream, w);
  // A warp a token, as many blocks as run at a time: 52,000 tokens of 40 heads take 165 us (more blocks: 170 and up, two warps a
  // token: 172).  Few tokens are shared by more warps, as long as these have heads: 64 of 40 heads take 6.4 us with one, 4.4 with 8.
  constexpr int kBlocks = 2 * 152;
  const int per = 32 / (w.dim >> 4), all = w.heads[0] + w.heads[1];
  int split = 1;
  while (split < kWarps && static_cast<int64_t>(w.rows) * split < kBlocks * kWarps && split * per < all) split *= 2;
  const int64_t blocks = (static_cast<int64_t>(w.rows) * split + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(blocks < kBlocks ? blocks : kBlocks);
  return launch_early(w.adjacent ? rope_units_kernel<E, true> : rope_units_kernel<E, false>, dim3(grid), dim3(kThreads), 0, stream, w, split);
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
  if ((d.dtype == SV_BF16 ? launch<uint16_t>(w, stream) : launch<float>(w, stream)) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
