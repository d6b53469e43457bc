// The target's 8-bit cache: append (quantise and write), read back, commit
// the accepted path.  All three are bound by HBM for long inputs and by the
// chain of dependent loads (lengths, page id, scale, data) for short ones.
#include "sv_kv.cuh"

namespace sv {

namespace {

// Block-wide unsigned maximum; `scratch` holds THREADS / 32 entries.
template <int THREADS>
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v, uint32_t* scratch) {
  v = __reduce_max_sync(0xffffffffu, v);
  if (THREADS == 32) return v;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  v = scratch[0];
#pragma unroll
  for (int i = 1; i < THREADS / 32; ++i) v = max(v, scratch[i]);
  return v;
}

// 4 codes times `ratio`, rounded to codes again (NaN codes become 0).
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
  const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(codes & 0xffffu));
  const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(codes >> 16));
  const auto z = [&](float x) { return x == x ? x * ratio : 0.0f; };
  return floats_to_e4m3x2(z(a.x), z(a.y)) | floats_to_e4m3x2(z(b.x), z(b.y)) << 16;
}

// The first `held` tokens of (page, head) follow a scale that grew by 1 / ratio.
template <int THREADS>
__device__ __forceinline__ void regrow(const KvView& w, uint8_t* cache, int page, int head, int held, float ratio) {
  const int words = w.dim / 4;
  for (int i = threadIdx.x; i < held * words; i += THREADS) {
    const int t = i / words;
    if (!kv_slot_in(w, t)) return;
    uint32_t* p = reinterpret_cast<uint32_t*>(cache + kv_offset(w, page, head, t)) + (i - t * words);
    *p = rescale4(*p, ratio);
  }
}

// ---------------------------------------------------------------- append ----

template <typename E> struct Packed;  // 16 bytes of input
template <> struct Packed<uint16_t> {
  static constexpr int kN = 8;
  // largest |x| of the vector as the bits of a float; NaN and infinity compare above every finite value
  __device__ __forceinline__ static uint32_t magnitude(const uint4& v, uint32_t m) {
    m = __vmaxu2(m, v.x & 0x7fff7fffu);
    m = __vmaxu2(m, v.y & 0x7fff7fffu);
    m = __vmaxu2(m, v.z & 0x7fff7fffu);
    return __vmaxu2(m, v.w & 0x7fff7fffu);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return max(m & 0xffff0000u, m << 16); }
};
template <> struct Packed<float> {
  static constexpr int kN = 4;
  __device__ __forceinline__ static uint32_t magnitude(const uint4& v, uint32_t m) {
    m = max(max(m, v.x & 0x7fffffffu), v.y & 0x7fffffffu);
    return max(max(m, v.z & 0x7fffffffu), v.w & 0x7fffffffu);
  }
  __device__ __forceinline__ static uint32_t bits(uint32_t m) { return m; }
};

// 16 bytes from rows that need not be 16-byte aligned.
template <typename E, bool VEC>
__device__ __forceinline__ uint4 load_row16(const E* p) {
  if (VEC) return ldg_stream(p);
  uint32_t r[4];
  if (sizeof(E) == 2) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __ldg(h + 2 * i) | static_cast<uint32_t>(__ldg(h + 2 * i + 1)) << 16;
  } else {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __ldg(u + i);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

template <typename E, bool FINITE>
__device__ __forceinline__ void quantise_store(const uint4& v, float inv, uint8_t* to) {
  float x[Packed<E>::kN];
  unpack<E>(v, x);
  uint32_t r[Packed<E>::kN / 4];
#pragma unroll
  for (int i = 0; i < Packed<E>::kN; ++i) {
    if (!FINITE) x[i] = x[i] == x[i] ? x[i] : 0.0f;
    x[i] *= inv;
  }
#pragma unroll
  for (int i = 0; i < Packed<E>::kN / 4; ++i)
    r[i] = floats_to_e4m3x2(x[4 * i], x[4 * i + 1]) | floats_to_e4m3x2(x[4 * i + 2], x[4 * i + 3]) << 16;
  if constexpr (Packed<E>::kN == 8)
    *reinterpret_cast<uint2*>(to) = make_uint2(r[0], r[1]);
  else
    *reinterpret_cast<uint32_t*>(to) = r[0];
}

struct AppendRows {
  const void* x[2];           // keys, values
  int64_t row_stride[2], head_stride[2];
};

// Bound by HBM where there is much: 24,000 prompt tokens of 8 heads of 128 dims
// take 58 us, 5.4 TB/s read and written, 80% of a copy's rate (the largest value
// of a page is known before its first code is written, so a block's loads and
// stores do not overlap); one token for each of 64 sequences 4.6 us of latency.
// One block per (touched page, head, K or V), heads first: blocks that run
// together read and write what lies together in the rows of new tokens (the
// other way round 24,000 prompt tokens took 82 us).  The new tokens of the page
// are read once: up to kHeld vectors a thread stay in registers between the
// maximum and the rounding, what is beyond them is read again (from L2).
constexpr int kHeld = 16;

template <typename E, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(KvView w, AppendRows rows) {
  constexpr int kN = Packed<E>::kN;
  __shared__ uint32_t scratch[THREADS / 32];
  const int b = blockIdx.z, span = blockIdx.x / (2 * w.kv_heads), part = blockIdx.x - span * (2 * w.kv_heads);
  const int head = part >> 1, which = part & 1;
  const KvSpan s = kv_span(w, b);
  if (!s.ok) {
    if (blockIdx.x == 0 && threadIdx.x == 0) kv_flag(w, b, SV_ROW_BAD_LENGTH);
    return;
  }
  const int col = (s.ctx >> w.page_shift) + span;
  if (s.n <= 0 || col >= w.max_pages) return;
  const int page0 = col << w.page_shift;  // < 2^31: col < max_pages
  const int lo = max(s.ctx, page0);
  const int tokens = min(s.ctx + s.n - lo, page0 + (1 << w.page_shift) - lo);
  if (tokens <= 0) return;
  // a thread takes the same vector of every per-th token
  const int vpr = w.dim / kN, per = THREADS / vpr;
  const int t0 = threadIdx.x / vpr, ch = threadIdx.x - t0 * vpr;
  const int mine = t0 < per ? tokens : 0;  // THREADS may be no multiple of vpr
  const int64_t rs = rows.row_stride[which];
  const E* x = static_cast<const E*>(rows.x[which]) + head * rows.head_stride[which] +
               static_cast<int64_t>(s.row0 + (lo - s.ctx) + t0) * rs + ch * kN;
  const int64_t step = per * rs;
  const int row = s.row0 + (lo - s.ctx) + t0;
  uint4 held_v[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    held_v[j] = t0 + j * per < mine && kv_row_in(w, row + j * per) ? load_row16<E, VEC>(x + j * step) : make_uint4(0, 0, 0, 0);
  const int page = kv_page(w, b, col);
  if (page < 0) return;  // the same for the whole block
  uint8_t* cache = which ? w.c.v : w.c.k;
  float* scale = (which ? w.c.v_scale : w.c.k_scale) + static_cast<int64_t>(page) * w.kv_heads + head;
  const int held = lo - page0;
  const float old = held > 0 ? *scale : 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) m = Packed<E>::magnitude(held_v[j], m);
  for (int t = t0 + kHeld * per, j = kHeld; t < mine && kv_row_in(w, row + j * per); t += per, ++j) m = Packed<E>::magnitude(load_row16<E, VEC>(x + j * step), m);
  uint32_t top = block_max_u32<THREADS>(Packed<E>::bits(m), scratch);
  const bool finite = top < 0x7f800000u;
  if (!finite) {
    top = 0;
    for (int t = t0, j = 0; t < mine && kv_row_in(w, row + j * per); t += per, ++j) {
      const uint4 v = load_row16<E, VEC>(x + j * step);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const uint32_t u = __float_as_uint(Elem<E>::at(v, k)) & 0x7fffffffu;
        if (u < 0x7f800000u) top = max(top, u);
      }
    }
    top = block_max_u32<THREADS>(top, scratch);
    if (threadIdx.x == 0) kv_flag(w, b, SV_ROW_NOT_FINITE);
  }
  const float grown = fmaxf(old, kv_scale_for(__uint_as_float(top)));
  const float inv = 1.0f / grown;
  if (held > 0 && grown > old) regrow<THREADS>(w, cache, page, head, held, old * inv);
  __syncthreads();  // every thread has read the old scale
  if (threadIdx.x == 0) *scale = grown;
  uint8_t* to = cache + kv_offset(w, page, head, held + t0) + ch * kN;
  const int64_t to_step = per * w.token_stride;
  if (finite) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
      if (t0 + j * per < mine && kv_slot_in(w, held + t0 + j * per)) quantise_store<E, true>(held_v[j], inv, to + j * to_step);
  }
  for (int j = finite ? kHeld : 0, t = t0 + j * per; t < mine && kv_row_in(w, row + j * per) && kv_slot_in(w, held + t); t += per, ++j)
    quantise_store<E, false>(load_row16<E, VEC>(x + j * step), inv, to + j * to_step);
}

// ------------------------------------------------------------------ read ----

struct ReadRows {
  void* x[2];
  int64_t row_stride[2], head_stride[2];
};

template <typename E, bool VEC>
__device__ __forceinline__ void store_codes16(const uint4& c, float s, E* to) {
  float x[16];
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2(w[i] & 0xffffu));
    const float2 b = f16x2_to_float2(e4m3x2_to_f16x2(w[i] >> 16));
    x[4 * i] = a.x * s;
    x[4 * i + 1] = a.y * s;
    x[4 * i + 2] = b.x * s;
    x[4 * i + 3] = b.y * s;
  }
  uint32_t r[4 * sizeof(E)];
#pragma unroll
  for (int i = 0; i < 4 * static_cast<int>(sizeof(E)); ++i)
    r[i] = sizeof(E) == 2 ? floats_to_bf16x2(x[2 * i & 15], x[(2 * i + 1) & 15]) : __float_as_uint(x[i & 15]);
  if (VEC) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(E)); ++i)
      reinterpret_cast<uint4*>(to)[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
  } else if (sizeof(E) == 2) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      reinterpret_cast<uint16_t*>(to)[i] = static_cast<uint16_t>((i & 1) ? r[i >> 1] >> 16 : r[i >> 1] & 0xffffu);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) reinterpret_cast<uint32_t*>(to)[i] = r[i];
  }
}

// Bound by HBM: 2 x 65537 tokens of 8 heads of 128 dims take 108 us, 6.0 TB/s
// read and written, 89% of a copy's rate; one short stretch 8 us of latency.
// One block per (tile of kTile tokens, head, sequence); a thread takes the
// same 16 codes of every rows_per_pass-th token, keys and values.
template <typename E, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(KvView w, ReadRows rows, int tile) {
  const int b = blockIdx.z, block = blockIdx.x / w.kv_heads, head = blockIdx.x - block * w.kv_heads;
  const KvSpan s = kv_span(w, b);
  if (!s.ok && blockIdx.x == 0 && threadIdx.x == 0) kv_flag(w, b, SV_ROW_BAD_LENGTH);
  const int cpr = w.dim >> 4;
  const int per = THREADS / cpr;  // tokens of a pass
  const int t0 = threadIdx.x / cpr, chunk = threadIdx.x - t0 * cpr;
  const int count = min(tile, s.n - tile * block);  // (counted from the tile's first: sums with t0 could pass 2^31)
  if (t0 >= per) return;
#pragma unroll 4
  for (int i = t0; i < count; i += per) {
    const int t = tile * block + i, pos = s.ctx + t;
    const int page = s.ok ? kv_page(w, b, pos >> w.page_shift) : -1;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    float ks = 0.0f, vs = 0.0f;
    if (page >= 0) {
      const int64_t o = kv_offset(w, page, head, pos & ((1 << w.page_shift) - 1)) + chunk * 16;
      k = ldg_stream(w.c.k + o);
      v = ldg_stream(w.c.v + o);
      ks = __ldg(w.c.k_scale + static_cast<int64_t>(page) * w.kv_heads + head);
      vs = __ldg(w.c.v_scale + static_cast<int64_t>(page) * w.kv_heads + head);
    }
    const int64_t row = s.row0 + t;
    if (!kv_row_in(w, row)) break;
    store_codes16<E, VEC>(k, ks, static_cast<E*>(rows.x[0]) + row * rows.row_stride[0] + head * rows.head_stride[0] + chunk * 16);
    store_codes16<E, VEC>(v, vs, static_cast<E*>(rows.x[1]) + row * rows.row_stride[1] + head * rows.head_stride[1] + chunk * 16);
  }
}

// ---------------------------------------------------------------- commit ----

constexpr int kMaxPath = SV_MAX_TREE_DEPTH + 1;

// Bound by its chain of dependent loads (length, path, page, codes, scale): 64
// trees of depth 5 take 6.2 us, 256 of depth 16 8.3.
// One block per (head and K or V, sequence): the path's codes go to shared
// memory, then each page they land in is written by append's rule.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) kv_commit_kernel(KvView w, int nodes, int path_len, const int32_t* path,
                                                            const int32_t* accept_len, int32_t* new_lens) {
  extern __shared__ uint4 codes4[];  // [path_len][dim / 16]
  __shared__ float s_scale[kMaxPath];
  __shared__ uint32_t s_top[kMaxPath];  // largest magnitude code
  const int b = blockIdx.y, head = blockIdx.x >> 1, which = blockIdx.x & 1;
  const bool first = blockIdx.x == 0 && threadIdx.x == 0;
  const int ctx = __ldg(w.ctx_lens + b);
  const int a = __ldg(accept_len + b);
  const int32_t* p = path + static_cast<int64_t>(b) * path_len;
  const bool length = ctx >= 0 && static_cast<int64_t>(ctx) + nodes <= (static_cast<int64_t>(w.max_pages) << w.page_shift);
  bool good = a >= 0 && a < path_len;
  const bool none = __ldg(p) == -1;
  if (good)
    for (int i = threadIdx.x; i <= a; i += THREADS) {
      const int n = __ldg(p + i);
      good = good && n < nodes && (i == 0 ? n == 0 : n > __ldg(p + i - 1));
    }
  good = __syncthreads_and(good);
  const bool keep = length && good && !none;
  if (first) {
    new_lens[b] = keep ? ctx + a + 1 : ctx;
    if (!length) kv_flag(w, b, SV_ROW_BAD_LENGTH);
    if (!none && !good) kv_flag(w, b, SV_ROW_BAD_PATH);
  }
  if (!keep) return;
  uint8_t* cache = which ? w.c.v : w.c.k;
  float* scales = which ? w.c.v_scale : w.c.k_scale;
  const int mask = (1 << w.page_shift) - 1;
  const int cpr = w.dim >> 4;
  for (int i = threadIdx.x; i <= a; i += THREADS) s_top[i] = 0;
  __syncthreads();
  for (int n = threadIdx.x; n < (a + 1) * cpr; n += THREADS) {  // a thread per 16 codes
    const int i = n / cpr, ch = n - i * cpr;
    if (!sv_in(i, path_len)) break;
    const int pos = ctx + __ldg(p + i);
    const int page = kv_page(w, b, pos >> w.page_shift);
    uint4 c = make_uint4(0, 0, 0, 0);
    if (page >= 0) c = *reinterpret_cast<const uint4*>(cache + kv_offset(w, page, head, pos & mask) + ch * 16);
    if (ch == 0) s_scale[i] = page >= 0 ? scales[static_cast<int64_t>(page) * w.kv_heads + head] : 0.0f;
    uint32_t m = 0;
    const uint32_t word[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = (word[k] >> (8 * j)) & 0x7fu;
        m = u == 0x7fu ? m : max(m, u);
      }
    codes4[n] = c;
    atomicMax(&s_top[i], m);
  }
  __syncthreads();
  const uint32_t* words = reinterpret_cast<const uint32_t*>(codes4);
  const int wpr = w.dim >> 2;
  for (int col = ctx >> w.page_shift; col <= (ctx + a) >> w.page_shift; ++col) {
    const int page0 = col << w.page_shift;
    const int lo = max(ctx, page0), hi = min(ctx + a, page0 + mask) + 1;
    const int page = kv_page(w, b, col);
    if (page < 0) continue;
    float* scale = scales + static_cast<int64_t>(page) * w.kv_heads + head;
    const int held = lo - page0;
    const float old = held > 0 ? *scale : 0.0f;
    float top = 0.0f;
    for (int i = lo - ctx; i < hi - ctx; ++i) top = fmaxf(top, f16x2_to_float2(e4m3x2_to_f16x2(s_top[i])).x * s_scale[i]);
    const float grown = fmaxf(old, kv_scale_for(top));
    const float inv = 1.0f / grown;
    if (held > 0 && grown > old) regrow<THREADS>(w, cache, page, head, held, old * inv);
    __syncthreads();  // every thread has read the old scale
    if (threadIdx.x == 0) *scale = grown;
    uint8_t* to = cache + kv_offset(w, page, head, held);
    for (int i = threadIdx.x; i < (hi - lo) * wpr; i += THREADS) {
      const int t = i / wpr, k = i - t * wpr;
      const int src = lo - ctx + t;
      if (!sv_in(src, path_len) || !kv_slot_in(w, held + t)) break;
      // (beyond float only where all of the path's codes here are zeros, which stay)
      reinterpret_cast<uint32_t*>(to + t * w.token_stride)[k] = rescale4(words[src * wpr + k], fminf(s_scale[src] * inv, 0x1p127f));
    }
  }
}

__global__ void kv_lengths_kernel(KvView w) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < w.batch && !kv_span(w, b).ok) kv_flag(w, b, SV_ROW_BAD_LENGTH);
}

template <typename E, int THREADS>
void launch_append(const KvView& w, const AppendRows& rows, bool vec, const dim3& grid, cudaStream_t stream) {
  if (vec)
    kv_append_kernel<E, THREADS, true><<<grid, THREADS, 0, stream>>>(w, rows);
  else
    kv_append_kernel<E, THREADS, false><<<grid, THREADS, 0, stream>>>(w, rows);
}

// What a block takes stays in registers, so the fewest threads that hold it,
// each with much in flight: 24,000 prompt tokens in pages of 128 take 58 us
// with 128 threads of 16 vectors, 72 us with 256 of 8 and 93 us with 512 of 4;
// in pages of 64, 64 us with the fewest threads and 77 us with twice as many.
// A token's vectors are spread over threads of their own, so no fewer than those.
template <typename E>
void launch_append(const KvView& w, const AppendRows& rows, bool vec, int tokens, dim3 grid, cudaStream_t stream) {
  const int vectors = w.dim / Packed<E>::kN, all = tokens * vectors;
  if (all <= 32 * kHeld && vectors <= 32)
    launch_append<E, 32>(w, rows, vec, grid, stream);
  else if (all <= 64 * kHeld)
    launch_append<E, 64>(w, rows, vec, grid, stream);
  else if (all <= 128 * kHeld)
    launch_append<E, 128>(w, rows, vec, grid, stream);
  else
    launch_append<E, 256>(w, rows, vec, grid, stream);
}

bool rows_aligned16(const void* k, const void* v, const sv_kv_rows_desc& r) {
  const int64_t e = r.dtype == SV_BF16 ? 2 : 4;
  const int64_t all = (r.k_row_stride | r.k_head_stride | r.v_row_stride | r.v_head_stride) * e;
  return ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) == 0 && all % 16 == 0;
}

// Clears the callers' status words; the kernels set bits in them.
bool clear_status(int32_t* status, int batch, cudaStream_t stream) {
  return !status || cudaMemsetAsync(status, 0, static_cast<size_t>(batch) * sizeof(int32_t), stream) == cudaSuccess;
}

}  // namespace

sv_status kv_check_lengths(const KvView& w, cudaStream_t stream) {
  if (!w.status) return SV_OK;
  kv_lengths_kernel<<<(w.batch + 127) / 128, 128, 0, stream>>>(w);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

sv_status kv_append(const sv_kv_desc& d, const sv_kv_rows_desc& r, const void* k, const void* v, const KvCache& c,
                    const int32_t* ctx_lens, const int32_t* new_start, int32_t* row_status, cudaStream_t stream) {
  start_phases(stream);
  if (!clear_status(row_status, d.batch, stream)) return SV_ERR_CUDA;
  const KvView w = kv_view(d, c, ctx_lens, new_start, r.max_new, r.total_new, row_status);
  if (r.max_new == 0 || r.total_new == 0) return kv_check_lengths(w, stream);
  const AppendRows rows{{k, v}, {r.k_row_stride, r.v_row_stride}, {r.k_head_stride, r.v_head_stride}};
  // pages that max_new tokens touch at most: the first may start at its last slot
  const int64_t spans = (static_cast<int64_t>(r.max_new) + 2 * d.page_size - 2) / d.page_size;
  if (spans * 2 * d.kv_heads > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(spans * 2 * d.kv_heads), 1, d.batch);
  const bool vec = rows_aligned16(k, v, r);
  const int tokens = r.max_new < d.page_size ? r.max_new : d.page_size;
  if (r.dtype == SV_BF16)
    launch_append<uint16_t>(w, rows, vec, tokens, grid, stream);
  else
    launch_append<float>(w, rows, vec, tokens, grid, stream);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

sv_status kv_read(const sv_kv_desc& d, const sv_kv_rows_desc& r, void* k, void* v, const KvCache& c,
                  const int32_t* first, const int32_t* new_start, int32_t* row_status, cudaStream_t stream) {
  start_phases(stream);
  if (!clear_status(row_status, d.batch, stream)) return SV_ERR_CUDA;
  const KvView w = kv_view(d, c, first, new_start, r.max_new, r.total_new, row_status);
  if (r.max_new == 0 || r.total_new == 0) return kv_check_lengths(w, stream);
  const ReadRows rows{{k, v}, {r.k_row_stride, r.v_row_stride}, {r.k_head_stride, r.v_head_stride}};
  constexpr int kThreads = 256;
  const int tile = 4 * (kThreads / (d.head_dim / 16));  // four passes
  const int64_t blocks = (static_cast<int64_t>(r.max_new) + tile - 1) / tile * d.kv_heads;
  if (blocks > INT32_MAX) return SV_ERR_UNSUPPORTED;
  const dim3 grid(static_cast<unsigned>(blocks), 1, d.batch);
  const bool vec = rows_aligned16(k, v, r);
  if (r.dtype == SV_BF16)
    vec ? kv_read_kernel<uint16_t, kThreads, true><<<grid, kThreads, 0, stream>>>(w, rows, tile)
        : kv_read_kernel<uint16_t, kThreads, false><<<grid, kThreads, 0, stream>>>(w, rows, tile);
  else
    vec ? kv_read_kernel<float, kThreads, true><<<grid, kThreads, 0, stream>>>(w, rows, tile)
        : kv_read_kernel<float, kThreads, false><<<grid, kThreads, 0, stream>>>(w, rows, tile);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

sv_status kv_commit(const sv_kv_desc& d, int nodes, int path_len, const KvCache& c, const int32_t* ctx_lens,
                    const int32_t* path, const int32_t* accept_len, int32_t* new_lens, int32_t* row_status,
                    cudaStream_t stream) {
  start_phases(stream);
  if (!clear_status(row_status, d.batch, stream)) return SV_ERR_CUDA;
  const KvView w = kv_view(d, c, ctx_lens, nullptr, nodes, d.batch * nodes, row_status);
  constexpr int kThreads = 64;
  // 65 tokens of 256 dims: 16,640 bytes, within the default limit
  const size_t smem = static_cast<size_t>(path_len) * d.head_dim;
  kv_commit_kernel<kThreads><<<dim3(2 * d.kv_heads, d.batch), kThreads, smem, stream>>>(w, nodes, path_len, path,
                                                                                       accept_len, new_lens);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
