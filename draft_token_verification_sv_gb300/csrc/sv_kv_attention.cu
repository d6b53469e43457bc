// Attention of few query rows for each kv head over the 8-bit cache: decoding
// steps and short chains.
//
// O = sum_j 2^(s_j - m) v_j, one pass over the visible tokens with a running
// maximum m for each row.  Both products run on the tensor cores
// (m16n8k16): the 16 rows (or two times 16) are the query heads that share a
// kv head (times the new tokens), the codes are widened to fp16, which holds
// every e4m3 value, and queries and weights are fp16 (a power of two for each
// row keeps queries in range; fp32 queries and weights are the sum of two fp16,
// bf16 queries fit one, and their weights are rounded to 2^-11, an eighth of
// what the result's type keeps).  Scales of K and V are one factor for each
// page, on scores and weights.  Weights become fp16 times their page's V scale
// and a power of two of their row's own, which follows the row's largest such
// product: pages of large values without weight cost the others no bits.
// Sums and statistics are fp32.
//
// A warp streams its own steps of 16 tokens through its own ring of
// asynchronous copies, so that no barrier stands between a block's four warps;
// they are joined where an item ends.  A 16-row tile that reads the whole cache
// is bound by HBM (a step of 64 sequences of up to 8192 tokens, 8 kv heads of
// 128 dims: 113 us, 5.5 TB/s, 80% of a copy's rate); two tiles by the
// instructions that widen codes and weigh scores (chains of 8 on up to 32768
// tokens: 155 us, 3.8 TB/s); short calls by latency (500 tokens of one
// sequence: 9.7 us with the join, of which about 8 pass before the first
// product when nothing is in the caches).
#include "sv_kv_schedule.cuh"

#include <type_traits>

namespace sv {

namespace {

// ------------------------------------------------------------ primitives ----

__device__ __forceinline__ uint32_t smem_address(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// 16 bytes to shared memory, zeros where !live.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0));
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(live ? 4 : 0));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N));
}

// c += a b, 16 x 16 times 16 x 8.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t floats_to_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// The rest of two floats behind their fp16 values.
__device__ __forceinline__ uint32_t rest_f16x2(float a, float b, uint32_t hi) {
  const float2 h = f16x2_to_float2(hi);
  return floats_to_f16x2(a - h.x, b - h.y);
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// 16 consecutive query values (zeros unless `live`).
template <typename E>
__device__ __forceinline__ void load_query16(const E* p, bool live, bool vec, float (&x)[16]) {
  constexpr int kV = sizeof(E) == 2 ? 8 : 4;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 16 / kV; ++i) {
    uint4 v;
    if (vec) {
      v = *reinterpret_cast<const uint4*>(p + i * kV);
    } else {
      E* e = reinterpret_cast<E*>(&v);
#pragma unroll 1
      for (int j = 0; j < kV; ++j) e[j] = __ldg(p + i * kV + j);
    }
    unpack<E>(v, x + i * kV);
  }
}

// ----------------------------------------------------------------- shape ----

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Empty tiles ahead of an item.  A step of 64 sequences of up to 8192 tokens, 16 chains of 8 on up to 32768 and a window in fp32 take
// 120, 163 and 34.4 us without, 114, 159 and 31.8 with 3, 113, 155 and 31.4 with 6, 114, 153 and 32.6 with 8, 118, 155 and 33.4 with 12.
constexpr int kOpen = 6;

constexpr float kMost = 8192.0f;  // sum of a thread's four weights of a row as they become fp16
// Scales are 2^-100 or larger.  Where the scale is part of the weights' exponent, pages 2^100 and more below what carries a row's
// weight (zeros may be: they have the smallest scale) count as 2^-100 of it, so that their weights still count in the row's sum.
constexpr float kMostLift = 106.0f, kLeastUnit = -100.0f, kLeastScale = 0x1p-110f;

// The largest power of two that is no larger, of a positive normal number.
__device__ __forceinline__ float power_of_two(float x) { return __uint_as_float(__float_as_uint(x) & 0x7f800000u); }

// log2 of a positive normal number, exact for powers of two (lg2.approx is not below 1): of the exponent and of the rest.
__device__ __forceinline__ float scale_log2(float x) {
  const uint32_t u = __float_as_uint(x);
  float rest;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(rest) : "f"(__uint_as_float((u & 0x7fffffu) | 0x3f800000u)));
  return __uint_as_float(u >> 23 | 0x4b000000u) - 8388735.0f + rest;  // 2^23 + exponent + 127
}

// DP: head_dim rounded up to 64, 128 or 256 (the rest is zeros).  MT: tiles of
// 16 rows.  What the rows take in registers (values' sums 16 DP, queries 8 DP,
// for fp32 16 DP, floats of a warp) sets how many blocks an SM holds.
template <typename E, int DP, int MT> struct Shape {
  static constexpr bool kSplit = sizeof(E) == 4;  // queries and weights as two fp16 each
  // Queries in registers, or read from shared memory for every step, where sums and queries together do not fit them: a step of 64
  // sequences at 256 dims takes 222 us reading and 231 holding them (fp32 283 and 467), chains of 8 at 64 dims 106.5 and 115.
  static constexpr bool kQueriesStay = DP == 64 ? MT == 1 || kSplit : DP == 128 && MT == 1;
  // A step's V scale and its rows' lift: in the exponent of the weights, or multiplied to them.  Chains of 8 (two tiles) take 157 and
  // 159.6 us, a step of 64 sequences (one tile, where what stands between two products counts for more) 115 and 112.7.
  static constexpr bool kFold = MT == 2;
  static constexpr int kRows = 16 * MT;
  static constexpr int kStages = DP == 64 ? 6 : DP == 128 ? 4 : kSplit ? 2 : 3;
  static constexpr int kBlocksPerSm = MT == 1 && !kSplit ? (DP == 64 ? 4 : DP == 128 ? 3 : 2) : DP == 64 && !(kSplit && MT == 2) ? 3 : 2;
  static constexpr int kStageBytes = 2 * kStep * DP;          // keys, values
  static constexpr int kRing = kStages * (kStageBytes + 16);  // and their two scales
  static constexpr int kMerge = kRows * DP * 4;               // a warp's values in the join of a block's warps
  static constexpr int kPerWarp = kRing > kMerge ? kRing : kMerge;
  static constexpr int kQueryBytes = kRows * DP * 2;          // queries as fp16 (for fp32 twice)
  static constexpr int kShared = kWarps * kPerWarp + (kSplit ? 2 : 1) * kQueryBytes;
  static constexpr int kBlocks = kSMs * kBlocksPerSm;
  static constexpr int kPart = kRows * (DP + 2);  // floats of a part in the workspace
};

// Where 16-byte chunk c of a token's row lies in a stage: the order makes
// both reads below free of bank conflicts (two lanes' share of a value row
// at DP = 64 excepted).  Keys: 8 lanes read 4 chunks of 2 rows.  Values: 8 or
// 16 lanes read 32 bytes of each of 4 rows that lie two apart.
template <int DP>
__device__ __forceinline__ int key_chunk(int t, int c) {
  if (DP == 64) return t * 4 + c;
  return t * (DP / 16) + (c ^ ((t & 1) << 2));
}
template <int DP>
__device__ __forceinline__ int value_chunk(int t, int c) {
  if (DP == 64) return ((t & ~1) | ((t ^ (t >> 1)) & 1)) * 4 + (c ^ (((t >> 2) & 1) << 1));
  return t * (DP / 16) + (c ^ (((t >> 1) & 3) << 1));
}

// ---------------------------------------------------------------- kernel ----

template <typename E, int DP, int MT>
__global__ void __launch_bounds__(kThreads, Shape<E, DP, MT>::kBlocksPerSm) kv_attention_kernel(AttentionParams a) {
  using S = Shape<E, DP, MT>;
  constexpr bool SPLIT = S::kSplit;
  constexpr int kRows = S::kRows;
  constexpr int NQ = DP / 64;          // 16-byte chunks of a row that a lane reads
  constexpr int NT = DP / 8;           // value tiles of 8 dims
  constexpr int NV = DP == 64 ? 8 : 16;  // value tiles that one of a lane's pieces of a token feeds
  constexpr int NC = kStep * DP / 16 / 32;  // chunks of keys (and of values) that a lane copies for a step
  extern __shared__ __align__(128) uint8_t shared[];
  __shared__ CursorScratch s_cursor;
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_factor[kRows];
  __shared__ int s_token[kRows], s_pos[kRows];
  const KvView& w = a.w;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane >> 2, col = lane & 3;  // of the fragments
  const int g = blockIdx.x, blocks = gridDim.x;
  uint8_t* ring = shared + warp * S::kPerWarp;
  const uint32_t ring_at = smem_address(ring);
  const int page_mask = (1 << w.page_shift) - 1;
  // what a lane copies of every step: chunk c0 of tokens tk0, tk0 + 512 / DP ..
  const int tk0 = lane / (DP / 16), c0 = lane % (DP / 16);
  const int64_t lane_at = tk0 * w.token_stride + c0 * 16, lane_step = (512 / DP) * w.token_stride;

  wait_for_stream();
  flag_sequences(a, g, blocks, kThreads);
  Cursor c = find_cursor<kThreads, kRows, kWarps, kOpen>(a, g, blocks, s_cursor);
  if (threadIdx.x == 0 && a.joins) a.joins[g].rows = 0;

  while (c.at < c.end) {
    const KvSpan s = c.span;
    const int32_t* parents = a.parents ? a.parents + s.row0 : nullptr;
    const int r0 = c.rt * kRows, rows = min(kRows, s.n * a.group - r0);
    const int i0 = r0 / a.group, i1 = (r0 + rows - 1) / a.group;
    const ItemSteps steps = item_steps(a, s, i0, i1);
    const int tiles = max(1, (steps.steps + kWarps - 1) / kWarps);
    const int done = static_cast<int>(min(static_cast<long long>(tiles - c.tile), c.end - c.at));
    if (c.tile + done <= 0) break;  // the range ends in the item's empty tiles
    const int tile0 = max(c.tile, 0);
    const int step0 = tile0 * kWarps + warp;                       // this warp's steps:
    const int step1 = min(steps.steps, (c.tile + done) * kWarps);   // step0, step0 + kWarps ..
    const int64_t head_at = c.h * w.head_stride + lane_at;

    // The stages in flight.  Bit of a stage in `bad`: its page is not there.  Page ids are looked up ahead of their use.
    unsigned bad = 0;
    int fill = 0;  // the next stage to fill
    const auto look_up = [&](int step) {
      if (step >= step1) return -1;
      const int column = steps.token(step) >> w.page_shift;
      return sv_in(column, w.max_pages) ? __ldg(w.c.page_table + c.b * w.table_stride + column) : -1;
    };
    const auto fetch = [&](int step, int page) {
      if (step < step1) {
        const int t0 = steps.token(step);
        const bool there = page >= 0 && page < w.num_pages;
        if (__builtin_expect(!there, 0)) {
          kv_flag(w, c.b, SV_ROW_BAD_PAGE);
          page = 0;
        }
        bad = (bad & ~(1u << fill)) | (there ? 0u : 1u << fill);
        int64_t o = page * w.page_stride + (t0 & page_mask) * w.token_stride + head_at;
        const int count = !there || c0 * 16 >= w.dim || !kv_slot_in(w, t0 & page_mask, kStep) ? 0 : steps.end - t0;
        const uint32_t to = ring_at + fill * S::kStageBytes;
#pragma unroll
        for (int i = 0; i < NC; ++i, o += lane_step) {
          const int t = tk0 + i * (512 / DP);
          copy16(to + key_chunk<DP>(t, c0) * 16, w.c.k + o, t < count);
          copy16(to + kStep * DP + value_chunk<DP>(t, c0) * 16, w.c.v + o, t < count);
        }
        if (lane < 2)
          copy4(ring_at + S::kStages * S::kStageBytes + fill * 16 + lane * 4,
                (lane ? w.c.v_scale : w.c.k_scale) + static_cast<int64_t>(page) * w.kv_heads + c.h, there);
      }
      copy_commit();
      fill = fill + 1 == S::kStages ? 0 : fill + 1;
    };
    int ahead;  // page id of the step to fetch next
    {
      int page[S::kStages - 1];
#pragma unroll
      for (int i = 0; i < S::kStages - 1; ++i) page[i] = look_up(step0 + i * kWarps);
      ahead = look_up(step0 + (S::kStages - 1) * kWarps);
#pragma unroll
      for (int i = 0; i < S::kStages - 1; ++i) fetch(step0 + i * kWarps, page[i]);
    }

    // Queries, by all threads into shared memory: a thread takes 16 dims of a row, the threads of a row lie together in a
    // warp.  Times a power of two that puts the row's largest at 2^14 .. 2^15: fp16 then keeps what is 2^-28 of it without
    // loss for bf16; a negative factor goes into the queries, so that larger products are larger scores.
    uint8_t* const queries = shared + kWarps * S::kPerWarp;
#pragma unroll 1
    for (int i = threadIdx.x; i < kRows * (DP / 16); i += kThreads) {
      const int r = i / (DP / 16), chunk = i % (DP / 16);
      const bool live = r < rows;
      const int at = r0 + min(r, rows - 1), token = at / a.group, head = c.h * a.group + at - token * a.group;
      const E* p = static_cast<const E*>(a.q) + (static_cast<int64_t>(s.row0) + token) * a.q_row_stride + head * a.q_head_stride + chunk * 16;
      float x[16];
      load_query16<E>(p, live && chunk * 16 < w.dim && kv_row_in(w, static_cast<int64_t>(s.row0) + token) && sv_in(head, a.heads), a.q_vec, x);
      float top = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) top = fmaxf(top, fabsf(x[j]));
#pragma unroll
      for (int n = 1; n < DP / 16; n <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, n));
      const int e = top > 0.0f && top < CUDART_INF_F ? min(120, 141 - static_cast<int>(__float_as_uint(top) >> 23)) : 0;
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (a.scale_log2 < 0.0f ? -1.0f : 1.0f);
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = x[2 * j] * up, v = x[2 * j + 1] * up;
        hi[j] = floats_to_f16x2(u, v);
        lo[j] = SPLIT ? rest_f16x2(u, v, hi[j]) : 0;
      }
      // in the order of the products' left side: of (16 rows, 64 dims, 16 of them, lane) four words
      uint32_t* to = reinterpret_cast<uint32_t*>(queries) + (((r >> 4) * NQ + (chunk >> 2)) * 4 * 32 + (r & 7) * 4 + (chunk & 3)) * 4 + ((r >> 3) & 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        to[(j >> 1) * 128 + 2 * (j & 1)] = hi[j];
        if constexpr (SPLIT) to[(j >> 1) * 128 + 2 * (j & 1) + S::kQueryBytes / 4] = lo[j];
      }
      if (chunk == 0) {
        s_factor[r] = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        int depth = token;
        if (parents) {
          depth = 0;
          for (int u = tree_parent(parents, token); u >= 0; u = tree_parent(parents, u)) ++depth;
        }
        s_token[r] = token;
        s_pos[r] = s.ctx + depth;
      }
      __syncwarp();
    }
    __syncthreads();
    // of each 16 rows row's and row + 8's, as the first product's left side
    const auto load_queries = [&](int mt, int i, int j, int part, uint32_t (&f)[4]) {
      const uint4 u = reinterpret_cast<const uint4*>(queries + part * S::kQueryBytes)[((mt * NQ + i) * 4 + j) * 32 + lane];
      f[0] = u.x;
      f[1] = u.y;
      f[2] = u.z;
      f[3] = u.w;
    };
    uint32_t q[S::kQueriesStay ? MT : 1][S::kQueriesStay ? NQ : 1][4][4], q_rest[SPLIT && S::kQueriesStay ? MT : 1][SPLIT && S::kQueriesStay ? NQ : 1][4][4];
    float factor[MT][2];  // scores in base 2 = factor * key scale * product, factor >= 0
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int k = 0; k < 2; ++k) factor[mt][k] = s_factor[16 * mt + row + 8 * k];
      if constexpr (S::kQueriesStay)
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            load_queries(mt, i, j, 0, q[mt][i][j]);
            if constexpr (SPLIT) load_queries(mt, i, j, 1, q_rest[mt][i][j]);
          }
    }
    // tokens before `all` are in every row's past; `far` is the furthest position of a row
    const int all = parents ? s.ctx : s.ctx + i0 + 1, far = s.ctx + i1;

    float o[MT][NT][4] = {};
    // m: a row's maximum so far (whole, base 2), l: its sum of weights.  Weights are multiplied by their page's V scale and by
    // the row's lift to become fp16: a power of two (its exponent, where folded) that put the largest such product at 2^6 and
    // more when it was taken.
    float m[MT][2], l[MT][2], lift[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[mt][k] = -CUDART_INF_F;
        l[mt][k] = 0.0f;
        lift[mt][k] = S::kFold ? 0.0f : 1.0f;
      }
    int stage = 0;
#pragma unroll 1
    for (int step = step0; step < step1; step += kWarps) {
      copy_wait<S::kStages - 2>();
      __syncwarp();
      const uint8_t* k_at = ring + stage * S::kStageBytes;
      const uint8_t* v_at = k_at + kStep * DP;
      const float* sc = reinterpret_cast<const float*>(ring + S::kStages * S::kStageBytes + stage * 16);
      const float k_scale = sc[0], v_scale = fmaxf(sc[1], kLeastScale), v_log2 = S::kFold ? scale_log2(v_scale) : 0.0f;
      // products of 16 tokens: x[n][0..1] row's, [2..3] row + 8's, tokens 8 n + 2 col + {0, 1}
      float x[MT][2][4] = {};
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if constexpr (!S::kQueriesStay) {
          uint32_t keys[2][4][2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint4 b = *reinterpret_cast<const uint4*>(k_at + 16 * key_chunk<DP>(8 * n + row, 4 * i + col));
            const uint32_t word[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              keys[n][j][0] = e4m3x2_to_f16x2(word[j] & 0xffffu);
              keys[n][j][1] = e4m3x2_to_f16x2(word[j] >> 16);
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t f[4];
              load_queries(mt, i, j, 0, f);
#pragma unroll
              for (int n = 0; n < 2; ++n) mma(x[mt][n], f[0], f[1], f[2], f[3], keys[n][j][0], keys[n][j][1]);
              if constexpr (SPLIT) {
                load_queries(mt, i, j, 1, f);
#pragma unroll
                for (int n = 0; n < 2; ++n) mma(x[mt][n], f[0], f[1], f[2], f[3], keys[n][j][0], keys[n][j][1]);
              }
            }
        } else {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint4 b = *reinterpret_cast<const uint4*>(k_at + 16 * key_chunk<DP>(8 * n + row, 4 * i + col));
            const uint32_t word[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t b0 = e4m3x2_to_f16x2(word[j] & 0xffffu), b1 = e4m3x2_to_f16x2(word[j] >> 16);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma(x[mt][n], q[mt][i][j][0], q[mt][i][j][1], q[mt][i][j][2], q[mt][i][j][3], b0, b1);
                if constexpr (SPLIT)
                  mma(x[mt][n], q_rest[mt][i][j][0], q_rest[mt][i][j][1], q_rest[mt][i][j][2], q_rest[mt][i][j][3], b0, b1);
              }
            }
          }
        }
      }
      const int t0 = steps.token(step);
      const bool lost = (bad >> stage) & 1u;
      const bool whole = !lost && t0 + kStep <= all && (a.window == 0 || far - t0 < a.window || t0 + kStep <= a.sinks);
      uint32_t p[MT][4], p_rest[SPLIT ? MT : 1][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        unsigned seen = 0xffu;  // bit 4 n + k: x[n][k]
        if (__builtin_expect(!whole, 0)) {
          seen = 0;
#pragma unroll 1
          for (int n = 0; n < 8; ++n) {  // (rolled: seldom run, and code is fetched anew by every launch)
            const int j = t0 + 8 * (n >> 2) + 2 * col + (n & 1), r = 16 * mt + row + 4 * (n & 2);
            if (!lost && j < steps.end && sees(a, parents, s.ctx, s_token[r], s_pos[r], j)) seen |= 1u << n;
          }
        }
        // Weights against the maximum so far; where they sum to 2^13 and more (infinity where there is no maximum yet) the rows'
        // maxima are raised, their lifts taken anew, and they are taken again.
        const float f[2] = {factor[mt][0] * k_scale, factor[mt][1] * k_scale};
        float e[2][4], sum[2], unit[2];
        const auto weigh = [&]() {
          float c[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            unit[k] = S::kFold ? fmaxf(v_log2 + lift[mt][k], kLeastUnit) : fminf(v_scale * lift[mt][k], 0x1p126f);
            c[k] = S::kFold ? unit[k] - m[mt][k] : -m[mt][k];
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) e[n][k] = ex2(fmaf(x[mt][n][k], f[k >> 1], c[k >> 1]));
          if (__builtin_expect(!whole, 0))
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int k = 0; k < 4; ++k) e[n][k] = seen >> (4 * n + k) & 1u ? e[n][k] : 0.0f;
#pragma unroll
          for (int k = 0; k < 2; ++k) sum[k] = (e[0][2 * k] + e[0][2 * k + 1]) + (e[1][2 * k] + e[1][2 * k + 1]);
        };
        weigh();
        if (__builtin_expect(__any_sync(0xffffffffu, (S::kFold ? sum[0] : sum[0] * unit[0]) > kMost || (S::kFold ? sum[1] : sum[1] * unit[1]) > kMost), 0)) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (seen >> (4 * n + 2 * k + i) & 1u) top = fmaxf(top, x[mt][n][2 * k + i] * f[k]);
            top = quad_max(top);
            const float up = fmaxf(m[mt][k], ceilf(top));
            const bool none = up == -CUDART_INF_F;  // the row sees nothing so far: no maximum, nothing to scale
            const float down = none ? 0.0f : m[mt][k] - up, l_fix = ex2(down);
            float to, o_fix;  // the lift that this step asks for, or what is left of the one so far
            if constexpr (S::kFold) {
              to = none ? lift[mt][k] : fminf(fminf(lift[mt][k] - down, 7.0f - ceilf(top - up + v_log2)), kMostLift);
              o_fix = ex2(down + (to - lift[mt][k]));
            } else {
              to = none ? lift[mt][k]
                        : power_of_two(fminf(fminf(__fdividef(lift[mt][k], l_fix), __fdividef(128.0f, ex2(top - up) * v_scale)), 0x1p106f));
              o_fix = l_fix > 0.0f ? l_fix * __fdividef(to, lift[mt][k]) : 0.0f;
            }
            m[mt][k] = up;
            lift[mt][k] = to;
            l[mt][k] *= l_fix;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              o[mt][t][2 * k] *= o_fix;
              o[mt][t][2 * k + 1] *= o_fix;
            }
          }
          weigh();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) l[mt][k] = S::kFold ? fmaf(sum[k], ex2(-unit[k]), l[mt][k]) : l[mt][k] + sum[k];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float u = S::kFold ? e[n][2 * k] : e[n][2 * k] * unit[k], v = S::kFold ? e[n][2 * k + 1] : e[n][2 * k + 1] * unit[k];
            p[mt][2 * n + k] = floats_to_f16x2(u, v);
            if constexpr (SPLIT) p_rest[mt][2 * n + k] = rest_f16x2(u, v, p[mt][2 * n + k]);
          }
      }
      // values: a lane reads NV / 16 of the row of its four tokens, whose bytes i are dims of tile i
#pragma unroll
      for (int h = 0; h < NT / NV; ++h) {
        uint32_t word[4][NV / 4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int token_at = 2 * col + (t & 1) + 8 * (t >> 1);
          if constexpr (DP == 64) {
            const uint2 b = *reinterpret_cast<const uint2*>(v_at + 16 * value_chunk<DP>(token_at, row >> 1) + 8 * (row & 1));
            word[t][0] = b.x;
            word[t][1] = b.y;
          } else {
            const uint4 b = *reinterpret_cast<const uint4*>(v_at + 16 * value_chunk<DP>(token_at, 8 * h + row));
            word[t][0] = b.x;
            word[t][1] = b.y;
            word[t][2] = b.z;
            word[t][3] = b.w;
          }
        }
#pragma unroll
        for (int i = 0; i < NV / 4; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t u = __byte_perm(word[0][i], word[1][i], half ? 0x7362 : 0x5140);
            const uint32_t v = __byte_perm(word[2][i], word[3][i], half ? 0x7362 : 0x5140);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t b0 = e4m3x2_to_f16x2(k ? u >> 16 : u & 0xffffu), b1 = e4m3x2_to_f16x2(k ? v >> 16 : v & 0xffffu);
              const int t = h * NV + 4 * i + 2 * half + k;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) {
                mma(o[mt][t], p[mt][0], p[mt][1], p[mt][2], p[mt][3], b0, b1);
                if constexpr (SPLIT) mma(o[mt][t], p_rest[mt][0], p_rest[mt][1], p_rest[mt][2], p_rest[mt][3], b0, b1);
              }
            }
          }
      }
      __syncwarp();
      fetch(step + (S::kStages - 1) * kWarps, ahead);
      ahead = look_up(step + S::kStages * kWarps);
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    copy_wait<0>();

    // The block's warps joined: maxima and sums, then values, in shared memory.
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[mt][k] = quad_sum(l[mt][k]);
        if (col == 0) {
          s_m[warp][16 * mt + row + 8 * k] = m[mt][k];
          s_l[warp][16 * mt + row + 8 * k] = l[mt][k];
        }
      }
    __syncthreads();  // and every warp has read its ring
    float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 16 * mt + row + 8 * k;
        float top = s_m[0][r];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) top = fmaxf(top, s_m[i][r]);
        const float fix = (m[mt][k] == -CUDART_INF_F ? (l[mt][k] == 0.0f ? 0.0f : 1.0f) : ex2(m[mt][k] - top)) * (S::kFold ? ex2(-lift[mt][k]) : 1.0f / lift[mt][k]);
        // a lane's dims of tiles h NV ..: 2 NV in a row, from h (8 NV) + 2 NV col
#pragma unroll
        for (int h = 0; h < NT / NV; ++h)
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < NV / 4; ++i) {
              const int d4 = h * (2 * NV) + col * (NV / 2) + half * (NV / 4) + i;  // in fours
              const int t = h * NV + 4 * i, e = 2 * k + half;
              *reinterpret_cast<float4*>(mine + r * DP + 4 * (d4 ^ ((row & 1) << 2 | col))) =
                  make_float4(o[mt][t][e] * fix, o[mt][t + 1][e] * fix, o[mt][t + 2][e] * fix, o[mt][t + 3][e] * fix);
            }
      }
    __syncthreads();
    const bool complete = tile0 == 0 && c.tile + done == tiles;
    float* part = complete ? nullptr : a.parts + (2 * static_cast<int64_t>(g) + (tile0 == 0 ? 1 : 0)) * S::kPart;
    for (int i = threadIdx.x; i < rows * (DP / 4); i += kThreads) {
      const int r = i / (DP / 4), d4 = i % (DP / 4);
      const int piece = d4 / (NV / 2) % 4;  // the lane column that wrote it
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float top = -CUDART_INF_F, total = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(shared + k * S::kPerWarp) + r * DP +
                                                          4 * (d4 ^ ((r & 1) << 2 | piece)));
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
        top = fmaxf(top, s_m[k][r]);
      }
#pragma unroll
      for (int k = 0; k < kWarps; ++k) total += s_m[k][r] == -CUDART_INF_F ? s_l[k][r] : s_l[k][r] * ex2(s_m[k][r] - top);
      if (!complete) {
        if (!sv_in(g, S::kBlocks)) break;  // the workspace's parts
        *reinterpret_cast<float4*>(part + r * DP + 4 * d4) = sum;
        if (d4 == 0) *reinterpret_cast<float2*>(part + kRows * DP + 2 * r) = make_float2(top, total);
      } else {
        store_result<E>(a, s.row0, r0 + r, c.h, 4 * d4, sum, top, total);
      }
    }
    if (!complete && tile0 == 0 && threadIdx.x == 0)
      a.joins[g] = JoinRecord{s.row0, r0, rows, c.h, tile_owner(c.at - c.tile + tiles - 1, c.total, c.blocks)};
    __syncthreads();  // the ring and the maxima are free again
    next_item<kRows, kOpen>(a, c, done);
  }
}

template <int N> using Int = std::integral_constant<int, N>;

int round_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <typename E, int DP, int MT>
sv_status launch(AttentionParams a, const sv_kv_attention_desc& d, void* workspace, cudaStream_t stream) {
  using S = Shape<E, DP, MT>;
  static FuncAttrCache attr;
  const auto kernel = kv_attention_kernel<E, DP, MT>;
  if (!attr.ensure(reinterpret_cast<const void*>(kernel), S::kShared, false)) return SV_ERR_CUDA;
  const int64_t row_tiles = (static_cast<int64_t>(d.max_new) * a.group + S::kRows - 1) / S::kRows;
  const int64_t tiles = (static_cast<int64_t>(d.kv.max_pages) * d.kv.page_size + kStep * kWarps - 1) / (kStep * kWarps);
  const int blocks = schedule_blocks(row_tiles * d.kv.batch * d.kv.kv_heads, tiles + kOpen, S::kBlocks);
  a.parts = static_cast<float*>(workspace);
  a.joins = reinterpret_cast<JoinRecord*>(a.parts + 2 * static_cast<int64_t>(S::kBlocks) * S::kPart);
  if (launch_early(kernel, dim3(blocks), dim3(kThreads), S::kShared, stream, a) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  if (blocks == 1 || tiles == 1) return SV_OK;  // no item has parts
  if (launch_join<E, DP, S::kRows>(a, blocks, stream) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

template <typename E, int DP, int MT>
size_t workspace_for() {
  using S = Shape<E, DP, MT>;
  return S::kBlocks * (2 * S::kPart * sizeof(float) + sizeof(JoinRecord));
}

// Calls f with the kernel's template arguments as types: one tile of 16 rows,
// or two where a kv head has more rows and the sums fit the registers.  Chains
// of 8 (32 rows) on contexts of up to 32768 tokens take 155 us with two tiles
// and 194 with one, which reads the cache twice, at 64 dims 101 and 129; 2000
// tokens of a prompt in fp32 1483 and 1953.
template <typename F>
auto with_shape(const sv_kv_attention_desc& d, F f) {
  const bool two = static_cast<int64_t>(d.max_new) * (d.heads / d.kv.kv_heads) > 16;
  const int dp = round_dim(d.kv.head_dim);
  if (d.dtype == SV_BF16) {
    if (dp == 64) return two ? f(uint16_t{}, Int<64>{}, Int<2>{}) : f(uint16_t{}, Int<64>{}, Int<1>{});
    if (dp == 128) return two ? f(uint16_t{}, Int<128>{}, Int<2>{}) : f(uint16_t{}, Int<128>{}, Int<1>{});
    return f(uint16_t{}, Int<256>{}, Int<1>{});
  }
  if (dp == 64) return two ? f(float{}, Int<64>{}, Int<2>{}) : f(float{}, Int<64>{}, Int<1>{});
  if (dp == 128) return two ? f(float{}, Int<128>{}, Int<2>{}) : f(float{}, Int<128>{}, Int<1>{});
  return f(float{}, Int<256>{}, Int<1>{});
}

}  // namespace

size_t kv_attention_workspace_bytes(const sv_kv_attention_desc& d) {
  if (kv_attention_takes_tiles(d)) return kv_attention_tiles_workspace(d);
  return align_up(with_shape(d, [](auto e, auto dp, auto mt) { return workspace_for<decltype(e), dp.value, mt.value>(); }), 256);
}

sv_status kv_attention(const sv_kv_attention_desc& d, const void* q, const KvCache& c, const int32_t* ctx_lens,
                       const int32_t* new_start, const int32_t* parents, void* out, float* lse, int32_t* row_status,
                       void* workspace, cudaStream_t stream) {
  start_phases(stream);
  if (row_status && cudaMemsetAsync(row_status, 0, static_cast<size_t>(d.kv.batch) * sizeof(int32_t), stream) != cudaSuccess)
    return SV_ERR_CUDA;
  if (d.max_new == 0 || d.total_new == 0)
    return kv_check_lengths(kv_view(d.kv, c, ctx_lens, new_start, d.max_new, d.total_new, row_status), stream);
  const int64_t e = d.dtype == SV_BF16 ? 2 : 4;
  const auto aligned = [&](const void* p, int64_t row, int64_t head, int to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && (row * e) % to == 0 && (head * e) % to == 0;
  };
  AttentionParams a{kv_view(d.kv, c, ctx_lens, new_start, d.max_new, d.total_new, row_status),
                    q, out, lse, parents,
                    d.q_row_stride, d.q_head_stride, d.out_row_stride, d.out_head_stride,
                    d.heads, d.heads / d.kv.kv_heads, d.window, d.sinks, d.scale * kLog2e,
                    aligned(q, d.q_row_stride, d.q_head_stride, 16), aligned(out, d.out_row_stride, d.out_head_stride, 16),
                    aligned(out, d.out_row_stride, d.out_head_stride, 32),
                    nullptr, nullptr};
  if (kv_attention_takes_tiles(d)) return kv_attention_tiles(a, d, workspace, stream);
  return with_shape(d, [&](auto e, auto dp, auto mt) { return launch<decltype(e), dp.value, mt.value>(a, d, workspace, stream); });
}

}  // namespace sv
