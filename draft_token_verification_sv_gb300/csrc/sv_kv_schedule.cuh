// How the attention kernels share out their work, and how parts of one item
// are joined.
//
// An item is one tile of query rows of one (sequence, kv head): row r of a
// sequence is query token r / group with head r % group of the kv head's
// group.  Its visible tokens are counted in steps of 16 (a step lies in one
// page), a few steps make a tile, and all items' tiles, in the order of
// (sequence, row tile, kv head), form one long list.  Block g of G takes
// tiles [g T / G, (g + 1) T / G): every block has the same work whatever the
// lengths are, which are read on the device.  A block that holds a whole
// item writes its result; parts of an item go to the workspace (a block has
// two at most: the end of an item that began before it, and the beginning of
// one that ends after it) and a second launch joins them, in order, so that
// the result does not depend on timing.
//
// Taking up an item and handing over its result cost a block as much as some
// tiles do.  So each item has that many empty tiles (OPEN, below 0) ahead of its
// own in the list, and blocks that take more items take fewer tiles.
#pragma once

#include "sv_kv.cuh"

namespace sv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kSMs = 152;
constexpr int kStep = 16;  // tokens

struct AttentionParams {
  KvView w;
  const void* q;
  void* out;
  float* lse;
  const int32_t* parents;
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  int heads, group, window, sinks;
  float scale_log2;  // scale * log2(e)
  bool q_vec, out_vec;  // rows on 16-byte boundaries
  bool out_vec32;       // and on 32-byte ones
  float* parts;         // [2 G][rows][DP + 2] fp32: values, then (maximum, sum) pairs of all rows
  struct JoinRecord* joins;  // [G]
};

// What the join needs of an item that block g began and did not end.
struct JoinRecord {
  int row0;   // first query row of the sequence in q / out
  int r0;     // first row of the item within the sequence
  int rows;   // 0: nothing to join
  int kv_head;
  int last;   // the last block with a part of it
};

// Parent of node i of a sequence whose rows start at `parents`, -1 for a root.
__device__ __forceinline__ int tree_parent(const int32_t* parents, int i) {
  const int p = __ldg(parents + i);
  return p >= 0 && p < i ? p : -1;
}

struct ItemSteps {
  int first;   // steps of the first tokens (sinks) ahead of the window's
  int start;   // the window's first step
  int steps;   // in all
  int end;     // tokens at or behind this are seen by no row
  // first token of step s
  __device__ __forceinline__ int token(int s) const { return kStep * (s < first ? s : start + s - first); }
};

// The steps that rows of query tokens i0..i1 have to look at.
__device__ __forceinline__ ItemSteps item_steps(const AttentionParams& a, const KvSpan& s, int i0, int i1) {
  ItemSteps x{0, 0, 0, 0};
  if (!s.ok) return x;
  x.end = s.ctx + i1 + 1;
  if (a.window > 0) {
    // a tree's node stands at most as far as its index: its window may begin with the root's
    const int lo = max(0, s.ctx + (a.parents ? 0 : i0) - a.window + 1);
    x.first = (min(a.sinks, x.end) + kStep - 1) / kStep;
    x.start = lo / kStep;
    if (x.start <= x.first) x.first = x.start = 0;
  }
  x.steps = x.first + (x.end + kStep - 1) / kStep - x.start;
  return x;
}

// Without the empty ones.
template <int ROWS, int TILE>
__device__ __forceinline__ int item_tiles(const AttentionParams& a, const KvSpan& s, int rt) {
  const int i0 = rt * ROWS / a.group;
  const int i1 = min(s.n - 1, ((rt + 1) * ROWS - 1) / a.group);
  return max(1, (item_steps(a, s, i0, i1).steps + TILE - 1) / TILE);
}

template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttentionParams& a, const KvSpan& s) {
  return s.n > 0 ? (s.n * a.group + ROWS - 1) / ROWS : 0;
}

template <int ROWS, int TILE, int OPEN>
__device__ __forceinline__ long long sequence_tiles(const AttentionParams& a, int b) {
  if (b >= a.w.batch) return 0;
  const KvSpan s = kv_span(a.w, b);
  const int rts = row_tiles<ROWS>(a, s);
  long long t = 0;
#pragma unroll 1
  for (int rt = 0; rt < rts; ++rt) t += OPEN + item_tiles<ROWS, TILE>(a, s, rt);
  return t * a.w.kv_heads;
}

// Where a block stands in the list.
struct Cursor {
  long long at, end;   // its tiles
  long long total;
  int blocks;          // that take part: each has a tile at least, if an empty one
  int b, rt, h;        // the item of tile `at`
  int tile;            // and the tile within it, below 0 for the empty ones
  KvSpan span;
};

struct CursorScratch {
  long long warp[32];
  long long before;
  int b;
};

// Sums every sequence's tiles and finds the block's first one.
template <int THREADS, int ROWS, int TILE, int OPEN>
__device__ __forceinline__ Cursor find_cursor(const AttentionParams& a, int g, int blocks, CursorScratch& scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Cursor c;
  const long long mine = sequence_tiles<ROWS, TILE, OPEN>(a, threadIdx.x);
  long long sum = mine;
#pragma unroll 1
  for (int b = threadIdx.x + THREADS; b < a.w.batch; b += THREADS) sum += sequence_tiles<ROWS, TILE, OPEN>(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) scratch.warp[warp] = sum;
  __syncthreads();
  c.total = 0;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) c.total += scratch.warp[i];
  c.blocks = static_cast<int>(min(static_cast<long long>(blocks), c.total));
  c.at = c.end = 0;
  if (g < c.blocks) {
    c.at = g * c.total / c.blocks;
    c.end = (g + 1) * c.total / c.blocks;
  }
  c.b = c.rt = c.h = c.tile = 0;
  if (c.at >= c.end) return c;
  long long base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.w.batch; b0 += THREADS) {
    const long long n = b0 == 0 ? mine : sequence_tiles<ROWS, TILE, OPEN>(a, b0 + threadIdx.x);
    long long x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) scratch.warp[warp] = x;
    __syncthreads();
    long long before = base, all = base;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += scratch.warp[i];
      all += scratch.warp[i];
    }
    x += before;  // inclusive
    if (c.at < x && c.at >= x - n) {
      scratch.b = b0 + threadIdx.x;
      scratch.before = x - n;
    }
    base = all;
    if (c.at < all) break;
  }
  __syncthreads();
  c.b = scratch.b;
  long long left = c.at - scratch.before;
  c.span = kv_span(a.w, c.b);
#pragma unroll 1
  for (c.rt = 0;; ++c.rt) {
    const int n = OPEN + item_tiles<ROWS, TILE>(a, c.span, c.rt);
    const long long all = static_cast<long long>(n) * a.w.kv_heads;
    if (left < all) {
      c.h = static_cast<int>(left / n);
      c.tile = static_cast<int>(left - static_cast<long long>(c.h) * n) - OPEN;
      break;
    }
    left -= all;
  }
  return c;
}

// The next item, `done` tiles on (which end an item).
template <int ROWS, int OPEN>
__device__ __forceinline__ void next_item(const AttentionParams& a, Cursor& c, int done) {
  c.at += done;
  c.tile = -OPEN;
  if (c.at >= c.end) return;
  if (++c.h < a.w.kv_heads) return;
  c.h = 0;
  if (++c.rt < row_tiles<ROWS>(a, c.span)) return;
  c.rt = 0;
#pragma unroll 1
  do {
    c.span = kv_span(a.w, ++c.b);
  } while (row_tiles<ROWS>(a, c.span) == 0);  // ends: at < total, so a sequence with tiles follows
}

// Tiles of the block's range that are not empty.
template <int ROWS, int TILE, int OPEN>
__device__ __forceinline__ long long full_tiles(const AttentionParams& a, Cursor c) {
  long long t = 0;
#pragma unroll 1
  while (c.at < c.end) {
    const int done = static_cast<int>(min(static_cast<long long>(item_tiles<ROWS, TILE>(a, c.span, c.rt) - c.tile), c.end - c.at));
    t += max(c.tile + done, 0) - max(c.tile, 0);
    next_item<ROWS, OPEN>(a, c, done);
  }
  return t;
}

// The block that takes tile t: the largest g with g T / G <= t.
__device__ __forceinline__ int tile_owner(long long t, long long total, int blocks) {
  return static_cast<int>(((t + 1) * blocks - 1) / total);
}

// Status bits of the sequences that this block looks after.
__device__ __forceinline__ void flag_sequences(const AttentionParams& a, int g, int blocks, int threads) {
  if (!a.w.status) return;
#pragma unroll 1
  for (int b = g; b < a.w.batch; b += blocks) {
    const KvSpan s = kv_span(a.w, b);
    if (!s.ok && threadIdx.x == 0) kv_flag(a.w, b, SV_ROW_BAD_LENGTH);
    if (!a.parents || !s.ok) continue;
    const int32_t* p = a.parents + s.row0;
#pragma unroll 1
    for (int i = threadIdx.x; i < s.n && kv_row_in(a.w, s.row0 + i); i += threads) {
      const int t = __ldg(p + i);
      if (i == 0 ? t != -1 : (t < 0 || t >= i)) kv_flag(a.w, b, SV_ROW_BAD_PARENT);
    }
  }
}

// Does a query at position pos (new token i) see token j?
__device__ __forceinline__ bool sees(const AttentionParams& a, const int32_t* parents, int ctx, int i, int pos, int j) {
  int at = j;
  if (j >= ctx) {
    const int t = j - ctx;
    if (!parents) {
      if (t > i) return false;
    } else {
      int u = i, back = 0;
#pragma unroll 1
      while (u > t) u = tree_parent(parents, u), ++back;
      if (u != t) return false;
      at = pos - back;
    }
  }
  return a.window == 0 || pos - at < a.window || at < a.sinks;
}

template <typename E>
__device__ __forceinline__ void store4(E* out, float4 v, bool vec) {
  if constexpr (sizeof(E) == 2) {
    const uint32_t lo = floats_to_bf16x2(v.x, v.y), hi = floats_to_bf16x2(v.z, v.w);
    if (vec) {
      *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
    } else {
      uint16_t* p = reinterpret_cast<uint16_t*>(out);
      p[0] = static_cast<uint16_t>(lo);
      p[1] = static_cast<uint16_t>(lo >> 16);
      p[2] = static_cast<uint16_t>(hi);
      p[3] = static_cast<uint16_t>(hi >> 16);
    }
  } else {
    float* p = reinterpret_cast<float*>(out);
    if (vec) {
      *reinterpret_cast<float4*>(p) = v;
    } else {
      p[0] = v.x;
      p[1] = v.y;
      p[2] = v.z;
      p[3] = v.w;
    }
  }
}

// log-sum-exp of a row from its maximum (base 2) and sum of weights
__device__ __forceinline__ float row_lse(float top, float total) {
  return total == 0.0f ? -CUDART_INF_F : (top + log2f(total)) * kLn2;
}

// Four values of a row's result from its weighted sum, maximum (base 2) and
// sum of weights, and with the first of them the log-sum-exp.
template <typename E>
__device__ __forceinline__ void store_result(const AttentionParams& a, int row0, int r, int kv_head, int d, float4 sum, float top,
                                             float total) {
  if (d >= a.w.dim) return;
  const int64_t row = static_cast<int64_t>(row0) + r / a.group;
  const int head = kv_head * a.group + r % a.group;
  if (!kv_row_in(a.w, row) || !sv_in(head, a.heads)) return;
  E* out = static_cast<E*>(a.out) + row * a.out_row_stride + head * a.out_head_stride + d;
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  store4<E>(out, make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv), a.out_vec);
  if (d == 0 && a.lse) a.lse[row * a.heads + head] = row_lse(top, total);
}

// Blocks (g, ..) for each part that began an item: its rows from all parts, in order, four values a thread.  2 to 4 us of latency.
template <typename E, int DP, int ROWS>
__global__ void __launch_bounds__(128) kv_attention_join_kernel(AttentionParams a) {
  wait_for_stream();  // the parts are written
  const int g = blockIdx.x;
  const JoinRecord j = a.joins[g];
  if (j.rows > 0 && (!sv_in(j.last, gridDim.x) || !sv_in(j.rows - 1, ROWS))) return;
  constexpr int kPart = ROWS * (DP + 2);
#pragma unroll 1
  for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < j.rows * (DP / 4); i += blockDim.x * gridDim.y) {
    const int r = i / (DP / 4), d4 = i % (DP / 4);
    const auto part = [&](int k) { return a.parts + (2 * static_cast<int64_t>(k) + (k == g ? 1 : 0)) * kPart; };
    float top = -CUDART_INF_F;
    for (int k = g; k <= j.last; ++k) top = fmaxf(top, part(k)[ROWS * DP + 2 * r]);
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float total = 0.0f;
#pragma unroll 4
    for (int k = g; k <= j.last; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(part(k) + ROWS * DP + 2 * r);
      const float4 v = *reinterpret_cast<const float4*>(part(k) + r * DP + 4 * d4);
      // a part that saw nothing has sums of 0 (or NaN, which stays)
      const float fix = ml.x == -CUDART_INF_F ? 1.0f : ex2(ml.x - top);
      total += ml.y * fix;
      sum.x += v.x * fix;
      sum.y += v.y * fix;
      sum.z += v.z * fix;
      sum.w += v.w * fix;
    }
    store_result<E>(a, j.row0, j.r0 + r, j.kv_head, 4 * d4, sum, top, total);
  }
}

template <typename E, int DP, int ROWS>
cudaError_t launch_join(const AttentionParams& a, int blocks, cudaStream_t stream) {
  return launch_early(kv_attention_join_kernel<E, DP, ROWS>, dim3(blocks, ROWS * DP / 512), dim3(128), 0, stream, a);
}

// Blocks for a call that can have at most so many items of so many tiles.
inline int schedule_blocks(int64_t items, int64_t tiles, int most) {
  return items >= most || tiles >= most || items * tiles >= most ? most : static_cast<int>(items * tiles);
}

// Attention for many rows of a kv head (sv_kv_attention_tiles.cu).
bool kv_attention_takes_tiles(const sv_kv_attention_desc& d);
size_t kv_attention_tiles_workspace(const sv_kv_attention_desc& d);
sv_status kv_attention_tiles(AttentionParams a, const sv_kv_attention_desc& d, void* workspace, cudaStream_t stream);

}  // namespace sv
