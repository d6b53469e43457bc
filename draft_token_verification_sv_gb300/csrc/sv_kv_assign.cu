// Pages for the sequences' lengths, and a slot and a position for every new
// token.
//
// With g_b pages given and t_b taken by sequence b, page i of a sequence is at
// depth (sum of g, or t, of the sequences before) + i of what moves, so sums up
// to each sequence say where every page lies, and no page waits for another:
// the i-th taken is the i-th given or what lies that deep on the stack.
//
// A decoding step is bound by latency, a chain of dependent loads and block
// barriers: 64 sequences of one token 4.3 us, of 32 tree nodes 5.6 us, a launch
// among them.  Prompts are bound by the searches for each token's sequence and
// the writing of slots and positions: 250 prompts of up to 8191 tokens on pages
// of 16 take 31 us with the pages given back (58 us when one block moved all
// pages and a second launch placed the tokens).
#include "sv_kv.cuh"

#include <algorithm>

namespace sv {

namespace {

constexpr int kThreads = 1024;

struct AssignView {
  KvView w;           // lengths, rows, page_table and status; the cache itself is not used
  int32_t* free_pages;
  int32_t* free_count;
  int32_t* table;     // w.c.page_table
  int32_t* held;
  const int32_t* parents;
  int64_t* slots;
  int32_t* positions;
};

// What a sequence holds and shall hold.
struct Need {
  int held, want;
  bool ok;
};

__device__ __forceinline__ Need need_of(const AssignView& a, int b) {
  const KvSpan s = kv_span(a.w, b);
  Need n;
  n.held = a.held[b];
  n.ok = s.ok && n.held >= 0 && n.held <= a.w.max_pages;
  n.want = n.ok ? static_cast<int>((static_cast<int64_t>(s.ctx) + s.n + (1 << a.w.page_shift) - 1) >> a.w.page_shift) : n.held;
  return n;
}

// Sum of the block's values up to and with this thread's; `scratch` holds 33 entries, the last gets the total.
__device__ __forceinline__ long long block_inclusive(long long v, long long* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  __syncthreads();
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += up;
    }
    scratch[lane] = w;
    if (lane == 31) scratch[32] = w;
  }
  __syncthreads();
  return v + (warp > 0 ? scratch[warp - 1] : 0);
}

// The first of the block's sequences whose inclusive sum is above i (which the last one's is).  Without branches, so that several
// searches run at a time.
__device__ __forceinline__ int owner(const long long* sums, long long i) {
  int k = 0;
#pragma unroll
  for (int step = kThreads / 2; step > 0; step >>= 1) k += sums[k + step - 1] <= i ? step : 0;
  return k;
}

// Depth of node i of a tree; what is wrong with its own parent is flagged.
__device__ __forceinline__ int depth_of(const AssignView& a, int b, const int32_t* parents, int i) {
  int depth = 0;
  for (int u = i; u >= 0;) {
    const int p = __ldg(parents + u);
    if (u == i && (u == 0 ? p != -1 : (p < 0 || p >= u))) kv_flag(a.w, b, SV_ROW_BAD_PARENT);
    u = p >= 0 && p < u ? p : -1;
    depth += u >= 0;
  }
  return depth;
}

// The slot of token j on a page (flagged, and -1, outside the pool).
__device__ __forceinline__ int64_t slot_on(const AssignView& a, int b, int page, int j) {
  if (page >= 0 && page < a.w.num_pages) return (static_cast<int64_t>(page) << a.w.page_shift) + (j & ((1 << a.w.page_shift) - 1));
  kv_flag(a.w, b, SV_ROW_BAD_PAGE);
  return -1;
}

// ---- up to 1024 sequences ----

// Every block scans what all sequences give, lack and bring, a thread a
// sequence, and then moves its share of the pages and places its share of the
// tokens, one to a thread: the i-th page taken is the i-th given, or what lies
// that deep on the stack, and a new token's page is known before it is in the
// table, so that no block waits for another.  Lengths, the stack's count and
// the flags change in one block alone, when all others are done: with kAll in
// the same launch, which then is of one block, else in one of its own.
enum { kAll, kMove, kUpdate };

template <int WHAT>
__global__ void __launch_bounds__(kThreads) kv_assign_few_kernel(AssignView a) {
  __shared__ long long scratch[33], gives[kThreads], lacks[kThreads], brings[kThreads];
  __shared__ int ctxs[kThreads], rows[kThreads], helds[kThreads], wants[kThreads];  // wants: -1 where the sequence is left out
  const int tid = threadIdx.x, batch = a.w.batch, size = a.w.num_pages, shift = a.w.page_shift;
  wait_for_stream();
  const int count = min(max(*a.free_count, 0), size);
  Need n{0, 0, false};
  KvSpan s{0, 0, 0, false};
  if (tid < batch) {
    s = kv_span(a.w, tid);
    n = need_of(a, tid);
  }
  const int gave = max(n.held - n.want, 0), lack = max(n.want - n.held, 0);
  const long long given_upto = block_inclusive(gave, scratch), given = scratch[32];
  const long long lacked = block_inclusive(lack, scratch);
  const long long there = min(count + given, static_cast<long long>(size));
  const bool refused = lack > 0 && lacked > there;
  const long long taken = min(block_inclusive(refused ? 0 : lack, scratch), there), all_taken = scratch[32];
  const int flag = tid >= batch || (n.ok && !refused) ? 0 : n.ok ? SV_ROW_NO_PAGE : SV_ROW_BAD_LENGTH;
  if (WHAT == kAll && tid < batch && a.w.status) a.w.status[tid] = flag;
  if (WHAT != kUpdate) {
    gives[tid] = given_upto;
    lacks[tid] = taken;
    const bool tokens = a.slots || a.positions;
    brings[tid] = block_inclusive(tokens && s.n > 0 ? s.n : 0, scratch);
    const long long brought = scratch[32];
    ctxs[tid] = s.ctx;
    rows[tid] = s.row0;
    helds[tid] = n.held;
    wants[tid] = !n.ok ? -1 : refused ? n.held : n.want;
    __syncthreads();
    const long long first = static_cast<long long>(blockIdx.x) * kThreads + tid, step = static_cast<long long>(gridDim.x) * kThreads;
    // the i-th page given
    const auto given_page = [&](long long i) {
      const int k = owner(gives, i), col = wants[k] + static_cast<int>(i - (k > 0 ? gives[k - 1] : 0));
      return sv_in(col, a.w.max_pages) ? a.table[k * a.w.table_stride + col] : -1;
    };
    // and the i-th page taken (there are no more given than the stack has room for, or the first ones given are lost)
    const auto taken_page = [&](long long i) {
      const long long at = there - 1 - i;
      return at >= count ? given_page(count + given - 1 - at) : sv_in(at, size) ? a.free_pages[at] : -1;
    };
#pragma unroll 4
    for (long long i = first; i < given; i += step) {
      const long long at = count + given - 1 - i;
      if (at < size && sv_in(at, size)) a.free_pages[at] = given_page(i);
    }
#pragma unroll 4
    for (long long i = first; i < all_taken; i += step) {
      const int k = owner(lacks, i), col = helds[k] + static_cast<int>(i - (k > 0 ? lacks[k - 1] : 0));
      if (sv_in(col, a.w.max_pages)) a.table[k * a.w.table_stride + col] = taken_page(i);
    }
#pragma unroll 4
    for (long long i = first; i < brought; i += step) {
      const int k = owner(brings, i), t = static_cast<int>(i - (k > 0 ? brings[k - 1] : 0));
      const int64_t row = rows[k] + static_cast<int64_t>(t);
      if (!kv_row_in(a.w, row)) continue;
      int64_t slot = -1;
      int position = 0;
      if (wants[k] >= 0) {
        const int j = ctxs[k] + t, col = j >> shift;
        position = a.parents ? ctxs[k] + depth_of(a, k, a.parents + rows[k], t) : j;
        // (a sequence that got no pages has fewer than its tokens need)
        const int tokens_of = static_cast<int>(brings[k] - (k > 0 ? brings[k - 1] : 0));
        if (a.slots && static_cast<int64_t>(wants[k]) << shift >= static_cast<int64_t>(ctxs[k]) + tokens_of && sv_in(col, a.w.max_pages))
          slot = slot_on(a, k, col < helds[k] ? a.table[k * a.w.table_stride + col] : taken_page((k > 0 ? lacks[k - 1] : 0) + col - helds[k]), j);
      }
      if (a.slots) a.slots[row] = slot;
      if (a.positions) a.positions[row] = position;
    }
  }
  if (WHAT != kMove) {
    if (tid < batch && n.ok && !refused) a.held[tid] = n.want;
    if (WHAT == kUpdate && flag) kv_flag(a.w, tid, flag);
    if (tid == 0) *a.free_count = static_cast<int>(there - all_taken);
  }
}

// ---- any number of sequences ----

// One block: pages move in the order that the sequences have, whatever the
// launch, so it scans what they give and lack, 1024 at a time, and moves the
// pages one to a thread.
__global__ void __launch_bounds__(kThreads) kv_assign_pages_kernel(AssignView a) {
  __shared__ long long scratch[33], sums[kThreads];
  __shared__ int first[kThreads];  // the first column that a sequence gives or takes
  const int batch = a.w.batch, tid = threadIdx.x;
  const int size = a.w.num_pages;
  const int count = min(max(*a.free_count, 0), size);

  long long given = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const Need n = base + tid < batch ? need_of(a, base + tid) : Need{0, 0, false};
    given += max(n.held - n.want, 0);
  }
  block_inclusive(given, scratch);
  given = scratch[32];
  const long long there = min(count + given, static_cast<long long>(size));
  if (given > 0) {
    long long before = 0;
    for (int base = 0; base < batch; base += kThreads) {
      const Need n = base + tid < batch ? need_of(a, base + tid) : Need{0, 0, false};
      sums[tid] = block_inclusive(max(n.held - n.want, 0), scratch);
      first[tid] = n.want;
      const long long here = scratch[32];
      __syncthreads();
      for (long long i = tid; i < here; i += kThreads) {
        const int k = owner(sums, i);
        const int col = first[k] + static_cast<int>(i - (k > 0 ? sums[k - 1] : 0));
        const long long at = count + given - 1 - (before + i);
        if (at < size && sv_in(at, size) && sv_in(col, a.w.max_pages)) a.free_pages[at] = a.table[(base + k) * a.w.table_stride + col];
      }
      before += here;
      __syncthreads();
    }
  }
  // (the stack is complete for all threads: the barrier of the next scan, at the latest, lies between)
  long long lacked = 0, taken = 0;
  for (int base = 0; base < batch; base += kThreads) {
    const int b = base + tid;
    const Need n = b < batch ? need_of(a, b) : Need{0, 0, false};
    const int lack = max(n.want - n.held, 0);
    const long long upto = block_inclusive(lack, scratch);
    const bool refused = lack > 0 && lacked + upto > there;
    sums[tid] = upto;
    first[tid] = refused ? -1 : n.held;
    const long long here = scratch[32];
    __syncthreads();
    for (long long i = tid; i < here && lacked + i < there; i += kThreads) {
      const int k = owner(sums, i);
      if (first[k] < 0) continue;
      const int col = first[k] + static_cast<int>(i - (k > 0 ? sums[k - 1] : 0));
      const long long at = there - 1 - (lacked + i);
      if (sv_in(at, size) && sv_in(col, a.w.max_pages)) a.table[(base + k) * a.w.table_stride + col] = a.free_pages[at];
    }
    if (b < batch) {
      if (!refused) a.held[b] = n.want;
      if (a.w.status) a.w.status[b] = n.ok ? refused ? SV_ROW_NO_PAGE : 0 : SV_ROW_BAD_LENGTH;
    }
    taken += refused ? 0 : lack;
    lacked += here;
    __syncthreads();
  }
  block_inclusive(taken, scratch);
  if (tid == 0) *a.free_count = static_cast<int>(there - scratch[32]);
}

// A thread a token: tx tokens at a time of each of 256 / tx sequences to a block.
constexpr int kPlaceThreads = 256;

__device__ void place_token(const AssignView& a, int b, const KvSpan& s, int held, int i) {
  const int64_t row = s.row0 + static_cast<int64_t>(i);
  if (!kv_row_in(a.w, row)) return;
  if (!s.ok || held < 0 || held > a.w.max_pages) {
    if (a.slots) a.slots[row] = -1;
    if (a.positions) a.positions[row] = 0;
    return;
  }
  if (a.positions) a.positions[row] = s.ctx + (a.parents ? depth_of(a, b, a.parents + s.row0, i) : i);
  if (!a.slots) return;
  const int j = s.ctx + i, col = j >> a.w.page_shift;
  const bool served = static_cast<int64_t>(held) << a.w.page_shift >= static_cast<int64_t>(s.ctx) + s.n && sv_in(col, a.w.max_pages);
  a.slots[row] = served ? slot_on(a, b, a.table[b * a.w.table_stride + col], j) : -1;
}

__global__ void __launch_bounds__(kPlaceThreads) kv_assign_places_kernel(AssignView a, int tx_shift) {
  const int tx = 1 << tx_shift;
  const int b = blockIdx.y * (kPlaceThreads >> tx_shift) + (threadIdx.x >> tx_shift);
  wait_for_stream();
  if (b >= a.w.batch) return;
  const KvSpan s = kv_span(a.w, b);
  const int held = a.held[b];
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * tx + (threadIdx.x & (tx - 1)); i < s.n; i += static_cast<int64_t>(gridDim.x) * tx)
    place_token(a, b, s, held, static_cast<int>(i));
}

// From this many new tokens to place, or pages that may move, on, several blocks do that, in two launches behind a memset of the
// flags.  64 sequences with a token each take 4.3 us in one block and 10.3 in several (6.7 without flags); without flags 2048 tokens
// take 5.6 in one and 6.6 in several, 4000 7.1 and 6.5, 8000 10.5 and 6.5; pages cost one block 0.5 us for 1000 that move.  A call
// of new tokens takes about the pages that these fill, whatever the table has room for (64 sequences with room for 2048 pages each:
// 4.6 us, 10.3 where the room decided), and a call without any may give back all that the pool has.  (Should a call of few tokens
// move 120,000 pages, they take 62 us more than in several blocks.)
constexpr int64_t kManyPages = 16384, kManyTokens = 4000;

}  // namespace

sv_status kv_assign(const sv_kv_assign_desc& d, int32_t* free_pages, int32_t* free_count, int32_t* page_table, int32_t* held,
                    const int32_t* ctx_lens, const int32_t* new_start, const int32_t* parents, int64_t* slots,
                    int32_t* positions, int32_t* row_status, cudaStream_t stream) {
  start_phases(stream);
  sv_kv_desc k{};
  k.batch = d.batch;
  k.page_size = d.page_size;
  k.num_pages = d.num_pages;
  k.max_pages = d.max_pages;
  k.table_stride = d.table_stride;
  KvCache c{};
  c.page_table = page_table;
  const AssignView a{kv_view(k, c, ctx_lens, new_start, d.max_new, d.total_new, row_status),
                     free_pages, free_count, page_table, held, parents, slots, positions};
  if (d.batch <= kThreads) {
    const int64_t tokens = slots || positions ? d.total_new : 0;
    const int64_t room = std::min<int64_t>(static_cast<int64_t>(d.batch) * d.max_pages, d.num_pages);
    const int64_t pages = std::min<int64_t>(room, d.total_new > 0 ? d.total_new / d.page_size + d.batch : room);
    if (pages <= kManyPages && tokens <= kManyTokens) {
      if (launch_early(kv_assign_few_kernel<kAll>, dim3(1), dim3(kThreads), 0, stream, a) != cudaSuccess) return SV_ERR_CUDA;
      note_launch(stream);
      return SV_OK;
    }
    if (row_status && cudaMemsetAsync(row_status, 0, static_cast<size_t>(d.batch) * sizeof(int32_t), stream) != cudaSuccess) return SV_ERR_CUDA;
    const int64_t share = std::max(room, tokens) / (2 * kThreads) + 1;
    const unsigned blocks = static_cast<unsigned>(std::min<int64_t>(share, 152));
    if (launch_early(kv_assign_few_kernel<kMove>, dim3(blocks), dim3(kThreads), 0, stream, a) != cudaSuccess) return SV_ERR_CUDA;
    note_launch(stream);
    if (launch_early(kv_assign_few_kernel<kUpdate>, dim3(1), dim3(kThreads), 0, stream, a) != cudaSuccess) return SV_ERR_CUDA;
    note_launch(stream);
    return SV_OK;
  }
  kv_assign_pages_kernel<<<1, kThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  if (d.max_new == 0 || d.total_new == 0 || (!slots && !positions)) return SV_OK;
  int shift = 0;
  while ((1 << shift) < d.max_new && (1 << shift) < kPlaceThreads) ++shift;
  const int per = kPlaceThreads >> shift;
  // (max_new may be far more than any sequence brings)
  constexpr int64_t kPlaceBlocks = 152 * 64;
  const int64_t y = (d.batch + per - 1) / per, x = (static_cast<int64_t>(std::min(d.max_new, d.total_new)) + (1 << shift) - 1) >> shift;
  const dim3 grid(static_cast<unsigned>(std::min(x, std::max<int64_t>(kPlaceBlocks / y, 1))), static_cast<unsigned>(y));
  if (launch_early(kv_assign_places_kernel, grid, dim3(kPlaceThreads), 0, stream, a, shift) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
