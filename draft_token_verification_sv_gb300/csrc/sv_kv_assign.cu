// Pages for the sequences' lengths, and a slot and a position for every new
// token.  Bound by latency for a decoding step (dependent loads: lengths, the
// stack's count, page ids), by the slots and positions written for prompts.
#include "sv_kv.cuh"

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

// The first of the block's sequences whose inclusive sum is above i.
__device__ __forceinline__ int owner(const long long* sums, long long i) {
  int lo = 0, hi = kThreads - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

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

// A thread a token: tx tokens of each of 256 / tx sequences to a block.
constexpr int kPlaceThreads = 256;

__global__ void __launch_bounds__(kPlaceThreads) kv_assign_places_kernel(AssignView a, int tx_shift) {
  const int tx = 1 << tx_shift;
  const int b = blockIdx.y * (kPlaceThreads >> tx_shift) + (threadIdx.x >> tx_shift);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * tx + (threadIdx.x & (tx - 1));
  wait_for_stream();
  if (b >= a.w.batch) return;
  const KvSpan s = kv_span(a.w, b);
  if (i >= s.n) return;
  const int64_t row = s.row0 + i;
  if (!kv_row_in(a.w, row)) return;
  const int held = a.held[b];
  const bool ok = s.ok && held >= 0 && held <= a.w.max_pages;
  if (!ok) {
    if (a.slots) a.slots[row] = -1;
    if (a.positions) a.positions[row] = 0;
    return;
  }
  int depth = static_cast<int>(i);
  if (a.parents) {
    const int32_t* parents = a.parents + s.row0;
    depth = 0;
    for (int u = static_cast<int>(i); u >= 0;) {
      const int p = __ldg(parents + u);
      if (u == i && (u == 0 ? p != -1 : (p < 0 || p >= u))) kv_flag(a.w, b, SV_ROW_BAD_PARENT);
      u = p >= 0 && p < u ? p : -1;
      depth += u >= 0;
    }
  }
  if (a.positions) a.positions[row] = s.ctx + depth;
  if (!a.slots) return;
  const int j = s.ctx + static_cast<int>(i), col = j >> a.w.page_shift;
  int64_t slot = -1;
  if (static_cast<int64_t>(held) << a.w.page_shift >= static_cast<int64_t>(s.ctx) + s.n && sv_in(col, a.w.max_pages)) {
    const int page = a.table[b * a.w.table_stride + col];
    if (page >= 0 && page < a.w.num_pages)
      slot = (static_cast<int64_t>(page) << a.w.page_shift) + (j & ((1 << a.w.page_shift) - 1));
    else
      kv_flag(a.w, b, SV_ROW_BAD_PAGE);
  }
  a.slots[row] = slot;
}

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
  kv_assign_pages_kernel<<<1, kThreads, 0, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  if (d.max_new == 0 || d.total_new == 0 || (!slots && !positions)) return SV_OK;
  int shift = 0;
  while ((1 << shift) < d.max_new && (1 << shift) < kPlaceThreads) ++shift;
  const int per = kPlaceThreads >> shift;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(d.max_new) + (1 << shift) - 1) >> shift),
                  static_cast<unsigned>((d.batch + per - 1) / per));
  if (launch_early(kv_assign_places_kernel, grid, dim3(kPlaceThreads), 0, stream, a, shift) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace sv
