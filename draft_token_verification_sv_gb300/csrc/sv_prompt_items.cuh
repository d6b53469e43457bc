// How the tensor core kernels of prompt attention share their work out.
//
// An item is one kv head and 128 rows of queries, or NQ times 128: row r of a
// tile is token r / group and head r % group of those that share the kv head,
// so that short prompts and odd groups fill tiles, too, and a tile's keys end
// close behind its tokens.
#pragma once

#include "sv_prompt.cuh"
#include "sv_tcgen05.cuh"

#include <algorithm>

namespace sv {

constexpr int kRows = 128;  // of a tile of queries

// A block's tile of keys or values that is never loaded, in builds that test what happens when waits run out.
#ifndef SV_PROMPT_LOST_TILE
#define SV_PROMPT_LOST_TILE -1
#endif

struct Item {
  int row0, n, h;        // the sequence's rows, the kv head
  int tok0;              // first token
  int tiles;             // of keys, -1: no more items
  int count[2];          // of them for each tile of queries
  int first, window;     // tiles of the first tokens (sinks), then from this tile on
  int dirty;             // not 0: values that are not finite were taken out
};

// Sequences where they are few: the longest first, their rows, and the items up to and with each.  Where they are more, packed ones:
// the items up to and with each of at most kSorted runs of them (padded ones need none: all have as many).
constexpr int kSorted = 96;
struct Sequences {
  union {
    struct {
      int n[kSorted], row0[kSorted];
    } few;
    long long upto[kSorted];
  };
  int items[kSorted];
};

// Of how many sequences a run is, where they are more than kSorted.
__device__ __forceinline__ int run_of(const PromptView& a) { return (a.batch + kSorted - 1) / kSorted; }

// Items of the runs, a warp a run, and their sums: without them a search went through all sequences (16,000 padded ones of 8 tokens
// took 112 ms).
__device__ __forceinline__ void sum_runs(const PromptView& a, Sequences& sq, int per, int threads) {
  const int run = run_of(a), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < kSorted; r += threads >> 5) {
    const int end = min((r + 1) * run, a.batch);
    long long own = 0;
    for (int b = r * run + lane; b < end; b += 32) own += static_cast<long long>((prompt_span(a, b).n + per - 1) / per) * a.kv_heads;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) own += __shfl_down_sync(0xffffffffu, own, o);
    if (lane == 0) sq.upto[r] = own;
  }
  __syncthreads();
  if (warp == 0) {
    long long before = 0;
    for (int r = lane; r < kSorted; r += 32) {
      long long upto = sq.upto[r];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      sq.upto[r] = before + upto;
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
}

// By all threads of the block, of `per` tokens to an item; complete behind its next barrier.
__device__ __forceinline__ void sort_sequences(const PromptView& a, Sequences& sq, int per, int threads) {
  if (a.batch > kSorted) {
    if (a.new_start) sum_runs(a, sq, per, threads);
    return;
  }
  for (int b = threadIdx.x; b < a.batch; b += threads) sq.items[b] = prompt_span(a, b).n;
  __syncthreads();
  int rank = -1, before = 0;
  PromptSpan s{};
  for (int b = threadIdx.x; b < a.batch; b += threads) {  // (one for a thread at most: no block is smaller than kSorted)
    s = prompt_span(a, b);
    rank = 0;
    for (int o = 0; o < a.batch; ++o) {
      const int n = sq.items[o];
      if (n > s.n || (n == s.n && o <= b)) {
        rank += o != b;
        before += (n + per - 1) / per * a.kv_heads;
      }
    }
  }
  __syncthreads();
  if (rank >= 0) {
    sq.few.n[rank] = s.n;
    sq.few.row0[rank] = s.row0;
    sq.items[rank] = before;
  }
}

// Flags of sequences that are left out, by one block's threads.
__device__ __forceinline__ void flag_lengths(const PromptView& a, int threads) {
  if (a.status)
    for (int b = threadIdx.x; b < a.batch; b += threads)
      if (!prompt_span(a, b).ok) prompt_flag(a, b, SV_ROW_BAD_LENGTH);
}

// First key of the item's tile t.
template <int KEYS>
__device__ __forceinline__ int key_of(const Item& it, int t) {
  return KEYS * (t < it.first ? t : it.window + t - it.first);
}

// Does every row of tile i of queries see all of the tile at key kb?
template <int KEYS>
__device__ __forceinline__ bool whole(const PromptView& a, const Item& it, int tpt, int i, int kb) {
  const int first = it.tok0 + i * tpt, last = min(first + tpt, it.n) - 1;
  return kb + KEYS - 1 <= first && (a.window == 0 || last - kb < a.window || kb + KEYS - 1 < a.sinks);
}

// Are there rows that do not see all of tile t?
template <int KEYS, int NQ>
__device__ __forceinline__ bool partly_seen(const PromptView& a, const Item& it, int tpt, int t) {
  bool all = true;
#pragma unroll
  for (int i = 0; i < NQ; ++i) all = all && (t >= it.count[i] || whole<KEYS>(a, it, tpt, i, key_of<KEYS>(it, t)));
  return !all;
}

// The u-th of an item's tiles of keys and values in the order in which they are loaded and used: each tile's keys and then its
// values or, AHEAD, the next tile's keys, whose scores are formed meanwhile, before the values.
struct Turn {
  bool keys;
  int t;
};
template <bool AHEAD>
__device__ __forceinline__ Turn turn_of(int u, int tiles) {
  if (!AHEAD) return Turn{(u & 1) == 0, u >> 1};
  const bool last = u == 2 * tiles - 1;
  const bool keys = !last && (u == 0 || (u & 1));
  return Turn{keys, keys ? (u + 1) >> 1 : last ? tiles - 1 : (u >> 1) - 1};
}

// The lowest n bits, none for less, all for more.
__device__ __forceinline__ uint32_t bits_below(int n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(32 - min(max(n, 0), 32)));  // (which moves by 32, too)
  return r;
}

// Finds items by their numbers: sequences in order (longest first where they are few), in each the last tokens first, kv heads
// innermost.  One warp.  (32 sequences of a run are looked at at a time, 683 at most.)
struct Finder {
  int at;            // sequences passed
  long long before;  // items of those

  template <int KEYS, int NQ>
  __device__ __forceinline__ bool find(const PromptView& a, const Sequences& sq, int tpt, long long index, Item& it) {
    const int per = NQ * tpt;
    int local;  // the item's number among its sequence's
    if (a.batch <= kSorted) {
      if (!find_sorted(a, sq, index, it, local)) return false;
    } else if (a.new_start ? !find_packed(a, sq, per, index, it, local) : !find_padded(a, per, index, it, local)) {
      return false;
    }
    const int group = local / a.kv_heads;
    it.h = local - group * a.kv_heads;
    it.tok0 = ((it.n - 1) / per - group) * per;
    const int from = a.window ? max(0, it.tok0 - a.window + 1) : 0;
    it.window = from / KEYS;
    it.first = a.window ? min(it.window, a.sinks / KEYS + (a.sinks % KEYS != 0)) : 0;
    it.tiles = 0;
    it.dirty = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int first = it.tok0 + i * tpt, last = min(it.n, first + tpt) - 1;
      it.count[i] = i < NQ && first < it.n ? it.first + last / KEYS - it.window + 1 : 0;
      it.tiles = max(it.tiles, it.count[i]);
    }
    return true;
  }

  __device__ __forceinline__ bool find_sorted(const PromptView& a, const Sequences& sq, long long index, Item& it, int& local) {
    for (int base = 0; base < a.batch; base += 32) {
      const int o = base + (threadIdx.x & 31);
      const unsigned past = __ballot_sync(0xffffffffu, o < a.batch && sq.items[o] > index);
      if (past == 0) continue;
      const int who = base + __ffs(past) - 1;
      it.n = sq.few.n[who];
      it.row0 = sq.few.row0[who];
      local = static_cast<int>(index) - (who > 0 ? sq.items[who - 1] : 0);
      return true;
    }
    return false;
  }

  // (There are fewer than 2^31 items, and an index is less than 2^30 beyond.)
  __device__ __forceinline__ bool find_padded(const PromptView& a, int per, long long index, Item& it, int& local) {
    const unsigned own = static_cast<unsigned>((a.max_new + per - 1) / per) * static_cast<unsigned>(a.kv_heads), i = static_cast<unsigned>(index);
    const unsigned who = own > 0 ? i / own : static_cast<unsigned>(a.batch);
    if (who >= static_cast<unsigned>(a.batch)) return false;
    it.n = a.max_new;
    it.row0 = static_cast<int>(who) * a.max_new;
    local = static_cast<int>(i - who * own);
    return true;
  }

  __device__ __forceinline__ bool find_packed(const PromptView& a, const Sequences& sq, int per, long long index, Item& it, int& local) {
    const int lane = threadIdx.x & 31, run = run_of(a);
    // the run that holds it, from its first sequence on or from where the last search ended
    int r = 0;
    for (; r < kSorted; r += 32) {
      const unsigned past = __ballot_sync(0xffffffffu, sq.upto[r + lane] > index);
      if (past == 0) continue;
      r += __ffs(past) - 1;
      break;
    }
    if (r >= kSorted) return false;
    if (at < r * run || at >= (r + 1) * run || before > index) {
      at = r * run;
      before = r > 0 ? sq.upto[r - 1] : 0;
    }
    for (; at < a.batch;) {
      const PromptSpan s = at + lane < a.batch ? prompt_span(a, at + lane) : PromptSpan{0, 0, false};
      const long long own = static_cast<long long>((s.n + per - 1) / per) * a.kv_heads;
      long long upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + upto > index);
      if (past == 0) {
        before += __shfl_sync(0xffffffffu, upto, 31);
        at += 32;
        continue;
      }
      const int who = __ffs(past) - 1;
      it.n = __shfl_sync(0xffffffffu, s.n, who);
      it.row0 = __shfl_sync(0xffffffffu, s.row0, who);
      local = static_cast<int>(index - before - __shfl_sync(0xffffffffu, upto - own, who));
      return true;
    }
    return false;
  }
};

// A row of the call's results for row r of tile i, or -1.
struct Place {
  int64_t row;
  int token, head;
};
__device__ __forceinline__ Place place_of(const PromptView& a, const Item& it, int tpt, int i, int r) {
  Place p;
  const int t = r / a.group;
  p.token = it.tok0 + i * tpt + t;
  p.head = it.h * a.group + r - t * a.group;
  p.row = t < tpt && p.token < it.n && sv_in(it.row0 + static_cast<int64_t>(p.token), a.total_new) ? it.row0 + static_cast<int64_t>(p.token) : -1;
  return p;
}

// A block for each item (of `per` tokens): of packed sequences it is not known on the host how many there are, at most one more a
// sequence and head than their tokens fill.  Blocks take items beyond the grid, too.
inline unsigned prompt_blocks(const PromptView& a, int per) {
  const int64_t blocks = a.new_start ? (static_cast<int64_t>(a.total_new) / per + std::min<int64_t>(a.batch, 4096 / a.kv_heads + 1)) * a.kv_heads
                                     : static_cast<int64_t>(a.batch) * ((a.max_new + per - 1) / per) * a.kv_heads;
  return static_cast<unsigned>(std::min<int64_t>(std::max<int64_t>(blocks, 1), 1 << 30));
}

__device__ __forceinline__ float value_of(const float* p) { return __ldg(p); }
__device__ __forceinline__ float value_of(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16); }
__device__ __forceinline__ void put_value(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_value(uint16_t* p, float v) { *p = static_cast<uint16_t>(floats_to_bf16x2(v, 0.0f)); }

__device__ __forceinline__ float held_at(const float* p) { return *p; }
__device__ __forceinline__ float held_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }

// Adds to a row's results what it sees of values that are not finite and were taken out: those of tiles that every row sees, which
// were added up (NULL: none were taken out), and, token by token, those of the few others.
template <int KEYS, typename E>
__device__ __noinline__ void add_rest(const PromptView& a, const Item& it, int tpt, int token, E* out, const volatile float* whole_tiles) {
  if (whole_tiles)
    for (int d = 0; d < a.dim; ++d) {
      const float y = whole_tiles[d];
      if (y != 0.0f) put_value(out + d, held_at(out + d) + y);
    }
  const E* v = static_cast<const E*>(a.v) + static_cast<int64_t>(it.row0) * a.v_row + it.h * a.v_head;
  for (int t = 0; t < it.tiles; ++t) {
    if (!partly_seen<KEYS, 2>(a, it, tpt, t)) continue;
    const int kb = key_of<KEYS>(it, t);
    for (int j = kb; j < kb + KEYS && j <= token; ++j) {
      if (a.window != 0 && token - j >= a.window && j >= a.sinks) continue;
      if (!sv_in(it.row0 + static_cast<int64_t>(j), a.total_new)) break;
      for (int d = 0; d < a.dim; ++d) {
        const float y = value_of(v + j * a.v_row + d);
        if (!(fabsf(y) < CUDART_INF_F)) put_value(out + d, held_at(out + d) + y);
      }
    }
  }
}

// A wait ran out: results of the item are not valid.
template <typename E>
__device__ __noinline__ void spoil(const PromptView& a, const Item& it, int tpt, int nq, int thread, int threads) {
  for (int b = thread; b < a.batch; b += threads) {
    const PromptSpan s = prompt_span(a, b);
    if (s.ok && s.row0 == it.row0 && s.n == it.n) prompt_flag(a, b, SV_ROW_TIMEOUT);
  }
  for (int r = thread; r < nq * kRows; r += threads) {
    const Place p = place_of(a, it, tpt, r / kRows, r % kRows);
    if (p.row < 0) continue;
    E* out = static_cast<E*>(a.out) + p.row * a.out_row + p.head * a.out_head;
    for (int d = 0; d < a.dim; ++d) put_value(out + d, CUDART_NAN_F);
    if (a.lse) a.lse[p.row * a.heads + p.head] = CUDART_NAN_F;
  }
}

}  // namespace sv
