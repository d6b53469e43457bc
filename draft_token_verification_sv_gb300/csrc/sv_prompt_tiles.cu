// Causal attention of bf16 prompts on the 5th-generation tensor cores.
//
// A block takes 128 rows, or two times 128, of one kv head's queries at a time
// (sv_prompt_items.cuh).  S = Q K^T and O += P V run against tiles of 128 keys:
// Q, K and V come by tensor copies to shared memory, S and O are in tensor
// memory, where the weights P take the place of their scores.
// Roles of a block's warps:
//   one loads: it finds the items and copies queries, keys and values;
//   one issues the products;
//   two look at the values of tiles that some rows do not see whole (below);
//   four for each 128 rows turn scores into weights, a row a thread.
// Weights are exp2(s - m) with m the largest of the first scores that the row
// sees: bf16 weights have float's range, so m moves (and O is scaled anew) only
// where a tile's weights get large against it (a sum of more than 2^13), and
// what a weight loses by a small m is nothing.  Weights are rounded to bf16 (2^-8),
// the type that the products ask for beside bf16 values; their sum is taken
// before that, in fp32.
// What a row does not see has weight 0, but 0 times what is not finite is not
// 0: values of partly seen tiles that are not finite become 0 in shared memory
// before their product, and rows that do see them get them where results are
// written.
//
// Two prompts of up to 8192 tokens (32 heads of 128 dims) take 575 to 631 us, by
// what power allows: 1680 to 1530 TFLOP/s, 85 to 77% of the measured rate of a
// matrix product.  The tensor core bounds it, two tiles of queries against 128
// keys at a time, one of which has its scores turned into weights while the
// other's products run.  Prompts of up to
// 836 tokens (80 us) are bound by each item's chain: its first and its masked
// tiles, its results, and the instructions of these, which are fetched anew for
// each item.  256 dims leave room for one tile of queries, so each tile of keys and
// values, 128 KB, is read for that alone, and nothing but the next tile's scores
// runs beside a tile's weights (68 us for three prompts of up to 2011 tokens with
// 14 heads, 930 TFLOP/s; the tensor core is active for half of it, the banks of
// shared memory for 17% in reads and 12% in writes, as far as these count).
#include "sv_prompt_items.cuh"

#include <type_traits>

namespace sv {

namespace {

constexpr int kKeys = 128;   // of a tile of keys
constexpr int kItems = 4;    // items that may be known ahead
constexpr int kSoftmaxRegisters = 208, kOtherRegisters = 88;  // of 168 at launch, where there are three groups of four warps
static_assert(8 * kSoftmaxRegisters + 4 * kOtherRegisters <= 12 * 168, "registers of a block");
constexpr float kLargeSum = 8192.0f, kLargeLog = 13.0f;

template <int DP> struct Config {
  static constexpr int NQ = DP == 256 ? 1 : 2;           // tiles of queries
  static constexpr int kHalves = DP == 256 ? 2 : 1;      // copies of a tile of keys or values, of 128 dims at most
  static constexpr int kUnitDims = DP / kHalves;
  static constexpr int kUnitBytes = kKeys * kUnitDims * 2;
  static constexpr int kBlockBytes = kKeys * 128;        // 64 dims of a tile
  static constexpr int kQueryBytes = kRows * DP * 2;
  static constexpr int kStages = DP == 64 ? 10 : 5;
  static constexpr int kShared = NQ * kQueryBytes + kStages * kUnitBytes + 1024;
  static constexpr int kSoftmaxWarps = 4 * NQ, kCheckWarps = 2;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
  // tensor memory, in columns: two places for scores, then O
  static constexpr int kS = 0, kO = 2 * kKeys;
};

struct Shared {
  uint64_t item_full[kItems], item_free[kItems];
  uint64_t q_full[2], q_free[2];
  uint64_t kv_full[10], kv_free[10], checked[10];
  uint64_t s_full[2], p_ready[2], pv_done[2], o_free[2], last, answer;
  uint4 block;           // what ask_for_block brings
  Item item[kItems];
  Sequences sequences;
  uint32_t tmem;
  int gave_up;
  int look[10];          // of the values in a stage the last ones that some rows do not see
  int claimed, finished[8];  // items known, and done with by each warp that writes results
};

__device__ __forceinline__ bool warp_wait(Shared& sh, uint64_t& bar, int n) {
  return __all_sync(0xffffffffu, tc::barrier_wait(tc::smem_address(&bar), static_cast<uint32_t>(n & 1), &sh.gave_up));
}
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::barrier_arrive(tc::smem_address(&bar));
}

// ---- loading ----

struct Maps {
  CUtensorMap q, k, v;
};

// What the loading warp has under way.
struct Loads {
  int units, queries[2];  // copies of keys and values, of queries
  int answers;            // questions for a block that were answered
  bool asked;             // and one that was not
  long long next;         // the number of the item that is published next
};

template <int DP>
__device__ __forceinline__ bool find_item(const PromptView& a, const Sequences& sq, int tpt, Finder& finder, long long index, Item& it) {
  return finder.find<kKeys, Config<DP>::NQ>(a, sq, tpt, index, it);
}

template <int DP>
__device__ bool load_role(const PromptView& a, const Maps& maps, int tpt, Shared& sh, uint32_t q_at, uint32_t kv_at, Finder& finder, Loads& under) {
  using C = Config<DP>;
  const int lane = threadIdx.x & 31;
  int items = 0, tile = 0;
  Item it;
  for (int x = blockIdx.x; x >= 0;) {
    if (lane == 0) {
      const uint32_t bar = tc::smem_address(&sh.answer);
      tc::barrier_expect(bar, sizeof(sh.block));
      tc::ask_for_block(tc::smem_address(&sh.block), bar);
    }
    under.asked = true;
    under.next = x;
    while (find_item<DP>(a, sh.sequences, tpt, finder, under.next, it)) {
      if (items >= kItems && !warp_wait(sh, sh.item_free[items % kItems], items / kItems - 1)) return false;
      if (lane == 0) {
        sh.item[items % kItems] = it;
        sh.claimed = items + 1;
      }
      warp_arrive(sh.item_full[items % kItems]);
      ++items;
      under.next += gridDim.x;
#pragma unroll 1
      for (int i = 0; i < C::NQ; ++i) {
        if ((i ? it.count[1] : it.count[0]) == 0) continue;
        const int before = i ? under.queries[1] : under.queries[0];
        if (before > 0 && !warp_wait(sh, sh.q_free[i], before - 1)) return false;
        const uint32_t bar = tc::smem_address(&sh.q_full[i]);
        if (lane == 0) {
          tc::barrier_expect(bar, tpt * a.group * DP * 2);
#pragma unroll
          for (int d = 0; d < DP; d += 64)
            tc::copy_box(q_at + i * C::kQueryBytes + d / 64 * (kRows * 128), &maps.q, d, it.h * a.group, it.row0 + it.tok0 + i * tpt, bar);
        }
        (i ? under.queries[1] : under.queries[0]) = before + 1;
      }
#pragma unroll 1
      for (int u = 0; u < 2 * it.tiles; ++u) {
        if (tile++ == SV_PROMPT_LOST_TILE) return false;
        const Turn turn = turn_of<C::NQ == 1>(u, it.tiles);
        const int kb = key_of<kKeys>(it, turn.t);
        const CUtensorMap* map = turn.keys ? &maps.k : &maps.v;
        // (without a window every row sees those up to the first token)
        const int look = turn.keys || !partly_seen<kKeys, C::NQ>(a, it, tpt, turn.t) ? 0 : a.window ? kKeys : kKeys - max(0, it.tok0 + 1 - kb);
#pragma unroll 1
        for (int half = 0; half < C::kHalves; ++half) {
          const int unit = under.units, stage = unit % C::kStages;
          if (unit >= C::kStages && !warp_wait(sh, sh.kv_free[stage], unit / C::kStages - 1)) return false;
          const uint32_t bar = tc::smem_address(&sh.kv_full[stage]);
          if (lane == 0) {
            sh.look[stage] = look;
            tc::barrier_expect(bar, C::kUnitBytes);
#pragma unroll
            for (int d = 0; d < C::kUnitDims; d += 64)
              tc::copy_box(kv_at + stage * C::kUnitBytes + d / 64 * C::kBlockBytes, map, half * C::kUnitDims + d, it.h, it.row0 + kb, bar);
          }
          ++under.units;
        }
      }
    }
    if (!warp_wait(sh, sh.answer, under.answers)) return false;
    ++under.answers;
    under.asked = false;
    x = tc::taken_block(tc::smem_address(&sh.block));
    __syncwarp();
    tc::publish_shared();  // (read before the next answer is written)
  }
  if (items >= kItems && !warp_wait(sh, sh.item_free[items % kItems], items / kItems - 1)) return false;
  if (lane == 0) sh.item[items % kItems].tiles = -1;
  warp_arrive(sh.item_full[items % kItems]);
  return true;
}

// What is under way when the loading warp gives up ends before its memory does: the last copies to each place, which no other
// role may have waited for, and the answer.  Items that no other role knows of are spoilt here.
template <int DP>
__device__ __noinline__ void end_loads(const PromptView& a, int tpt, Shared& sh, Finder& finder, Loads& under) {
  using C = Config<DP>;
  int unused = 0;
  for (int u = max(0, under.units - C::kStages); u < under.units; ++u)
    tc::barrier_wait(tc::smem_address(&sh.kv_full[u % C::kStages]), u / C::kStages & 1, &unused, tc::kEndCycles);
  for (int i = 0; i < C::NQ; ++i)
    if (under.queries[i] > 0) tc::barrier_wait(tc::smem_address(&sh.q_full[i]), under.queries[i] - 1 & 1, &unused, tc::kEndCycles);
  Item it;
  for (;;) {
    for (; find_item<DP>(a, sh.sequences, tpt, finder, under.next, it); under.next += gridDim.x) spoil<uint16_t>(a, it, tpt, C::NQ, threadIdx.x & 31, 32);
    if (!under.asked) return;
    under.asked = false;
    const bool answered = tc::barrier_wait(tc::smem_address(&sh.answer), under.answers & 1, &unused, tc::kEndCycles);
    under.next = __all_sync(0xffffffffu, answered) ? tc::taken_block(tc::smem_address(&sh.block)) : -1;
    if (under.next < 0) return;
  }
}

// ---- values that are not finite ----

// Both values of a word, 0 where they are not finite.
__device__ __forceinline__ uint32_t finite_of(uint32_t w) { return w & ~__vcmpgeu2(w & 0x7fff7fffu, 0x7f807f80u); }

// The top bit of each half is set where its value is not finite: an exponent of ones carries into it.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; }

// It takes part in every copy's way, so that it is never a round of the stages behind.  (The last tile's sums wait for it: with all
// of its values looked at, 256 dims took 72 us.)
template <int DP>
__device__ bool check_role(Shared& sh, uint8_t* kv) {
  using C = Config<DP>;
  const int tid = threadIdx.x - 32 * (C::kSoftmaxWarps + 2);
  int unit = 0;
  for (int items = 0;; ++items) {
    if (!warp_wait(sh, sh.item_full[items % kItems], items / kItems)) return false;
    Item& it = sh.item[items % kItems];
    const int tiles = it.tiles;
    if (tiles < 0) return true;
#pragma unroll 1
    for (int u = 0; u < 2 * C::kHalves * tiles; ++u, ++unit) {
      const int stage = unit % C::kStages;
      if (!warp_wait(sh, sh.kv_full[stage], unit / C::kStages)) return false;
      if (const int look = sh.look[stage]) {
        bool found = false;
#pragma unroll 1
        for (int block = 0; block < C::kUnitBytes; block += C::kBlockBytes) {
          uint4* at = reinterpret_cast<uint4*>(kv + stage * C::kUnitBytes + block) + (kKeys - look) * 8;
#pragma unroll 2
          for (int c = tid; c < look * 8; c += 32 * C::kCheckWarps) {
            const uint4 v = at[c];
            if ((not_finite(v.x) | not_finite(v.y) | not_finite(v.z) | not_finite(v.w)) & 0x80008000u) {
              found = true;
              at[c] = make_uint4(finite_of(v.x), finite_of(v.y), finite_of(v.z), finite_of(v.w));
            }
          }
        }
        if (found) it.dirty = 1;
        tc::publish_shared();
        warp_arrive(sh.checked[stage]);
      }
      warp_arrive(sh.kv_free[stage]);
    }
    warp_arrive(sh.item_free[items % kItems]);
  }
}

// ---- products ----

// A place in the ring of stages, and the parity of its barriers' phase.
template <int STAGES>
struct Ring {
  int stage;
  uint32_t parity;
  __device__ __forceinline__ Ring next() const {
    return stage + 1 == STAGES ? Ring{0, parity ^ 1u} : Ring{stage + 1, parity};
  }
};

// One thread.  Eight products or so may wait for the tensor core, 65 cycles each: what the thread does between two batches is kept
// shorter than that (parities in bits, each tile of keys and values waited for once).
template <int DP>
__device__ bool product_role(const PromptView& a, Shared& sh, uint32_t q_at, uint32_t kv_at, uint32_t tmem) {
  using C = Config<DP>;
  constexpr uint32_t kScores = tc::product_kind_bf16(kKeys, false), kValues = tc::product_kind_bf16(C::kUnitDims, true);
  const auto wait = [&](uint64_t& bar, uint32_t parity) { return tc::barrier_wait(tc::smem_address(&bar), parity & 1u, &sh.gave_up); };
  const auto arrive = [&](uint64_t& bar) { tc::products_arrive(tc::smem_address(&bar)); };
  const uint64_t k0 = tc::tile_descriptor(kv_at, 16, 1024), q0 = tc::tile_descriptor(q_at, 16, 1024);
  const uint64_t v0 = tc::tile_descriptor(kv_at, C::kBlockBytes, 1024);
  // S in place s (+)= tile i of queries, from `half` on, with the keys of a stage
  const auto score = [&](int i, int half, int s, int stage) {
    const uint64_t q = q0 + (i * C::kQueryBytes + half * (kRows * 256) >> 4), k = k0 + (stage * C::kUnitBytes >> 4);
#pragma unroll
    for (int d = 0; d < C::kUnitDims / 16; ++d) {
      const int off = (d >> 2) * (kRows * 128) + (d & 3) * 32 >> 4;  // (tiles of queries and keys are of one height)
      tc::product_f16(tmem + C::kS + s * kKeys, q + off, k + off, kScores, d > 0 || half > 0);
    }
  };
  // O of tile i, from `half` on, (+)= P in place s times the values of a stage
  const auto weigh = [&](int i, int half, int s, int stage, bool add) {
    const uint64_t v = v0 + (stage * C::kUnitBytes >> 4);
#pragma unroll
    for (int k = 0; k < kKeys / 16; ++k)
      tc::product_f16(tmem + C::kO + i * DP + half * C::kUnitDims, tmem + C::kS + s * kKeys + k * 8, v + (k * 2048 >> 4), kValues, k > 0 || add);
  };
  uint32_t checks = 0;                    // parity of `checked` for each stage
  uint32_t q_par = 0, p_par = 0, o_par = 3;  // of q_full, p_ready and o_free for each tile (a barrier's phase before its first is over)
  const auto values_ready = [&](const Ring<C::kStages>& v) {
    if (!wait(sh.kv_full[v.stage], v.parity)) return false;
    if (sh.look[v.stage]) {
      if (!wait(sh.checked[v.stage], checks >> v.stage)) return false;
      checks ^= 1u << v.stage;
    }
    return true;
  };
  Ring<C::kStages> at{0, 0};
  int tile = 0;
  for (int items = 0;; ++items) {
    if (!wait(sh.item_full[items % kItems], items / kItems)) return false;
    const int tiles = sh.item[items % kItems].tiles, count0 = sh.item[items % kItems].count[0], count1 = sh.item[items % kItems].count[1];
    tc::barrier_arrive(tc::smem_address(&sh.item_free[items % kItems]));
    if (tiles < 0) return true;
    if (C::NQ == 2) {
      // after a tile's sums the next one's scores, which take the place of its weights
      Ring<C::kStages> k = at, v = at;
#pragma unroll 1
      for (int t = -1;; ++t) {
        bool k_ready = false, v_ready = false;
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const int count = i ? count1 : count0;
          // (the last of the tiles of queries that need a tile of keys lets it go)
          if (t >= 0 && t < count) {
            if (t == 0) {
              if (!wait(sh.o_free[i], o_par >> i)) return false;
              o_par ^= 1u << i;
            }
            if (!v_ready && !values_ready(v)) return false;
            v_ready = true;
            if (!wait(sh.p_ready[i], p_par >> i)) return false;
            p_par ^= 1u << i;
            tc::fence_after();
            weigh(i, 0, i, v.stage, t > 0);
            if (i == 1 || t >= count1) arrive(sh.kv_free[v.stage]);
            arrive(sh.pv_done[i]);
          }
          if (t + 1 < count) {
            if (t < 0) {
              if (!wait(sh.q_full[i], q_par >> i)) return false;
              q_par ^= 1u << i;
            }
            if (!k_ready && !wait(sh.kv_full[k.stage], k.parity)) return false;
            k_ready = true;
            tc::fence_after();
            score(i, 0, i, k.stage);
            if (i == 1 || t + 1 >= count1) arrive(sh.kv_free[k.stage]);
            arrive(sh.s_full[i]);
            if (t + 2 == count) arrive(sh.q_free[i]);
          }
        }
        if (t + 1 == tiles) break;
        v = k.next();
        k = v.next();
      }
      at = k;
    } else {
      // each tile's scores before the sums of the one before it
#pragma unroll 1
      for (int t = -1; t < tiles; ++t) {
        if (t + 1 < tiles) {
          if (t < 0) {
            if (!wait(sh.q_full[0], q_par)) return false;
            q_par ^= 1u;
          }
#pragma unroll 1
          for (int half = 0; half < C::kHalves; ++half, at = at.next()) {
            if (!wait(sh.kv_full[at.stage], at.parity)) return false;
            tc::fence_after();
            score(0, half, tile + t + 1 & 1, at.stage);
            arrive(sh.kv_free[at.stage]);
          }
          arrive(sh.s_full[tile + t + 1 & 1]);
          if (t + 2 == tiles) arrive(sh.q_free[0]);
        }
        if (t < 0) continue;
        if (t == 0) {
          if (!wait(sh.o_free[0], o_par)) return false;
          o_par ^= 1u;
        }
        if (!wait(sh.p_ready[tile + t & 1], static_cast<uint32_t>(tile + t >> 1))) return false;
#pragma unroll 1
        for (int half = 0; half < C::kHalves; ++half, at = at.next()) {
          if (!values_ready(at)) return false;
          tc::fence_after();
          weigh(0, half, tile + t & 1, at.stage, t > 0);
          arrive(sh.kv_free[at.stage]);
        }
        arrive(sh.pv_done[0]);
      }
      tile += tiles;
    }
  }
}

// ---- scores to weights, and results ----

// 32 scores to weights 2^(x f + c), packed into w; their sum.
template <bool MASKED>
__device__ __forceinline__ float weights32(const uint32_t (&x)[32], uint32_t seen, float f, float c, uint32_t (&w)[16]) {
  const uint64_t ff = tc::pair(f, f), cc = tc::pair(c, c);
  uint64_t sum[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float2 e = tc::unpair(tc::fma2(tc::pair(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), ff, cc));
    e.x = ex2(e.x);
    e.y = ex2(e.y);
    if (MASKED) {
      e.x = seen >> (2 * k) & 1u ? e.x : 0.0f;
      e.y = seen >> (2 * k + 1) & 1u ? e.y : 0.0f;
    }
    sum[k & 1] = tc::add2(sum[k & 1], tc::pair(e.x, e.y));
    w[k] = floats_to_bf16x2(e.x, e.y);
  }
  const float2 s = tc::unpair(tc::add2(sum[0], sum[1]));
  return s.x + s.y;
}

template <bool MASKED>
__device__ __forceinline__ float largest32(const uint32_t (&x)[32], uint32_t seen, float f) {
  float v[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k & 3] = fmaxf(v[k & 3], MASKED && !(seen >> k & 1u) ? -CUDART_INF_F : __uint_as_float(x[k]) * f);
  return fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
}

// (What runs once an item, or for a few of its tiles, is kept short: its instructions are fetched anew each time.)
template <int DP>
__device__ bool softmax_role(const PromptView& a, int tpt, float f, Shared& sh, uint32_t tmem, bool out_vec32) {
  using C = Config<DP>;
  const int i = threadIdx.x / kRows, r = threadIdx.x & (kRows - 1), quarter = (threadIdx.x >> 5) & 3;
  const uint32_t mine = tmem + (quarter << 21);  // the warp's 32 lanes
  const uint32_t own_o = mine + C::kO + i * DP;
  const auto wait = [&](uint64_t& bar, int n) {
    const bool ok = warp_wait(sh, bar, n);
    tc::fence_after();
    return ok;
  };
  const int row_token = r / a.group, row_head = r - row_token * a.group;
  int tile = 0;
  for (int items = 0;; ++items) {
    if (!wait(sh.item_full[items % kItems], items / kItems)) return false;
    const Item& it = sh.item[items % kItems];
    if (it.tiles < 0) return true;
    const int count = it.count[i];
    if (count > 0) {
      const int token = it.tok0 + i * tpt + row_token;
      const bool held = row_token < tpt && token < it.n && sv_in(it.row0 + static_cast<int64_t>(token), a.total_new);
      const int from = a.window ? max(0, token - a.window + 1) : 0, sinks = a.window ? min(a.sinks, token + 1) : 0;
      float m = held ? -CUDART_INF_F : 0.0f, l = 0.0f;  // what scores are taken from (base 2), the sum of weights
#pragma unroll 1
      for (int t = 0; t < count; ++t, ++tile) {
        const int s = C::NQ == 2 ? i : tile & 1, uses = C::NQ == 2 ? tile : tile >> 1;
        const int kb = key_of<kKeys>(it, t);
        const uint32_t scores = mine + C::kS + s * kKeys;
        bool slow = !whole<kKeys>(a, it, tpt, i, kb);
        if (!wait(sh.s_full[s], uses)) return false;
        if (!slow && __any_sync(0xffffffffu, m == -CUDART_INF_F)) {  // the first tile: a few of its scores will do for m
          uint32_t x[32];
          tc::tmem_load32(scores, x);
          tc::wait_loads(x);
          const float top = largest32<false>(x, 0, f);
          m = m == -CUDART_INF_F ? top : m;
          slow = __any_sync(0xffffffffu, m == -CUDART_INF_F);
        }
        if (!slow) {
          uint32_t x[2][32], w[4][16];
          float sum = 0.0f;
          tc::tmem_load32(scores, x[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tc::wait_loads(x[c & 1]);
            if (c < 3) tc::tmem_load32(scores + 32 * (c + 1), x[c + 1 & 1]);
            sum += weights32<false>(x[c & 1], 0, f, -m, w[c]);
          }
          slow = __any_sync(0xffffffffu, held && sum > kLargeSum);
          if (!slow) {
            l += sum;
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::tmem_store(scores + 16 * c, w[c]);
          }
        }
        if (slow) {
          uint32_t x[32], w[16];
          // a row sees keys [lo, hi) of the tile and, under a window, those before `low`; no row of the warp sees any from `end` on
          const int lo = from - kb, hi = held ? token + 1 - kb : 0, low = held ? sinks - kb : 0;
          const auto seen = [&](int c) {
            const uint32_t past = bits_below(hi - 32 * c);
            return a.window ? (past & ~bits_below(lo - 32 * c)) | bits_below(low - 32 * c) : past;
          };
          const int end = (__reduce_max_sync(0xffffffffu, max(min(hi, kKeys), 0)) + 31) >> 5;
          float top = m;
#pragma unroll 1
          for (int c = 0; c < end; ++c) {
            tc::tmem_load32(scores + 32 * c, x);
            const uint32_t mask = seen(c);
            tc::wait_loads(x);
            top = fmaxf(top, largest32<true>(x, mask, f));
          }
          // rows that need nothing keep what they have, to the bit
          float fix = 1.0f;
          if (held && top > m + kLargeLog) {
            fix = m == -CUDART_INF_F ? 1.0f : ex2(m - top);
            m = top;
            l *= fix;
          }
          if (t > 0 && __any_sync(0xffffffffu, fix != 1.0f)) {
            if (!wait(sh.pv_done[i], tile - 1)) return false;
#pragma unroll 1
            for (int d = 0; d < DP; d += 16) {
              tc::tmem_load16(own_o + d, w);
              tc::wait_loads(w);
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(__uint_as_float(w[k]) * fix);
              tc::tmem_store(own_o + d, w);
            }
          }
          const float base = m == -CUDART_INF_F ? 0.0f : m;
          float sum = 0.0f;
#pragma unroll 1
          for (int c = 0; c < end; ++c) {
            tc::tmem_load32(scores + 32 * c, x);
            const uint32_t mask = seen(c);
            tc::wait_loads(x);
            sum += weights32<true>(x, mask, f, -base, w);
            tc::tmem_store(scores + 16 * c, w);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) w[k] = 0;
#pragma unroll 1
          for (int c = end; c < 4; ++c) tc::tmem_store(scores + 16 * c, w);
          l += sum;
        }
        tc::wait_stores();
        // (with one tile of queries the scores do not say that the sums before them are done, and a barrier is never two phases ahead)
        if (C::NQ == 1 && t > 0 && !wait(sh.pv_done[i], tile - 1)) return false;
        tc::fence_before();
        warp_arrive(sh.p_ready[s]);
      }
      const float inv = 1.0f / l;  // (a row sees its own token: l is 0 where all of its scores are -inf, and its results NaN)
      const int64_t row = it.row0 + static_cast<int64_t>(token);
      const int head = it.h * a.group + row_head;
      uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_row + head * a.out_head;
      if (held && a.lse) a.lse[row * a.heads + head] = (m + log2f(l)) * 0.69314718055994530942f;
      if (!wait(sh.pv_done[i], tile - 1)) return false;
#pragma unroll 1
      for (int d = 0; d < DP; d += 32) {
        uint32_t o[32];
        tc::tmem_load32(own_o + d, o);
        tc::wait_loads(o);
        if (d + 32 >= DP) {
          tc::fence_before();
          warp_arrive(sh.o_free[i]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = floats_to_bf16x2(__uint_as_float(o[16 * h + 2 * k]) * inv, __uint_as_float(o[16 * h + 2 * k + 1]) * inv);
          uint16_t* to = out + d + 16 * h;
          if (!held || d + 16 * h >= a.dim) continue;
          if (out_vec32) {
            tc::store_32(to, y);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              to[2 * k] = static_cast<uint16_t>(y[k]);
              to[2 * k + 1] = static_cast<uint16_t>(y[k] >> 16);
            }
          }
        }
        __syncwarp();
      }
      if (*const_cast<const volatile int*>(&it.dirty) != 0 && held) add_rest<kKeys, uint16_t>(a, it, tpt, token, out, nullptr);
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) sh.finished[threadIdx.x >> 5] = items + 1;
    warp_arrive(sh.item_free[items % kItems]);
  }
}

static_assert(Config<128>::kShared + sizeof(Shared) <= 227 * 1024, "shared memory of a block");

template <int DP>
__global__ void __launch_bounds__(Config<DP>::kThreads, 1)
    prompt_tiles_kernel(const __grid_constant__ PromptView a, const __grid_constant__ Maps maps, int tpt, float f, int out_vec32) {
  using C = Config<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t at = tc::smem_address(raw);
  uint8_t* tiles = raw + ((at + 1023u & ~1023u) - at);
  const uint32_t q_at = tc::smem_address(tiles), kv_at = q_at + C::NQ * C::kQueryBytes;
  const int warp = threadIdx.x >> 5, tid = threadIdx.x;
  if (tid == 0) {
    sh.gave_up = 0;
    sh.claimed = 0;
    for (int i = 0; i < 8; ++i) sh.finished[i] = 0;
    tc::prefetch_map(&maps.q);
    tc::prefetch_map(&maps.k);
    tc::prefetch_map(&maps.v);
    for (int i = 0; i < kItems; ++i) {
      tc::barrier_init(tc::smem_address(&sh.item_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.item_free[i]), C::kSoftmaxWarps + C::kCheckWarps + 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      tc::barrier_init(tc::smem_address(&sh.kv_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.kv_free[i]), 1 + C::kCheckWarps);
      tc::barrier_init(tc::smem_address(&sh.checked[i]), C::kCheckWarps);
    }
    for (int i = 0; i < 2; ++i) {
      tc::barrier_init(tc::smem_address(&sh.q_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.q_free[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.s_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.p_ready[i]), 4);
      tc::barrier_init(tc::smem_address(&sh.pv_done[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.o_free[i]), 4);
    }
    tc::barrier_init(tc::smem_address(&sh.last), 1);
    tc::barrier_init(tc::smem_address(&sh.answer), 1);
    tc::publish_shared();
  }
  wait_for_stream();  // (before tensor memory is taken, which the launch before may still need)
  if (warp == 0) tc::tmem_alloc(tc::smem_address(&sh.tmem), 512);
  sort_sequences(a, sh.sequences, C::NQ * tpt, C::kThreads);
  if (blockIdx.x == 0) flag_lengths(a, C::kThreads);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp < C::kSoftmaxWarps) {
    if constexpr (C::NQ == 2) tc::registers_up<kSoftmaxRegisters>();
    softmax_role<DP>(a, tpt, f, sh, tmem, out_vec32);
  } else {
    if constexpr (C::NQ == 2) tc::registers_down<kOtherRegisters>();
    if (warp == C::kSoftmaxWarps) {
      Finder finder{};
      Loads under{};
      if (!load_role<DP>(a, maps, tpt, sh, q_at, kv_at, finder, under)) end_loads<DP>(a, tpt, sh, finder, under);
    } else if (warp == C::kSoftmaxWarps + 1) {
      if (tc::elected()) {
        product_role<DP>(a, sh, q_at, kv_at, tmem);
        int unused = 0;
        tc::products_arrive(tc::smem_address(&sh.last));
        tc::barrier_wait(tc::smem_address(&sh.last), 0, &unused, tc::kEndCycles);
      }
      __syncwarp();
    } else {
      check_role<DP>(sh, tiles + C::NQ * C::kQueryBytes);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (sh.gave_up) {
    int done = sh.finished[0];
    for (int i = 1; i < C::kSoftmaxWarps; ++i) done = min(done, sh.finished[i]);
    for (int k = done; k < sh.claimed; ++k) spoil<uint16_t>(a, sh.item[k % kItems], tpt, C::NQ, tid, C::kThreads);
  }
  if (warp == 0) tc::tmem_free(tmem, 512);
}

// Boxes of 64 dims (zeros behind the last) of `heads` heads of `rows` rows.
bool rows_map(CUtensorMap* map, const void* at, int dim, int heads, int rows, int64_t head_stride, int64_t row_stride, int box_heads, int box_rows) {
  const tc::EncodeTiled encode = tc::encoder();
  if (!encode) return false;
  const cuuint64_t size[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[2] = {static_cast<cuuint64_t>(head_stride) * 2, static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)}, step[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(at), size, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
sv_status launch(const PromptView& a, cudaStream_t stream) {
  using C = Config<DP>;
  static FuncAttrCache attr;
  const auto kernel = prompt_tiles_kernel<DP>;
  if (!attr.ensure(reinterpret_cast<const void*>(kernel), C::kShared, false)) return SV_ERR_CUDA;
  const int tpt = kRows / a.group;
  Maps maps;
  if (!rows_map(&maps.q, a.q, a.dim, a.heads, a.total_new, a.q_head, a.q_row, a.group, tpt) ||
      !rows_map(&maps.k, a.k, a.dim, a.kv_heads, a.total_new, a.k_head, a.k_row, 1, kKeys) ||
      !rows_map(&maps.v, a.v, a.dim, a.kv_heads, a.total_new, a.v_head, a.v_row, 1, kKeys))
    return SV_ERR_UNSUPPORTED;
  const bool vec32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.out_row % 16 == 0 && a.out_head % 16 == 0;
  if (launch_early(kernel, dim3(prompt_blocks(a, C::NQ * tpt)), dim3(C::kThreads), C::kShared, stream, a, maps, tpt, a.scale * 1.44269504088896340736f,
                   static_cast<int>(vec32)) != cudaSuccess)
    return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace

bool prompt_takes_tiles(const PromptView& a, sv_dtype dtype) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  const int64_t strides = a.q_row | a.q_head | a.k_row | a.k_head | a.v_row | a.v_head;
  // (a tensor map holds strides of less than 2^40 bytes)
  return dtype == SV_BF16 && at % 16 == 0 && strides % 8 == 0 && strides < int64_t{1} << 39 && a.total_new > 0;
}

sv_status prompt_tiles(const PromptView& a, cudaStream_t stream) {
  return a.dim <= 64 ? launch<64>(a, stream) : a.dim <= 128 ? launch<128>(a, stream) : launch<256>(a, stream);
}

}  // namespace sv
