// Attention of many query rows for each kv head over the 8-bit cache: token
// trees, long chains, stretches of a prompt.
//
// 128 query rows at a time against tiles of 64 tokens on the 5th-generation
// tensor cores: S = Q K^T and O += P V.  Accumulators and the left sides are
// in tensor memory, where the weights P take the place of the scores they
// come from.  One block per SM, five roles:
//   1 warp plans: it walks the block's tiles and looks pages and scales up;
//   1 warp fetches codes, a box of 16 tokens of a page to a copy, three tiles
//     ahead of the widening (eight of up to 64 dims);
//   4 warps widen keys and values to fp16 (which holds them all), to where the
//     products read them, swizzled;
//   1 warp issues the products: S of tile t before P V of tile t - 2;
//   2 groups of 4 warps turn scores into weights, a row a thread, one group
//     the even tiles and the other the odd ones, each with its own running
//     maximum and its own O, which are joined where an item's part ends.
//     The maximum moves only when weights reach 2^7 times it (then O is
//     scaled anew), so that scores are read once and no maximum is taken.
// Both products are fp16.  A power of two for each row puts its largest query
// at 2^14 and more, so that a bf16 query keeps all its bits down to 2^-31 of
// the row's largest.  (8-bit scores, of queries as the sum of two e4m3 values
// and keys as they come, were 2% to 3% faster, 124 and 364 us, but rounded what
// lies below 2^-17 of it: one dim far above the others cost the others theirs.)
// Weights would not fit 8 bits either: a long even tail of a softmax lies below
// e4m3's range.
// Work is shared out as in sv_kv_schedule.cuh.
//
// 2000 tokens of two prompts behind 4096 cached ones, 32 heads of 128 dims: 375
// us, 780 TFLOP/s of useful work, bound by the step from scores to weights (two
// tiles of it under way at a time, 1.4 thousand cycles each) and what each step
// of a tile waits for the other.  64 trees of 32 nodes on up to 4096 tokens: 127
// us, 2.65 TB/s, a fifth of it spent at the ends of items.
#include "sv_kv_schedule.cuh"
#include "sv_tcgen05.cuh"

#include <type_traits>

namespace sv {

namespace {

constexpr int kRows = 128;
constexpr int kTileSteps = 4;
constexpr int kTokens = kStep * kTileSteps;
// Empty tiles ahead of an item: none, 5, 8 and 12 take 148, 131, 127 and 127 us for 64 trees of 32 nodes on contexts of up to
// 4096 tokens, 379, 374, 374 and 378 for 2000 tokens of two prompts behind 4096, 335, 208, 189 and 193 for 16 prompts of 836.
constexpr int kOpen = 8;
// weights: warps 0-7; widening: 8-11; products: 12; plan: 13; fetch: 14 (15 idle: registers move in fours of warps)
constexpr int kSoftmaxWarps = 8, kWidenWarps = 4;
constexpr int kWidenThreads = 32 * kWidenWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + kWidenWarps + 4);
constexpr int kSoftmaxRegisters = 176, kWidenRegisters = 96, kOtherRegisters = 64;
static_assert(kSoftmaxWarps * kSoftmaxRegisters + kWidenWarps * kWidenRegisters + 4 * kOtherRegisters <= 16 * 128,
              "registers of a block");
constexpr float kLift = 8.0f;  // weights are 2^8 times what they stand for: fp16 then keeps 2^-22 of a row's largest

constexpr int kMostCodeStages = 8;
constexpr int kValueStages = 6;  // tiles of widened values in shared memory,
constexpr int kScoreStages = 3;  // of widened keys, and of scores in tensor memory
constexpr int kLag = 2;          // tiles that scores are formed ahead of the sums over values

constexpr int kPiece = 80;       // 64 bytes of a row of queries, at a pitch free of bank conflicts

template <int DP> struct Tiles {
  // Tiles of codes in shared memory.  At 128 dims what it holds is better spent on widened values: 5 of codes and 4 of values, 4 and
  // 5, 3 and 6 take 130, 128 and 127 us for 64 trees of 32 nodes, 378, 375 and 375 for 2000 tokens of two prompts.
  static constexpr int kCodeStages = DP == 64 ? kMostCodeStages : 3;
  static constexpr int kCodeBytes = kTokens * DP;          // a tile's codes of keys (and of values) as they come,
  static constexpr int kTileBytes = kTokens * DP * 2;      // and in fp16,
  static constexpr int kBlockBytes = kTokens * 128;        // in blocks of 64 dims
  static constexpr int kOperands = (kValueStages + kScoreStages) * kTileBytes + kCodeStages * 2 * kCodeBytes + kSoftmaxWarps * 32 * kPiece;
  // 1 KB to find a 1024-byte boundary; more than half of an SM's shared memory keeps it to one block
  static constexpr int kShared = (kOperands > 118 * 1024 ? kOperands : 118 * 1024) + 1024;
  // tensor memory, in columns: two O, Q, three tiles of scores
  static constexpr int kO = 0, kQ = 2 * DP, kS = kQ + DP / 2;
  static constexpr int kColumns = 512;
  static constexpr int kPart = kRows * (DP + 2);  // floats of a part in the workspace
  static_assert(kPart * sizeof(float) % 32 == 0 && DP * sizeof(float) % 32 == 0, "parts are written 32 bytes at a time");
};
// Where the parts begin in the workspace, which callers align to 16 bytes: its size has room for rounding up.
constexpr size_t kPartAlign = 32;

constexpr int kPlans = 16;  // tiles that may be planned ahead
constexpr int kParts = 4;  // parts of items that may be
constexpr float kNoScale = -1000.0f;

// What the roles need of a tile.
struct TilePlan {
  int page[kTileSteps], slot[kTileSteps];  // where each step's codes lie
  int head;
  int token[kTileSteps];      // its first token
  int count[kTileSteps];      // tokens in sight, 0: nothing to fetch
  float k_scale[kTileSteps];
  float v_log2[kTileSteps];   // log2 of the values' scale, kNoScale for none
  int whole;                  // every row sees every token
};

// And of an item's part that the block works on.
struct Part {
  int b, h, ctx, row0;
  int r0, rows, i0, i1;       // rows of the item, their new tokens
  int tile0, count, tiles;    // first and number of the block's tiles, all of the item
  int join_last;              // the last block with a part of the item
};

struct Shared {
  CursorScratch cursor;
  uint64_t plan_full[kPlans], plan_free[kPlans], part_full[kParts], part_free[kParts];
  uint64_t codes_full[kMostCodeStages], codes_free[kMostCodeStages];
  uint64_t k_ready[kScoreStages], pv_ready[kValueStages], pv_done[kValueStages], s_full[kScoreStages], q_ready, last, both[4];
  float exchange[2][kRows][4];  // between the two threads of a row: maximum, sum, values' unit; the queries' largest
  TilePlan plan[kPlans];
  Part part[kParts];
  uint32_t tmem;
  int gave_up;
  int fetched;  // tiles that copies were issued for
  Cursor begin; // where the block's range begins
};

// Eight codes as fp16.
__device__ __forceinline__ uint4 widen(const uint2& c) {
  return make_uint4(e4m3x2_to_f16x2(c.x & 0xffffu), e4m3x2_to_f16x2(c.x >> 16), e4m3x2_to_f16x2(c.y & 0xffffu), e4m3x2_to_f16x2(c.y >> 16));
}

__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// Bits j of [from, to) for the 16 tokens from `base` on.
__device__ __forceinline__ uint32_t bits16(int base, int from, int to) {
  const int a = min(max(from - base, 0), 16), b = min(max(to - base, 0), 16);
  return ((1u << b) - 1u) & ~((1u << a) - 1u);
}

// Every lane waits (for the n-th phase of a barrier); the answer is the warp's.
__device__ __forceinline__ bool warp_wait(Shared& sh, uint64_t& bar, int n) {
  return __all_sync(0xffffffffu, tc::barrier_wait(tc::smem_address(&bar), static_cast<uint32_t>(n & 1), &sh.gave_up));
}
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::barrier_arrive(tc::smem_address(&bar));
}

// A block's tile that is never planned, in builds that test what happens when the other roles' waits run out.
#ifndef SV_LOST_TILE
#define SV_LOST_TILE -1
#endif

// ---- plans ----

// Eight tiles at a time, a lane to a step: page ids, then scales.
__device__ bool plan_role(const AttentionParams& a, Cursor c, Shared& sh) {
  const KvView& w = a.w;
  const int lane = threadIdx.x & 31, mine = lane / kTileSteps, step = lane % kTileSteps;
  const int page_mask = (1 << w.page_shift) - 1;
  int it = 0;
  for (int item = 0; c.at < c.end; ++item) {
    Part p;
    p.b = c.b;
    p.h = c.h;
    p.ctx = c.span.ctx;
    p.row0 = c.span.row0;
    p.r0 = c.rt * kRows;
    p.rows = min(kRows, c.span.n * a.group - p.r0);
    p.i0 = p.r0 / a.group;
    p.i1 = (p.r0 + p.rows - 1) / a.group;
    const ItemSteps steps = item_steps(a, c.span, p.i0, p.i1);
    p.tiles = max(1, (steps.steps + kTileSteps - 1) / kTileSteps);
    const int done = static_cast<int>(min(static_cast<long long>(p.tiles - c.tile), c.end - c.at));
    if (c.tile + done <= 0) break;  // the range ends in the item's empty tiles
    p.tile0 = max(c.tile, 0);
    p.count = c.tile + done - p.tile0;
    p.join_last = p.tile0 == 0 && p.count < p.tiles ? tile_owner(c.at - c.tile + p.tiles - 1, c.total, c.blocks) : 0;
    if (item >= kParts && !warp_wait(sh, sh.part_free[item % kParts], item / kParts - 1)) return false;
    if (lane == 0) sh.part[item % kParts] = p;
    warp_arrive(sh.part_full[item % kParts]);
    // tokens before `all` are in every row's past; `far` is the furthest position of a row
    const int all = a.parents ? p.ctx : p.ctx + p.i0 + 1, far = p.ctx + p.i1;
    for (int t0 = 0; t0 < p.count; t0 += 32 / kTileSteps) {
      const int s = (p.tile0 + t0 + mine) * kTileSteps + step;
      const bool live = t0 + mine < p.count && s < steps.steps;
      const int token = steps.token(s);
      int page = -1;
      if (live && sv_in(token >> w.page_shift, w.max_pages)) page = __ldg(w.c.page_table + p.b * w.table_stride + (token >> w.page_shift));
      const bool there = live && page >= 0 && page < w.num_pages;
      if (live && !there) kv_flag(w, p.b, SV_ROW_BAD_PAGE);
      float k_scale = 0.0f, v_scale = 0.0f;
      if (there) {
        k_scale = __ldg(w.c.k_scale + static_cast<int64_t>(page) * w.kv_heads + p.h);
        v_scale = __ldg(w.c.v_scale + static_cast<int64_t>(page) * w.kv_heads + p.h);
      }
      const bool full = there && token + kStep <= all &&
                        (a.window == 0 || far - token < a.window || token + kStep <= a.sinks);
      const unsigned fulls = __ballot_sync(0xffffffffu, full) >> (mine * kTileSteps) & ((1u << kTileSteps) - 1u);
      const uint32_t bits = __float_as_uint(v_scale);
      const float v_log2 = !(v_scale > 0.0f) ? kNoScale
                           : (bits & 0x7fffffu) == 0 && bits >= 0x00800000u ? static_cast<float>(static_cast<int>(bits >> 23) - 127)
                                                                            : log2f(v_scale);
      for (int i = 0; i < 32 / kTileSteps && t0 + i < p.count; ++i, ++it) {
        if (it == SV_LOST_TILE) return true;
        TilePlan& plan = sh.plan[it % kPlans];
        if (it >= kPlans && !warp_wait(sh, sh.plan_free[it % kPlans], it / kPlans - 1)) return false;
        if (mine == i) {
          plan.page[step] = page;
          plan.slot[step] = token & page_mask;
          plan.token[step] = token;
          plan.count[step] = there ? min(kStep, steps.end - token) : 0;
          plan.k_scale[step] = k_scale;
          plan.v_log2[step] = v_log2;
          if (step == 0) {
            plan.head = p.h;
            plan.whole = fulls == (1u << kTileSteps) - 1u;
          }
        }
        warp_arrive(sh.plan_full[it % kPlans]);
      }
    }
    next_item<kRows, kOpen>(a, c, done);
  }
  return true;
}

// ---- codes ----

// Two copies for each step that has tokens, a lane to a copy.
template <int DP>
__device__ bool fetch_role(const AttentionParams& a, const CUtensorMap* keys, const CUtensorMap* values, const int tiles, Shared& sh, uint32_t codes) {
  using T = Tiles<DP>;
  constexpr int kCodeStages = T::kCodeStages;
  const int lane = threadIdx.x & 31, step = lane % kTileSteps;
  const bool key = lane < kTileSteps;
  const CUtensorMap* map = key ? keys : values;
  const uint32_t to = codes + (key ? 0 : T::kCodeBytes) + step * (kStep * DP);
  for (int it = 0; it < tiles; ++it) {
    const TilePlan& plan = sh.plan[it % kPlans];
    const int stage = it % kCodeStages;
    if (!warp_wait(sh, sh.plan_full[it % kPlans], it / kPlans)) return false;
    const int slot = plan.slot[step], page = plan.page[step], head = plan.head;
    const bool live = lane < 2 * kTileSteps && plan.count[step] > 0 && kv_slot_in(a.w, slot, kStep) && sv_in(page, a.w.num_pages) &&
                      sv_in(head, a.w.kv_heads);
    const int copies = __popc(__ballot_sync(0xffffffffu, live));
    warp_arrive(sh.plan_free[it % kPlans]);
    if (it >= kCodeStages && !warp_wait(sh, sh.codes_free[stage], it / kCodeStages - 1)) return false;
    const uint32_t bar = tc::smem_address(&sh.codes_full[stage]);
    if (lane == 0) {
      tc::barrier_expect(bar, copies * (kStep * DP));
      sh.fetched = it + 1;
    }
    __syncwarp();
    if (live) tc::copy_box(to + stage * 2 * T::kCodeBytes, map, 0, slot, head, page, bar);
  }
  return true;
}

// A chunk of 16 codes becomes two of fp16, in rows of 64 dims, swizzled; lanes of the second block of dims, and those of odd
// tokens, do its halves the other way round (they use other banks then).  What is not a token in sight becomes 0, whatever its bytes.
template <int DP>
__device__ bool widen_role(const int tiles, Shared& sh, uint8_t* k_tiles, uint8_t* v_tiles, const uint8_t* codes) {
  using T = Tiles<DP>;
  constexpr int kCodeStages = T::kCodeStages;
  constexpr int kChunks = DP / 16;                        // of a token
  constexpr int kPer = kWidenThreads / kChunks;           // tokens of a pass, 16 or 32
  constexpr int NI = kTokens / kPer;                      // passes
  const int tid = threadIdx.x - 32 * kSoftmaxWarps;
  const int t0 = tid / kChunks, ch = tid % kChunks;
  const int turn = ((ch >> 2) ^ t0) & 1;
  const int to = (ch >> 2) * T::kBlockBytes + t0 * 128;
  const int half0 = to + (((2 * (ch & 3) + turn) ^ (t0 & 7)) << 4), half1 = to + (((2 * (ch & 3) + 1 - turn) ^ (t0 & 7)) << 4);
  uint2 c[NI][2];
  const auto load = [&](const uint8_t* from, unsigned seen) {
    from += t0 * DP + ch * 16;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool live = seen >> i & 1u;
      c[i][0] = live ? *reinterpret_cast<const uint2*>(from + i * kPer * DP + 8 * turn) : make_uint2(0, 0);
      c[i][1] = live ? *reinterpret_cast<const uint2*>(from + i * kPer * DP + 8 - 8 * turn) : make_uint2(0, 0);
    }
  };
  const auto store = [&](uint8_t* row) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      *reinterpret_cast<uint4*>(row + half0 + i * kPer * 128) = widen(c[i][0]);
      *reinterpret_cast<uint4*>(row + half1 + i * kPer * 128) = widen(c[i][1]);
    }
    tc::publish_shared();
  };
#pragma unroll 1
  for (int it = 0; it < tiles; ++it) {
    const int ks = it % kScoreStages, vs = it % kValueStages, stage = it % kCodeStages;
    const TilePlan& plan = sh.plan[it % kPlans];
    if (!warp_wait(sh, sh.plan_full[it % kPlans], it / kPlans) || !warp_wait(sh, sh.codes_full[stage], it / kCodeStages)) return false;
    unsigned seen = ~0u;  // bit i: the thread's token of pass i is in sight
    if (!plan.whole) {
      seen = 0;
#pragma unroll
      for (int i = 0; i < NI; ++i) seen |= (t0 % kStep < plan.count[(t0 + i * kPer) / kStep] ? 1u : 0u) << i;
    }
    warp_arrive(sh.plan_free[it % kPlans]);
    const uint8_t* from = codes + stage * 2 * T::kCodeBytes;
    load(from, seen);
    // (the scores of tile it - 3 have been formed, so its keys' place is free)
    if (it >= kScoreStages && !warp_wait(sh, sh.s_full[ks], it / kScoreStages - 1)) return false;
    store(k_tiles + ks * T::kTileBytes);
    warp_arrive(sh.k_ready[ks]);
    load(from + T::kCodeBytes, seen);
    warp_arrive(sh.codes_free[stage]);
    if (it >= kValueStages && !warp_wait(sh, sh.pv_done[vs], it / kValueStages - 1)) return false;
    store(v_tiles + vs * T::kTileBytes);
    warp_arrive(sh.pv_ready[vs]);
  }
  return true;
}

// ---- products ----

// One thread (elected of its warp): what it waits for delays the products, so it waits as little as it can.
template <int DP>
__device__ bool product_role(const int tiles, Shared& sh, uint32_t k_tiles, uint32_t v_tiles, uint32_t tmem) {
  using T = Tiles<DP>;
  constexpr uint32_t kScores = tc::product_kind(kTokens, false), kValues = tc::product_kind(DP, true);
  const auto wait = [&](uint64_t& bar, int n) {
    const bool ok = tc::barrier_wait(tc::smem_address(&bar), static_cast<uint32_t>(n & 1), &sh.gave_up);
    tc::fence_after();
    return ok;
  };
  const auto weigh = [&](int it, bool first) {  // O (+)= P V of tile it, its group's first of the part
    const int v = it % kValueStages;
    if (!wait(sh.pv_ready[v], it / kValueStages)) return false;
#pragma unroll
    for (int k = 0; k < kTokens / 16; ++k)
      tc::product_f16(tmem + T::kO + (it & 1) * DP, tmem + T::kS + it % kScoreStages * kTokens + k * 8,
                      tc::tile_descriptor(v_tiles + v * T::kTileBytes + k * 2048, T::kBlockBytes, 1024), kValues, !first || k > 0);
    tc::products_arrive(tc::smem_address(&sh.pv_done[v]));
    return true;
  };
  for (int it = 0, item = 0; it < tiles; ++item) {
    if (!wait(sh.part_full[item % kParts], item / kParts)) return false;
    const int count = sh.part[item % kParts].count;
    tc::barrier_arrive(tc::smem_address(&sh.part_free[item % kParts]));
    if (!wait(sh.q_ready, item)) return false;
    for (int t = 0; t < count; ++t, ++it) {
      const int s = it % kScoreStages;
      if (!wait(sh.k_ready[s], it / kScoreStages)) return false;
      // (these scores' place was tile it - 3's weights, whose products were issued before)
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)
        tc::product_f16(tmem + T::kS + s * kTokens, tmem + T::kQ + k * 8,
                        tc::tile_descriptor(k_tiles + s * T::kTileBytes + (k >> 2) * T::kBlockBytes + (k & 3) * 32, 16, 1024), kScores, k > 0);
      tc::products_arrive(tc::smem_address(&sh.s_full[s]));
      if (t >= kLag && !weigh(it - kLag, t - kLag < 2)) return false;
    }
    for (int n = min(count, kLag); n > 0; --n)
      if (!weigh(it - n, count - n < 2)) return false;
  }
  return true;
}

// ---- scores to weights, and results ----

// Which tokens of two of a tile's steps the thread's row sees.
__device__ __forceinline__ uint32_t seen_tokens(const AttentionParams& a, const TilePlan& plan, int step0, const int32_t* parents, int ctx,
                                                int token, int pos) {
  const int past = parents ? ctx : pos + 1;
  const int from = a.window ? max(0, pos - a.window + 1) : 0;
  uint32_t seen = 0;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (plan.count[step0 + i] <= 0) continue;
    const int base = plan.token[step0 + i];
    uint32_t b = bits16(base, from, past);
    if (a.window) b |= bits16(base, 0, min(a.sinks, past));
    if (parents && base + kStep > ctx)
      for (int u = token, back = 0; u >= 0; u = tree_parent(parents, u), ++back) {
        const int j = ctx + u - base;
        if (j >= 0 && j < kStep && (a.window == 0 || back < a.window || pos - back < a.sinks)) b |= 1u << j;
      }
    seen |= b << (16 * i);
  }
  __syncwarp();
  return seen;
}

// The largest of 16 scores (that are seen).
template <bool MASKED>
__device__ __forceinline__ float largest16(const uint32_t* x, uint32_t seen) {
  float v[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = MASKED && !(seen >> k & 1u) ? -CUDART_INF_F : __uint_as_float(x[k]);
#pragma unroll
  for (int n = 8; n > 0; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) v[k] = fmaxf(v[k], v[k + n]);
  return v[0];
}

// 32 scores to weights 2^(x f + c): packed into w, and their sums by steps.
template <bool MASKED>
__device__ __forceinline__ float2 weights32(const uint32_t (&x)[32], uint32_t seen, float f0, float f1, float c0, float c1, uint32_t* w) {
  float2 sums;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t f = tc::pair(h ? f1 : f0, h ? f1 : f0), c = tc::pair(h ? c1 : c0, h ? c1 : c0);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int n = 16 * h + 2 * k;
      float2 e = tc::unpair(tc::fma2(tc::pair(__uint_as_float(x[n]), __uint_as_float(x[n + 1])), f, c));
      e.x = ex2(e.x);
      e.y = ex2(e.y);
      if (MASKED) {
        e.x = seen >> n & 1u ? e.x : 0.0f;
        e.y = seen >> (n + 1) & 1u ? e.y : 0.0f;
      }
      sum[k & 1] = tc::add2(sum[k & 1], tc::pair(e.x, e.y));
      w[8 * h + k] = pack_f16x2(e.x, e.y);
    }
    const float2 s = tc::unpair(tc::add2(sum[0], sum[1]));
    (h ? sums.y : sums.x) = s.x + s.y;
  }
  return sums;
}

template <int DP>
__device__ bool softmax_role(const AttentionParams& a, const int tiles, Shared& sh, uint8_t* staging, uint32_t tmem, int g) {
  using T = Tiles<DP>;
  constexpr int kDims = DP / 2;  // a thread's share of a row of queries and results
  const int r = threadIdx.x & (kRows - 1), group = threadIdx.x / kRows, quarter = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t mine = tmem + (quarter << 21);  // the warp's 32 lanes
  const uint32_t own_o = mine + T::kO + group * DP;
  staging += (threadIdx.x >> 5) * 32 * kPiece;
  const auto wait = [&](uint64_t& bar, int n) {
    const bool ok = warp_wait(sh, bar, n);
    tc::fence_after();
    return ok;
  };
  const auto arrive = [&](uint64_t& bar) {
    tc::wait_stores();
    tc::fence_before();
    warp_arrive(bar);
  };
  // The row's two threads meet.
  int meetings = 0;
  const auto meet = [&]() {
    warp_arrive(sh.both[quarter]);
    return warp_wait(sh, sh.both[quarter], meetings++);
  };
  int it0 = 0;  // the part's first tile
  for (int item = 0; it0 < tiles; ++item) {
    if (!wait(sh.part_full[item % kParts], item / kParts)) return false;
    const Part& p = sh.part[item % kParts];
    const int32_t* parents = a.parents ? a.parents + p.row0 : nullptr;
    const int ctx = p.ctx, token = (p.r0 + min(r, p.rows - 1)) / a.group;
    // the row is the call's, and so is its place in q, out and lse
    const bool held = r < p.rows && kv_row_in(a.w, static_cast<int64_t>(p.row0) + token) && sv_in(g, kSMs);

    // the row's queries, scaled by a power of two
    float factor;
    {
      const int head = p.h * a.group + (p.r0 + min(r, p.rows - 1)) % a.group;
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + (static_cast<int64_t>(p.row0) + token) * a.q_row_stride +
                          head * a.q_head_stride + group * kDims;
      uint4 raw[kDims / 8];
      uint32_t top = 0;
      if (a.q_vec) {  // 8 rows' pieces of 64 bytes at a time: a lane that loads its own row alone touches a line for each 16 bytes
        const unsigned rows_held = __ballot_sync(0xffffffffu, held);
        uint64_t from[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) from[i] = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(q), 8 * i + (lane >> 2)) + 16 * (lane & 3);
#pragma unroll
        for (int i = 0; i < kDims / 8; ++i) {
          const bool live = rows_held >> (8 * (i & 3) + (lane >> 2)) & 1u && group * kDims + 32 * (i >> 2) + 8 * (lane & 3) < a.w.dim;
          raw[i] = live ? *reinterpret_cast<const uint4*>(from[i & 3] + 64 * (i >> 2)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < kDims / 32; ++n) {
#pragma unroll
          for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(staging + (8 * i + (lane >> 2)) * kPiece + 16 * (lane & 3)) = raw[4 * n + i];
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[4 * n + i] = *reinterpret_cast<const uint4*>(staging + lane * kPiece + 16 * i);
          __syncwarp();
        }
      } else {
#pragma unroll
        for (int i = 0; i < kDims / 8; ++i) {
          raw[i] = make_uint4(0, 0, 0, 0);
          if (held && group * kDims + i * 8 < a.w.dim) {
            const uint16_t* e = q + i * 8;
            raw[i] = make_uint4(__ldg(e) | __ldg(e + 1) << 16, __ldg(e + 2) | __ldg(e + 3) << 16,
                                __ldg(e + 4) | __ldg(e + 5) << 16, __ldg(e + 6) | __ldg(e + 7) << 16);
          }
        }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < kDims / 8; ++i) {
        top = __vmaxu2(__vmaxu2(top, raw[i].x & 0x7fff7fffu), raw[i].y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, raw[i].z & 0x7fff7fffu), raw[i].w & 0x7fff7fffu);
      }
      top = max(top >> 16, top & 0xffffu);
      // (read before the row's second meeting, so free for the next part; the other three before its next first one)
      sh.exchange[group][r][3] = __uint_as_float(top);
      if (!meet()) return false;
      top = max(top, __float_as_uint(sh.exchange[group ^ 1][r][3]));
      const int exponent = static_cast<int>(top >> 7);
      const int e = exponent == 255 || top == 0 ? 0 : min(120, 141 - exponent);
      // the largest becomes 2^14 .. 2^15, so that what is 2^-31 of it is kept whole; a negative factor goes into the queries, so
      // that larger products are larger scores
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (a.scale_log2 < 0.0f ? -1.0f : 1.0f);
      factor = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (exponent == 255) factor = CUDART_NAN_F;  // the row's scores are not numbers
#pragma unroll
      for (int n = 0; n < kDims / 32; ++n) {
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint4 c = raw[4 * n + (i >> 2)];
          const uint32_t two = (i & 3) == 0 ? c.x : (i & 3) == 1 ? c.y : (i & 3) == 2 ? c.z : c.w;
          h[i] = pack_f16x2(__uint_as_float(two << 16) * up, __uint_as_float(two & 0xffff0000u) * up);
        }
        tc::tmem_store(mine + T::kQ + group * (kDims / 2) + 16 * n, h);
      }
      arrive(sh.q_ready);
    }
    int pos = ctx + token;
    if (parents) {
      int depth = 0;
      for (int u = tree_parent(parents, token); u >= 0; u = tree_parent(parents, u)) ++depth;
      pos = ctx + depth;
      __syncwarp();
    }

    // m: the row's maximum so far (base 2), l: its sum of weights.  v_ref: m + v_ref is the largest sum so far of a score and
    // the log2 of its page's V scale; weights are multiplied by 2^(that log2 - v_ref), whatever larger scales carry no weight.
    float m = -CUDART_INF_F, l = 0.0f, v_ref = 0.0f;
    const int end = it0 + p.count;
    int it = it0 + ((it0 & 1) != group);
    const int begin = it;
    for (; it < end; it += 2) {
      const TilePlan& plan = sh.plan[it % kPlans];
      const int stage = it % kScoreStages;
      const uint32_t scores = mine + T::kS + stage * kTokens;
      if (!wait(sh.plan_full[it % kPlans], it / kPlans) || !wait(sh.s_full[stage], it / kScoreStages)) return false;
      // O is multiplied by `fix`, a power of two (where scales of V are)
      const auto rescale = [&](float fix) {
        if (it == begin) return true;
        if (!wait(sh.pv_done[(it - 2) % kValueStages], (it - 2) / kValueStages)) return false;
        uint32_t o[16];
#pragma unroll 1
        for (int i = 0; i < DP; i += 16) {
          tc::tmem_load16(own_o + i, o);
          tc::wait_loads(o);
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * fix);
          tc::tmem_store(own_o + i, o);
        }
        tc::wait_stores();  // a second change in the same tile loads them again
        return true;
      };
      const auto tile = [&](auto masked) {
        constexpr bool M = decltype(masked)::value;
        uint32_t seen0 = 0, seen1 = 0;
        if (M) {
          seen0 = seen_tokens(a, plan, 0, parents, ctx, token, pos);
          seen1 = seen_tokens(a, plan, 2, parents, ctx, token, pos);
        }
        const float* k = plan.k_scale;
        const float* v = plan.v_log2;
        // against the maximum so far, unless there is none; raised, and gone over again, where weights get too large.  Rows do
        // not depend on each other: one that needs nothing keeps its bits.
        bool mine = m == -CUDART_INF_F;
        bool raise = __any_sync(0xffffffffu, mine);
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          uint32_t x0[32], x1[32];
          if (__builtin_expect(raise, 0)) {
            tc::tmem_load32(scores, x0);
            tc::tmem_load32(scores + 32, x1);
            tc::wait_loads(x0);
            tc::wait_loads(x1);
            float top = -CUDART_INF_F, most = m + v_ref;  // of scores, and with their V scales
#pragma unroll
            for (int i = 0; i < kTileSteps; ++i) {  // whole: what is scaled anew is scaled exactly (fmaxf leaves out what is not a number)
              const float t = ceilf(largest16<M>(i < 2 ? &x0[16 * i] : &x1[16 * i - 32], (i < 2 ? seen0 : seen1) >> (16 * (i & 1))) * (factor * k[i]));
              top = fmaxf(top, t);
              most = fmaxf(most, t + v[i]);
            }
            top = fmaxf(m, top);
            float o_fix = 1.0f;
            if (mine && top > -CUDART_INF_F) {
              o_fix = ex2(m + v_ref - most);
              l *= ex2(m - top);
              m = top;
              v_ref = most - top;
            }
            if (!rescale(o_fix)) return false;
          }
          tc::tmem_load32(scores, x0);
          tc::tmem_load32(scores + 32, x1);
          // in units of their values' scales
          const float base = kLift - (m == -CUDART_INF_F ? 0.0f : m);
          float u0 = fmaxf(v[0] - v_ref, -100.0f), u1 = fmaxf(v[1] - v_ref, -100.0f);
          uint32_t w0[16], w1[16];
          tc::wait_loads(x0);
          float2 sums = weights32<M>(x0, seen0, factor * k[0], factor * k[1], base + u0, base + u1, w0);
          float most = fmaxf(sums.x, sums.y), sum = sums.x * ex2(-u0) + sums.y * ex2(-u1);
          u0 = fmaxf(v[2] - v_ref, -100.0f);
          u1 = fmaxf(v[3] - v_ref, -100.0f);
          tc::wait_loads(x1);
          sums = weights32<M>(x1, seen1, factor * k[2], factor * k[3], base + u0, base + u1, w1);
          most = fmaxf(most, fmaxf(sums.x, sums.y));
          sum += sums.x * ex2(-u0) + sums.y * ex2(-u1);
          mine = most > 32768.0f;
          raise = pass < 2 && __any_sync(0xffffffffu, mine);  // (the first pass may be for other rows; a raised row has sums below)
          if (!raise) {
            l += sum;
            tc::tmem_store(scores, w0);
            tc::tmem_store(scores + 16, w1);
            return true;
          }
        }
      };
      if (!(__builtin_expect(plan.whole, 1) ? tile(std::false_type{}) : tile(std::true_type{}))) return false;
      arrive(sh.pv_ready[it % kValueStages]);
      warp_arrive(sh.plan_free[it % kPlans]);
    }

    // The part's result: both threads of a row know both halves' sums, and each joins half of the dims.
    float* given = sh.exchange[group][r];
    given[0] = m;
    given[1] = l;
    given[2] = v_ref;
    if (!meet()) return false;
    const float* theirs = sh.exchange[group ^ 1][r];
    const float their_m = theirs[0], their_l = theirs[1], their_v = theirs[2];
    // masks: what a group without a tile of the part has in O is of another
    const uint32_t own = begin < end ? ~0u : 0u, other = p.count > 1 || !own ? ~0u : 0u;
    // the last tiles' products: all before them are done then
    if (!wait(sh.pv_done[(end - 1) % kValueStages], (end - 1) / kValueStages)) return false;
    const float top = fmaxf(m, their_m);
    const float lift = 1.0f / 256.0f;
    // (a group that saw nothing has sums of 0, or sums that are not numbers, which stay)
    const float fix = m == -CUDART_INF_F ? 1.0f : ex2(m - top), their_fix = their_m == -CUDART_INF_F ? 1.0f : ex2(their_m - top);
    const float total = (l * fix + their_l * their_fix) * lift;
    const bool complete = p.count == p.tiles;
    const float inv = !complete ? lift : total == 0.0f ? 0.0f : lift / total;
    const float scale = own ? fix * ex2(v_ref) * inv : 0.0f, their_scale = other ? their_fix * ex2(their_v) * inv : 0.0f;
    const int head = p.h * a.group + (p.r0 + min(r, p.rows - 1)) % a.group;
    const int64_t out_row = static_cast<int64_t>(p.row0) + token;
    uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * a.out_row_stride + head * a.out_head_stride;
    float* part = a.parts + (2 * static_cast<int64_t>(g) + (p.tile0 == 0 ? 1 : 0)) * T::kPart;
#pragma unroll 1
    for (int d = group * kDims; d < (group + 1) * kDims; d += 16) {  // (short: code that runs once a part is fetched anew)
      uint32_t x[16], y[16];
      tc::tmem_load16(own_o + d, x);
      tc::tmem_load16(mine + T::kO + (group ^ 1) * DP + d, y);
      tc::wait_loads(x);
      tc::wait_loads(y);
#pragma unroll
      for (int k = 0; k < 16; ++k)
        x[k] = __float_as_uint(fmaf(__uint_as_float(x[k] & own), scale, __uint_as_float(y[k] & other) * their_scale));
      if (held && !complete) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t o[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) o[n] = x[8 * k + n];
          tc::store_32(part + r * DP + d + 8 * k, o);
        }
      } else if (held && d < a.w.dim) {
        uint32_t o[8];
#pragma unroll
        for (int n = 0; n < 8; ++n) o[n] = floats_to_bf16x2(__uint_as_float(x[2 * n]), __uint_as_float(x[2 * n + 1]));
        if (a.out_vec32) {
          tc::store_32(out + d, o);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            out[d + 2 * n] = static_cast<uint16_t>(o[n]);
            out[d + 2 * n + 1] = static_cast<uint16_t>(o[n] >> 16);
          }
        }
      }
      __syncwarp();
    }
    if (group == 0 && held) {
      if (!complete)
        *reinterpret_cast<float2*>(part + kRows * DP + 2 * r) = make_float2(top, total);
      else if (a.lse)
        a.lse[out_row * a.heads + head] = row_lse(top, total);
    }
    if (!complete && p.tile0 == 0 && threadIdx.x == 0) a.joins[g] = JoinRecord{p.row0, p.r0, p.rows, p.h, p.join_last};
    warp_arrive(sh.part_free[item % kParts]);
    it0 = end;
  }
  return true;
}

// A wait ran out, so the block's results are not valid: every sequence that it had a part of is flagged, and its rows become
// NaN, those of whole items here, those of items in parts where the parts are joined.  By the warps that hand results over.
template <int DP>
__device__ __noinline__ void spoil(const AttentionParams& a, Cursor c, int g) {
  using T = Tiles<DP>;
  constexpr int kMine = 32 * kSoftmaxWarps;
  while (c.at < c.end) {
    const int r0 = c.rt * kRows, rows = min(kRows, c.span.n * a.group - r0);
    const int tiles = item_tiles<kRows, kTileSteps>(a, c.span, c.rt);
    const int done = static_cast<int>(min(static_cast<long long>(tiles - c.tile), c.end - c.at));
    if (c.tile + done <= 0) return;  // the range ends in the item's empty tiles
    const bool begins = c.tile <= 0, complete = begins && c.tile + done == tiles;
    if (threadIdx.x == 0) kv_flag(a.w, c.b, SV_ROW_TIMEOUT);
    float* part = a.parts + (2 * static_cast<int64_t>(g) + (begins ? 1 : 0)) * T::kPart;
    for (int r = threadIdx.x; r < rows; r += kMine) {
      if (!complete) {
        *reinterpret_cast<float2*>(part + kRows * DP + 2 * r) = make_float2(0.0f, CUDART_NAN_F);
        continue;
      }
      const int64_t row = static_cast<int64_t>(c.span.row0) + (r0 + r) / a.group;
      const int head = c.h * a.group + (r0 + r) % a.group;
      uint16_t* out = static_cast<uint16_t*>(a.out) + row * a.out_row_stride + head * a.out_head_stride;
      for (int d = 0; d < a.w.dim; ++d) out[d] = 0x7fff;
      if (a.lse) a.lse[row * a.heads + head] = CUDART_NAN_F;
    }
    if (!complete && begins && threadIdx.x == 0)
      a.joins[g] = JoinRecord{c.span.row0, r0, rows, c.h, tile_owner(c.at - c.tile + tiles - 1, c.total, c.blocks)};
    next_item<kRows, kOpen>(a, c, done);
  }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tiles_kernel(AttentionParams a, const __grid_constant__ CUtensorMap keys,
                                                                              const __grid_constant__ CUtensorMap values) {
  using T = Tiles<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t at = tc::smem_address(raw);
  uint8_t* tiles = raw + ((at + 1023u & ~1023u) - at);
  uint8_t* v_tiles = tiles;
  uint8_t* k_tiles = v_tiles + kValueStages * T::kTileBytes;
  uint8_t* codes = k_tiles + kScoreStages * T::kTileBytes;
  constexpr int kCodeStages = T::kCodeStages;
  const int warp = threadIdx.x >> 5, g = blockIdx.x;
  wait_for_stream();
  flag_sequences(a, g, gridDim.x, kThreads);
  if (threadIdx.x == 0) {
    a.joins[g].rows = 0;
    sh.gave_up = 0;
    sh.fetched = 0;
    tc::prefetch_map(&keys);
    tc::prefetch_map(&values);
    for (int i = 0; i < kCodeStages; ++i) {
      tc::barrier_init(tc::smem_address(&sh.codes_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.codes_free[i]), kWidenWarps);
    }
    for (int i = 0; i < kValueStages; ++i) {
      tc::barrier_init(tc::smem_address(&sh.pv_ready[i]), kWidenWarps + kSoftmaxWarps / 2);
      tc::barrier_init(tc::smem_address(&sh.pv_done[i]), 1);
    }
    for (int i = 0; i < kScoreStages; ++i) {
      tc::barrier_init(tc::smem_address(&sh.k_ready[i]), kWidenWarps);
      tc::barrier_init(tc::smem_address(&sh.s_full[i]), 1);
    }
    for (int i = 0; i < kPlans; ++i) {
      tc::barrier_init(tc::smem_address(&sh.plan_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.plan_free[i]), kWidenWarps + kSoftmaxWarps / 2 + 1);
    }
    for (int i = 0; i < kParts; ++i) {
      tc::barrier_init(tc::smem_address(&sh.part_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.part_free[i]), kSoftmaxWarps + 1);
    }
    for (int i = 0; i < 4; ++i) tc::barrier_init(tc::smem_address(&sh.both[i]), 2);
    tc::barrier_init(tc::smem_address(&sh.q_ready), kSoftmaxWarps);
    tc::barrier_init(tc::smem_address(&sh.last), 1);
    tc::publish_shared();
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_address(&sh.tmem), T::kColumns);
  const Cursor c = find_cursor<kThreads, kRows, kTileSteps, kOpen>(a, g, gridDim.x, sh.cursor);
  if (threadIdx.x == 0) sh.begin = c;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  const int tiles_here = static_cast<int>(full_tiles<kRows, kTileSteps, kOpen>(a, c));  // 2^31 tiles would take half an hour
  if (warp < kSoftmaxWarps) {
    tc::registers_up<kSoftmaxRegisters>();
    if (!tc::all_of<1, 32 * kSoftmaxWarps>(softmax_role<DP>(a, tiles_here, sh, codes + kCodeStages * 2 * T::kCodeBytes, tmem, g)))
      spoil<DP>(a, sh.begin, g);
  } else if (warp < kSoftmaxWarps + kWidenWarps) {
    tc::registers_down<kWidenRegisters>();
    widen_role<DP>(tiles_here, sh, k_tiles, v_tiles, codes);
  } else {
    tc::registers_down<kOtherRegisters>();
    if (warp == kSoftmaxWarps + kWidenWarps) {
      if (tc::elected()) {
        product_role<DP>(tiles_here, sh, tc::smem_address(k_tiles), tc::smem_address(v_tiles), tmem);
        // products in flight end before the memory that they use is given up
        int unused = 0;
        tc::products_arrive(tc::smem_address(&sh.last));
        tc::barrier_wait(tc::smem_address(&sh.last), 0, &unused, tc::kEndCycles);
      }
      __syncwarp();
    } else if (warp == kSoftmaxWarps + kWidenWarps + 1) {
      plan_role(a, c, sh);
    } else if (warp == kSoftmaxWarps + kWidenWarps + 2) {
      fetch_role<DP>(a, &keys, &values, tiles_here, sh, tc::smem_address(codes));
      // and copies in flight: the last of each stage, which no other role may have waited for
      int unused = 0;
      for (int it = max(0, sh.fetched - kCodeStages); it < sh.fetched; ++it)
        tc::barrier_wait(tc::smem_address(&sh.codes_full[it % kCodeStages]), it / kCodeStages & 1, &unused, tc::kEndCycles);
      __syncwarp();
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::tmem_free(tmem, T::kColumns);
}

// The driver's encoder of tensor maps, looked up through the runtime (the library does not link the driver).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encoder() {
  static const EncodeTiled found = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult how;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &how) != cudaSuccess ||
        how != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return found;
}

// Boxes of `width` dims (zeros behind the last) of 16 tokens of one head and page.
bool cache_map(CUtensorMap* map, const sv_kv_desc& d, const uint8_t* cache, int width) {
  const EncodeTiled encode = encoder();
  if (!encode) return false;
  const cuuint64_t size[4] = {static_cast<cuuint64_t>(d.head_dim), static_cast<cuuint64_t>(d.page_size),
                              static_cast<cuuint64_t>(d.kv_heads), static_cast<cuuint64_t>(d.num_pages)};
  const cuuint64_t stride[3] = {static_cast<cuuint64_t>(d.token_stride), static_cast<cuuint64_t>(d.head_stride),
                                static_cast<cuuint64_t>(d.page_stride)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(width), kStep, 1, 1}, step[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(cache), size, stride, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP>
sv_status launch(AttentionParams a, const sv_kv_attention_desc& d, void* workspace, cudaStream_t stream) {
  using T = Tiles<DP>;
  static FuncAttrCache attr;
  const auto kernel = kv_attention_tiles_kernel<DP>;
  if (!attr.ensure(reinterpret_cast<const void*>(kernel), T::kShared, false)) return SV_ERR_CUDA;
  const int64_t row_tiles = (static_cast<int64_t>(d.max_new) * a.group + kRows - 1) / kRows;
  const int64_t tiles = (static_cast<int64_t>(d.kv.max_pages) * d.kv.page_size + kTokens - 1) / kTokens;
  const int blocks = schedule_blocks(row_tiles * d.kv.batch * d.kv.kv_heads, tiles + kOpen, kSMs);
  a.parts = reinterpret_cast<float*>(align_up(reinterpret_cast<uintptr_t>(workspace), kPartAlign));
  a.joins = reinterpret_cast<JoinRecord*>(a.parts + 2 * static_cast<int64_t>(kSMs) * T::kPart);
  CUtensorMap keys, values;
  if (!cache_map(&keys, d.kv, a.w.c.k, DP) || !cache_map(&values, d.kv, a.w.c.v, DP))
    return SV_ERR_UNSUPPORTED;
  if (launch_early(kernel, dim3(blocks), dim3(kThreads), T::kShared, stream, a, keys, values) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  if (blocks == 1 || tiles == 1) return SV_OK;  // no item has parts
  if (launch_join<uint16_t, DP, kRows>(a, blocks, stream) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace

// More rows of a kv head than the other kernel's two tiles of 16.  Rows are
// padded to 128 here, which costs more than it gives up to 32 of them: chains of
// 8 (32 rows) on contexts of up to 32768 tokens take 171 us here and 155 there at
// 128 dims, 163 and 101 at 64.  From 33 on the other kernel reads the cache
// twice: chains of 12 (48 rows) take 173 us here and 279 there.
bool kv_attention_takes_tiles(const sv_kv_attention_desc& d) {
  return d.dtype == SV_BF16 && d.kv.head_dim <= 128 &&
         static_cast<int64_t>(d.max_new) * (d.heads / d.kv.kv_heads) > 32;
}

size_t kv_attention_tiles_workspace(const sv_kv_attention_desc& d) {
  const size_t part = d.kv.head_dim <= 64 ? Tiles<64>::kPart : Tiles<128>::kPart;
  return align_up(kPartAlign + kSMs * (2 * part * sizeof(float) + sizeof(JoinRecord)), 256);
}

sv_status kv_attention_tiles(AttentionParams a, const sv_kv_attention_desc& d, void* workspace, cudaStream_t stream) {
  return d.kv.head_dim <= 64 ? launch<64>(a, d, workspace, stream) : launch<128>(a, d, workspace, stream);
}

}  // namespace sv
