// Attention of many query rows for each kv head over the 8-bit cache: token
// trees, long chains, stretches of a prompt.
//
// 128 query rows at a time against tiles of 128 tokens on the 5th-generation
// tensor cores: S = Q K^T and O += P V, accumulators in tensor memory.  The
// left sides (Q, and the weights P, which take the place of the scores they
// come from) are in tensor memory too, so that only K and V are read from
// shared memory.  One block per SM, four roles:
//   1 warp plans: it walks the block's tiles and looks pages and scales up;
//   8 warps load codes three tiles ahead and lay them out for the products:
//     keys as they are, values widened to fp16 (which holds them all);
//   1 warp issues the products: S of tile t before P V of tile t - 1;
//   4 warps turn scores into weights, a row a thread, with a running maximum
//     that moves only when it is exceeded by 2^7 (then O is scaled anew).
// S is formed in 8 bits without loss: a bf16 query is the sum of two e4m3
// values (4 significant bits each, of 8; what lies below 2^-17 of the row's
// largest is rounded), so S is two products of queries with the codes
// themselves.  Weights would need more: a long even tail of a softmax lies
// below e4m3's range, so P V is fp16.
// Work is shared out as in sv_kv_schedule.cuh.
#include "sv_kv_schedule.cuh"
#include "sv_tcgen05.cuh"

#include <type_traits>

namespace sv {

namespace {

constexpr int kRows = 128;
constexpr int kTileSteps = 8;
constexpr int kTokens = kStep * kTileSteps;
// weights: warps 0-3; loads: 4-11; products: 12; plan: 13 (14, 15 idle: registers move in fours of warps)
constexpr int kSoftmaxWarps = 4, kLoadWarps = 8;
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kThreads = 32 * (kSoftmaxWarps + kLoadWarps + 4);
constexpr int kSoftmaxRegisters = 216, kLoadRegisters = 96, kProductRegisters = 96;
static_assert(4 * kSoftmaxRegisters + 8 * kLoadRegisters + 4 * kProductRegisters <= 16 * 128, "registers of a block");
constexpr float kLift = 8.0f;  // weights are 2^8 times what they stand for: fp16 then keeps 2^-22 of the largest

constexpr int kCodeStages = 4;

template <int DP> struct Tiles {
  static constexpr int kKeyBytes = kTokens * 128;          // a tile's keys: rows of 128 bytes (DP = 64 leaves half)
  static constexpr int kCodeBytes = kTokens * DP;          // its values' codes as they come,
  static constexpr int kValueBytes = kTokens * DP * 2;     // and in fp16,
  static constexpr int kBlockBytes = kTokens * 128;        // in blocks of 64 dims
  static constexpr int kOperands = 2 * kValueBytes + kCodeStages * (kKeyBytes + kCodeBytes);
  // 1 KB to find a 1024-byte boundary; more than half of an SM's shared memory keeps it to one block
  static constexpr int kShared = (kOperands > 118 * 1024 ? kOperands : 118 * 1024) + 1024;
  // tensor memory, in columns: O, Q, two tiles of scores
  static constexpr int kO = 0, kQ = DP, kS = DP + DP / 2;
  static constexpr int kColumns = 512;
  static constexpr int kPart = kRows * (DP + 2);
};

constexpr int kPlans = 8;  // tiles that may be planned ahead
constexpr int kParts = 4;  // parts of items that may be
constexpr float kNoScale = -1000.0f;

// What the roles need of a tile.
struct TilePlan {
  int64_t base[kTileSteps];   // of each step's codes, or -1
  int token[kTileSteps];      // its first token
  int count[kTileSteps];      // tokens in sight
  float k_scale[kTileSteps];
  float v_log2[kTileSteps];   // log2 of the values' scale, kNoScale for none
  int whole;                  // every row sees every token
  int first, last;            // of its part
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
  uint64_t k_full[kCodeStages], v_full[2], s_full[2], p_ready[2], pv_done[2], q_ready, last;
  TilePlan plan[kPlans];
  Part part[kParts];
  uint32_t tmem;
  int gave_up;
};

// 16 codes as fp16: 32 bytes.
__device__ __forceinline__ void widen(const uint4& c, uint4& lo, uint4& hi) {
  lo = make_uint4(e4m3x2_to_f16x2(c.x & 0xffffu), e4m3x2_to_f16x2(c.x >> 16), e4m3x2_to_f16x2(c.y & 0xffffu), e4m3x2_to_f16x2(c.y >> 16));
  hi = make_uint4(e4m3x2_to_f16x2(c.z & 0xffffu), e4m3x2_to_f16x2(c.z >> 16), e4m3x2_to_f16x2(c.w & 0xffffu), e4m3x2_to_f16x2(c.w >> 16));
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
__device__ __forceinline__ bool warp_wait(Shared& sh, uint64_t& bar, long long n) {
  return __all_sync(0xffffffffu, tc::barrier_wait(tc::smem_address(&bar), static_cast<uint32_t>(n & 1), &sh.gave_up));
}
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::barrier_arrive(tc::smem_address(&bar));
}

// ---- plans ----

// Four tiles at a time, a lane to a step: page ids, then scales.
__device__ bool plan_role(const AttentionParams& a, Cursor c, Shared& sh) {
  const KvView& w = a.w;
  const int lane = threadIdx.x & 31, mine = lane / kTileSteps, step = lane % kTileSteps;
  const int page_mask = (1 << w.page_shift) - 1;
  long long it = 0;
  for (long long item = 0; c.at < c.end; ++item) {
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
    p.tile0 = c.tile;
    p.count = static_cast<int>(min(static_cast<long long>(p.tiles - c.tile), c.end - c.at));
    p.join_last = p.tile0 == 0 && p.count < p.tiles ? tile_owner(c.at + p.tiles - 1, c.total, c.blocks) : 0;
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
      const unsigned fulls = __ballot_sync(0xffffffffu, full) >> (mine * kTileSteps) & 0xffu;
      const uint32_t bits = __float_as_uint(v_scale);
      const float v_log2 = !(v_scale > 0.0f) ? kNoScale
                           : (bits & 0x7fffffu) == 0 && bits >= 0x00800000u ? static_cast<float>(static_cast<int>(bits >> 23) - 127)
                                                                            : log2f(v_scale);
      for (int i = 0; i < 32 / kTileSteps && t0 + i < p.count; ++i, ++it) {
        TilePlan& plan = sh.plan[it % kPlans];
        if (it >= kPlans && !warp_wait(sh, sh.plan_free[it % kPlans], it / kPlans - 1)) return false;
        if (mine == i) {
          plan.base[step] = there ? kv_offset(w, page, p.h, token & page_mask) : -1;
          plan.token[step] = token;
          plan.count[step] = there ? min(kStep, steps.end - token) : 0;
          plan.k_scale[step] = k_scale;
          plan.v_log2[step] = v_log2;
          if (step == 0) {
            plan.whole = fulls == 0xffu;
            plan.first = t0 + i == 0;
            plan.last = t0 + i + 1 == p.count;
          }
        }
        warp_arrive(sh.plan_full[it % kPlans]);
      }
    }
    next_item<kRows>(a, c, p.count);
  }
  return true;
}

// ---- loading ----

template <int DP>
__device__ bool load_role(const AttentionParams& a, const long long tiles, Shared& sh, uint8_t* k_tiles, uint8_t* v_tiles,
                          uint8_t* codes) {
  using T = Tiles<DP>;
  constexpr int kChunks = DP / 16;                        // of a token
  constexpr int kPer = kLoadThreads / kChunks;            // tokens of a pass
  constexpr int NI = kTokens / kPer;                      // passes
  const KvView& w = a.w;
  const int tid = threadIdx.x - 32 * kSoftmaxWarps;
  const int t0 = tid / kChunks, ch = tid % kChunks;
  const bool in_dim = ch * 16 < w.dim;
  const int64_t within = (t0 % kStep) * w.token_stride + ch * 16;  // kPer is a multiple of a step
  // Asks for a tile's codes.  Keys go straight to where the product reads them (kPer is a multiple of 8: a thread's
  // rows are swizzled alike); a thread's value codes lie side by side, only it reads them again.
  const uint32_t key_at = tc::smem_address(k_tiles) + t0 * 128 + ((ch ^ (t0 & 7)) << 4);
  uint8_t* const mine = codes + tid * 16;
  const uint32_t code_at = tc::smem_address(mine);
  const auto ask = [&](long long it) {
    const TilePlan& plan = sh.plan[it % kPlans];
    if (!warp_wait(sh, sh.plan_full[it % kPlans], it / kPlans)) return false;
    const uint32_t stage = static_cast<uint32_t>(it % kCodeStages);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int s = (t0 + i * kPer) / kStep;
      const bool live = t0 % kStep < plan.count[s] && in_dim;
      const int64_t from = live ? plan.base[s] + within : 0;
      const int size = live ? 16 : 0;  // zeros for the rest
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(key_at + stage * T::kKeyBytes + i * kPer * 128),
                   "l"(w.c.k + from), "r"(size) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(code_at + stage * T::kCodeBytes + i * kLoadThreads * 16),
                   "l"(w.c.v + from), "r"(size) : "memory");
    }
    warp_arrive(sh.plan_free[it % kPlans]);
    return true;
  };
  // A chunk of values becomes two of fp16, in rows of 64 dims, swizzled; lanes of the second block of dims write theirs
  // the other way round (other banks).
  const int turn = ch >> 2 & 1;
  const int to = (ch >> 2) * T::kBlockBytes + t0 * 128;
  const int half0 = (2 * (ch & 3) + turn) ^ (t0 & 7), half1 = (2 * (ch & 3) + 1 - turn) ^ (t0 & 7);
  for (int i = 0; i < kCodeStages - 1; ++i) {
    if (i < tiles && !ask(i)) return false;
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  bool ok = true;
#pragma unroll 1
  for (long long it = 0; ok && it < tiles; ++it) {
    const int st = it & 1;
    asm volatile("cp.async.wait_group %0;" ::"n"(kCodeStages - 2) : "memory");
    tc::publish_shared();
    warp_arrive(sh.k_full[it % kCodeStages]);
    ok = it < 2 || warp_wait(sh, sh.pv_done[st], (it >> 1) - 1);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      uint4 lo, hi;
      widen(*reinterpret_cast<const uint4*>(mine + (it % kCodeStages) * T::kCodeBytes + i * kLoadThreads * 16), lo, hi);
      uint8_t* row = v_tiles + st * T::kValueBytes + to + i * kPer * 128;
      *reinterpret_cast<uint4*>(row + (half0 << 4)) = turn ? hi : lo;
      *reinterpret_cast<uint4*>(row + (half1 << 4)) = turn ? lo : hi;
    }
    tc::publish_shared();
    warp_arrive(sh.v_full[st]);
    // the next tile to ask for takes the stage of tile it - 1, whose keys the product must have read
    if (ok && it + kCodeStages - 1 < tiles)
      ok = (it == 0 || warp_wait(sh, sh.s_full[st ^ 1], (it - 1) >> 1)) && ask(it + kCodeStages - 1);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  return ok;
}

// ---- products ----

template <int DP>
__device__ bool product_role(const long long tiles, Shared& sh, uint32_t k_tiles, uint32_t v_tiles, uint32_t tmem) {
  using T = Tiles<DP>;
  constexpr uint32_t kScores = tc::product_kind(kTokens, false), kValues = tc::product_kind(DP, true);
  const auto wait = [&](uint64_t& bar, long long n) {
    const bool ok = warp_wait(sh, bar, n);
    tc::fence_after();
    return ok;
  };
  const auto weigh = [&](long long it, bool first) {  // O (+)= P V of tile it
    const int st = it & 1;
    if (!wait(sh.v_full[st], it >> 1) || !wait(sh.p_ready[st], it >> 1)) return false;
    if (tc::elected()) {
#pragma unroll
      for (int k = 0; k < kTokens / 16; ++k)
        tc::product_f16(tmem + T::kO, tmem + T::kS + st * kTokens + k * 8,
                        tc::tile_descriptor(v_tiles + st * T::kValueBytes + k * 2048, T::kBlockBytes, 1024), kValues, !first || k > 0);
      tc::products_arrive(tc::smem_address(&sh.pv_done[st]));
    }
    __syncwarp();
    return true;
  };
  bool first_before = false;  // the last tile was its part's first
  long long item = 0;
  for (long long it = 0; it < tiles; ++it) {
    const int st = it & 1;
    if (!wait(sh.plan_full[it % kPlans], it / kPlans)) return false;
    const bool first = sh.plan[it % kPlans].first, last = sh.plan[it % kPlans].last;
    warp_arrive(sh.plan_free[it % kPlans]);
    if (first && !wait(sh.q_ready, item++)) return false;
    if (!wait(sh.k_full[it % kCodeStages], it / kCodeStages)) return false;
    if (tc::elected()) {
#pragma unroll
      for (int k = 0; k < DP / 16; ++k)  // both parts of the queries with the same keys
        tc::product_e4m3(tmem + T::kS + st * kTokens, tmem + T::kQ + (k & 1) * (DP / 4) + (k >> 1) * 8,
                         tc::tile_descriptor(k_tiles + static_cast<uint32_t>(it % kCodeStages) * T::kKeyBytes + (k >> 1) * 32, 16, 1024),
                         kScores, k > 0);
      tc::products_arrive(tc::smem_address(&sh.s_full[st]));
    }
    __syncwarp();
    if (!first && !weigh(it - 1, first_before)) return false;
    if (last && !weigh(it, first)) return false;
    first_before = first;
  }
  return true;
}

// ---- scores to weights, and results ----

// Which of a tile's tokens the thread's row sees, 32 to a word.
__device__ __forceinline__ void seen_tokens(const AttentionParams& a, const TilePlan& plan, const int32_t* parents, int ctx, int token,
                                            int pos, uint32_t (&seen)[4]) {
  const int past = parents ? ctx : pos + 1;
  const int from = a.window ? max(0, pos - a.window + 1) : 0;
#pragma unroll
  for (int i = 0; i < kTileSteps; ++i) {
    uint32_t b = 0;
    if (plan.count[i] > 0) {
      const int base = plan.token[i];
      b = bits16(base, from, past);
      if (a.window) b |= bits16(base, 0, min(a.sinks, past));
      if (parents && base + kStep > ctx)
        for (int u = token, back = 0; u >= 0; u = tree_parent(parents, u), ++back) {
          const int j = ctx + u - base;
          if (j >= 0 && j < kStep && (a.window == 0 || back < a.window || pos - back < a.sinks)) b |= 1u << j;
        }
    }
    if (i & 1)
      seen[i >> 1] |= b << 16;
    else
      seen[i >> 1] = b;
  }
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
__device__ bool softmax_role(const AttentionParams& a, const long long tiles, Shared& sh, uint32_t tmem, int g) {
  using T = Tiles<DP>;
  const int r = threadIdx.x;
  const uint32_t mine = tmem + ((threadIdx.x >> 5) << 21);  // the warp's 32 lanes
  const auto wait = [&](uint64_t& bar, long long n) {
    const bool ok = warp_wait(sh, bar, n);
    tc::fence_after();
    return ok;
  };
  const auto arrive = [&](uint64_t& bar) {
    tc::wait_stores();
    tc::fence_before();
    warp_arrive(bar);
  };
  long long it = 0;
  for (long long item = 0; it < tiles; ++item) {
    if (!wait(sh.part_full[item % kParts], item / kParts)) return false;
    const Part p = sh.part[item % kParts];
    warp_arrive(sh.part_free[item % kParts]);
    const int32_t* parents = a.parents ? a.parents + p.row0 : nullptr;
    const int row = p.r0 + min(r, p.rows - 1);
    const int token = row / a.group, head = p.h * a.group + row % a.group;
    const int64_t out_row = static_cast<int64_t>(p.row0) + token;

    // the row's queries, scaled by a power of two, in two parts
    float factor;
    {
      const uint16_t* q = static_cast<const uint16_t*>(a.q) + out_row * a.q_row_stride + head * a.q_head_stride;
      uint4 raw[DP / 8];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (r < p.rows && i * 8 < a.w.dim) {
          if (a.q_vec) {
            raw[i] = *reinterpret_cast<const uint4*>(q + i * 8);
          } else {
            const uint16_t* e = q + i * 8;
            raw[i] = make_uint4(__ldg(e) | __ldg(e + 1) << 16, __ldg(e + 2) | __ldg(e + 3) << 16,
                                __ldg(e + 4) | __ldg(e + 5) << 16, __ldg(e + 6) | __ldg(e + 7) << 16);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        top = __vmaxu2(__vmaxu2(top, raw[i].x & 0x7fff7fffu), raw[i].y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, raw[i].z & 0x7fff7fffu), raw[i].w & 0x7fff7fffu);
      }
      const int exponent = static_cast<int>(max(top >> 16, top & 0xffffu) >> 7);
      const int e = exponent == 255 || top == 0 ? 0 : min(120, 134 - exponent);
      __syncwarp();
      // the largest becomes 2^7 .. 2^8; a negative factor goes into the queries, so that larger products are larger scores
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * (a.scale_log2 < 0.0f ? -1.0f : 1.0f);
      factor = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (exponent == 255) factor = CUDART_NAN_F;  // the row's scores are not numbers
      uint32_t hi[DP / 4], lo[DP / 4];
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        float f[8];
        unpack<uint16_t>(raw[i], f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t h[2], r[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float u = f[4 * k + 2 * n] * up, v = f[4 * k + 2 * n + 1] * up;
            h[n] = floats_to_e4m3x2(u, v);
            const float2 held = f16x2_to_float2(e4m3x2_to_f16x2(h[n]));
            r[n] = floats_to_e4m3x2(u - held.x, v - held.y);
          }
          hi[2 * i + k] = h[0] | h[1] << 16;
          lo[2 * i + k] = r[0] | r[1] << 16;
        }
      }
      if constexpr (DP == 128) {
        tc::tmem_store32(mine + T::kQ, hi);
        tc::tmem_store32(mine + T::kQ + 32, lo);
      } else {
        uint32_t both[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          both[i] = hi[i];
          both[16 + i] = lo[i];
        }
        tc::tmem_store32(mine + T::kQ, both);
      }
      arrive(sh.q_ready);
    }
    int pos = p.ctx + token;
    if (parents) {
      int depth = 0;
      for (int u = tree_parent(parents, token); u >= 0; u = tree_parent(parents, u)) ++depth;
      pos = p.ctx + depth;
      __syncwarp();
    }

    float m = -CUDART_INF_F, l = 0.0f, v_ref = kNoScale;  // v_ref: log2 of the values' unit
    for (int t = 0; t < p.count; ++t, ++it) {
      const int st = it & 1;
      const TilePlan& plan = sh.plan[it % kPlans];
      if (!wait(sh.plan_full[it % kPlans], it / kPlans) || !wait(sh.s_full[st], it >> 1)) return false;
      const uint32_t scores = mine + T::kS + st * kTokens;
      float v_top = kNoScale;
#pragma unroll
      for (int i = 0; i < kTileSteps; ++i) v_top = fmaxf(v_top, plan.v_log2[i]);
      // Twice over the scores, 64 at a time.  The loops stay rolled: the roles share the instruction cache, and this one
      // in a straight line took 2100 cycles a tile instead of 800.
      const auto tile = [&](auto masked) {
        constexpr bool M = decltype(masked)::value;
        uint32_t seen[4] = {};
        if (M) {
          seen_tokens(a, plan, parents, p.ctx, token, pos, seen);
          __syncwarp();
        }
        float top = -CUDART_INF_F;  // the tile's largest score in base 2
        uint32_t x0[32], x1[32];
        tc::tmem_load32(scores, x0);
#pragma unroll 1
        for (int i = 0; i < kTokens; i += 64) {
          const uint32_t b0 = i ? seen[2] : seen[0], b1 = i ? seen[3] : seen[1];
          const float* k = plan.k_scale + i / kStep;
          tc::wait_loads(x0);
          tc::tmem_load32(scores + i + 32, x1);
          top = fmaxf(top, fmaxf(largest16<M>(&x0[0], b0) * (factor * k[0]), largest16<M>(&x0[16], b0 >> 16) * (factor * k[1])));
          tc::wait_loads(x1);
          tc::tmem_load32(scores + (i + 64) % kTokens, x0);  // at the end the first again
          top = fmaxf(top, fmaxf(largest16<M>(&x1[0], b1) * (factor * k[2]), largest16<M>(&x1[16], b1 >> 16) * (factor * k[3])));
        }
        if (t == 0) {
          m = top;
          v_ref = v_top;
        } else if (__any_sync(0xffffffffu, top > m + 7.0f || v_top > v_ref)) {
          const float up = fmaxf(m, top);
          float fix = up == -CUDART_INF_F ? 1.0f : ex2(m - up);
          l *= fix;
          m = up;
          if (v_top > v_ref) {
            fix *= ex2(v_ref - v_top);
            v_ref = v_top;
          }
          if (!wait(sh.pv_done[(it - 1) & 1], (it - 1) >> 1)) return false;
#pragma unroll 1
          for (int i = 0; i < DP; i += 32) {
            tc::tmem_load32(mine + T::kO + i, x1);
            tc::wait_loads(x1);
#pragma unroll
            for (int k = 0; k < 32; ++k) x1[k] = __float_as_uint(__uint_as_float(x1[k]) * fix);
            tc::tmem_store32(mine + T::kO + i, x1);
          }
        }
        // weights, in the place of the scores' first half, in units of their values' scales
        const float base = kLift - (m == -CUDART_INF_F ? 0.0f : m);
#pragma unroll 1
        for (int i = 0; i < kTokens; i += 64) {
          const uint32_t b0 = i ? seen[2] : seen[0], b1 = i ? seen[3] : seen[1];
          const float* k = plan.k_scale + i / kStep;
          const float* v = plan.v_log2 + i / kStep;
          uint32_t w[32];
          float u[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) u[n] = fmaxf(v[n] - v_ref, -100.0f);
          tc::wait_loads(x0);
          tc::tmem_load32(scores + i + 32, x1);
          float2 sums = weights32<M>(x0, b0, factor * k[0], factor * k[1], base + u[0], base + u[1], w);
          l += sums.x * ex2(-u[0]) + sums.y * ex2(-u[1]);
          tc::wait_loads(x1);
          if (i == 0) tc::tmem_load32(scores + 64, x0);
          sums = weights32<M>(x1, b1, factor * k[2], factor * k[3], base + u[2], base + u[3], w + 16);
          l += sums.x * ex2(-u[2]) + sums.y * ex2(-u[3]);
          tc::tmem_store32(scores + i / 2, w);
        }
        return true;
      };
      if (!(plan.whole ? tile(std::false_type{}) : tile(std::true_type{}))) return false;
      arrive(sh.p_ready[st]);
      warp_arrive(sh.plan_free[it % kPlans]);
    }

    // the part's result
    if (!wait(sh.pv_done[(it - 1) & 1], (it - 1) >> 1)) return false;
    const bool complete = p.count == p.tiles;
    const float lift = 1.0f / 256.0f;
    l *= lift;
    const float scale = ex2(v_ref) * lift;
    if (complete) {
      uint16_t* out = static_cast<uint16_t*>(a.out) + out_row * a.out_row_stride + head * a.out_head_stride;
      const float inv = l == 0.0f ? 0.0f : scale / l;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        uint32_t x[32];
        tc::tmem_load32(mine + T::kO + 32 * i, x);
        tc::wait_loads(x);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t o[8];
#pragma unroll
          for (int n = 0; n < 8; ++n)
            o[n] = floats_to_bf16x2(__uint_as_float(x[16 * k + 2 * n]) * inv, __uint_as_float(x[16 * k + 2 * n + 1]) * inv);
          const int d = 32 * i + 16 * k;
          if (r < p.rows && d < a.w.dim) {
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
        }
        __syncwarp();
      }
      if (r < p.rows && a.lse) a.lse[out_row * a.heads + head] = row_lse(m, l);
    } else {
      float* part = a.parts + (2 * static_cast<int64_t>(g) + (p.tile0 == 0 ? 1 : 0)) * T::kPart;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        uint32_t x[32];
        tc::tmem_load32(mine + T::kO + 32 * i, x);
        tc::wait_loads(x);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t o[8];
#pragma unroll
          for (int n = 0; n < 8; ++n) o[n] = __float_as_uint(__uint_as_float(x[8 * k + n]) * scale);
          if (r < p.rows) tc::store_32(part + r * DP + 32 * i + 8 * k, o);
        }
        __syncwarp();
      }
      if (r < p.rows) *reinterpret_cast<float2*>(part + kRows * DP + 2 * r) = make_float2(m, l);
      if (p.tile0 == 0 && r == 0)
        a.joins[g] = JoinRecord{p.row0, p.r0, p.rows, p.h, p.join_last};
    }
    __syncwarp();
  }
  return true;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tiles_kernel(AttentionParams a) {
  using T = Tiles<DP>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t at = tc::smem_address(raw);
  uint8_t* tiles = raw + ((at + 1023u & ~1023u) - at);
  uint8_t* v_tiles = tiles;
  uint8_t* k_tiles = tiles + 2 * T::kValueBytes;
  const int warp = threadIdx.x >> 5, g = blockIdx.x;
  flag_sequences(a, g, gridDim.x, kThreads);
  if (threadIdx.x == 0) {
    a.joins[g].rows = 0;
    sh.gave_up = 0;
    for (int i = 0; i < kCodeStages; ++i) tc::barrier_init(tc::smem_address(&sh.k_full[i]), kLoadWarps);
    for (int i = 0; i < 2; ++i) {
      tc::barrier_init(tc::smem_address(&sh.v_full[i]), kLoadWarps);
      tc::barrier_init(tc::smem_address(&sh.s_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.p_ready[i]), kSoftmaxWarps);
      tc::barrier_init(tc::smem_address(&sh.pv_done[i]), 1);
    }
    for (int i = 0; i < kPlans; ++i) {
      tc::barrier_init(tc::smem_address(&sh.plan_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.plan_free[i]), kLoadWarps + kSoftmaxWarps + 1);
    }
    for (int i = 0; i < kParts; ++i) {
      tc::barrier_init(tc::smem_address(&sh.part_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.part_free[i]), kSoftmaxWarps);
    }
    tc::barrier_init(tc::smem_address(&sh.q_ready), kSoftmaxWarps);
    tc::barrier_init(tc::smem_address(&sh.last), 1);
    tc::publish_shared();
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_address(&sh.tmem), T::kColumns);
  const Cursor c = find_cursor<kThreads, kRows, kTileSteps>(a, g, gridDim.x, sh.cursor);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  const long long tiles_here = c.end - c.at;
  bool ok = true;
  if (warp < kSoftmaxWarps) {
    tc::registers_up<kSoftmaxRegisters>();
    ok = softmax_role<DP>(a, tiles_here, sh, tmem, g);
  } else if (warp < kSoftmaxWarps + kLoadWarps) {
    tc::registers_down<kLoadRegisters>();
    ok = load_role<DP>(a, tiles_here, sh, k_tiles, v_tiles, k_tiles + kCodeStages * T::kKeyBytes);
  } else {
    tc::registers_down<kProductRegisters>();
    if (warp == kSoftmaxWarps + kLoadWarps) {
      ok = product_role<DP>(tiles_here, sh, tc::smem_address(k_tiles), tc::smem_address(v_tiles), tmem);
      // products in flight end before the memory that they use is given up
      int unused = 0;
      if (tc::elected()) tc::products_arrive(tc::smem_address(&sh.last));
      ok = tc::barrier_wait(tc::smem_address(&sh.last), 0, &unused) && ok;
      __syncwarp();
    } else if (warp == kSoftmaxWarps + kLoadWarps + 1) {
      ok = plan_role(a, c, sh);
    }
  }
  if (!ok && (threadIdx.x & 31) == 0) kv_flag(a.w, min(c.b, a.w.batch - 1), SV_ROW_TIMEOUT);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::tmem_free(tmem, T::kColumns);
}

template <int DP>
sv_status launch(AttentionParams a, const sv_kv_attention_desc& d, void* workspace, cudaStream_t stream) {
  using T = Tiles<DP>;
  static FuncAttrCache attr;
  const auto kernel = kv_attention_tiles_kernel<DP>;
  if (!attr.ensure(reinterpret_cast<const void*>(kernel), T::kShared, false)) return SV_ERR_CUDA;
  const int64_t row_tiles = (static_cast<int64_t>(d.max_new) * a.group + kRows - 1) / kRows;
  const int64_t tiles = (static_cast<int64_t>(d.kv.max_pages) * d.kv.page_size + kTokens - 1) / kTokens;
  const int blocks = schedule_blocks(row_tiles * d.kv.batch * d.kv.kv_heads, tiles, kSMs);
  a.parts = static_cast<float*>(workspace);
  a.joins = reinterpret_cast<JoinRecord*>(a.parts + 2 * static_cast<int64_t>(kSMs) * T::kPart);
  kernel<<<blocks, kThreads, T::kShared, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  if (blocks == 1 || tiles == 1) return SV_OK;  // no item has parts
  if (launch_join<uint16_t, DP, kRows>(a, blocks, stream) != cudaSuccess) return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

}  // namespace

bool kv_attention_takes_tiles(const sv_kv_attention_desc& d) {
  return d.dtype == SV_BF16 && d.kv.head_dim <= 128 &&
         static_cast<int64_t>(d.max_new) * (d.heads / d.kv.kv_heads) > 16;
}

size_t kv_attention_tiles_workspace(const sv_kv_attention_desc& d) {
  const size_t part = d.kv.head_dim <= 64 ? Tiles<64>::kPart : Tiles<128>::kPart;
  return align_up(kSMs * (2 * part * sizeof(float) + sizeof(JoinRecord)), 256);
}

sv_status kv_attention_tiles(AttentionParams a, const sv_kv_attention_desc& d, void* workspace, cudaStream_t stream) {
  return d.kv.head_dim <= 64 ? launch<64>(a, d, workspace, stream) : launch<128>(a, d, workspace, stream);
}

}  // namespace sv
