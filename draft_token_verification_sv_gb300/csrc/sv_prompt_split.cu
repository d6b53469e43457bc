// Causal attention of float32 prompts, and of bf16 ones that tensor copies
// cannot read, on the 5th-generation tensor cores.
//
// A float32 value is the sum of three bf16 values (8 significant bits each,
// with signs, and float's range), so a product of two is the sum of the six
// products of their parts that are not below 2^-24 of it.  Tensor memory cuts
// sums off, it does not round them, so the sum of the five small products is
// formed beside that of the large one, and the sums over values are formed anew
// for each tile of keys and added to the results where they are rounded.
// (Scores of 256 dims lost 8.7 * 2^-23 of their size in the mean with all six in
// one sum, 0.8 with two.)
//
// Queries, keys and values are read with ordinary loads, split, and written to
// shared memory as the products want them; weights are split where they are
// made.  One tile of 128 query rows (sv_prompt_items.cuh) against tiles of 64
// keys, two of which are under way.  Roles of a block's warps:
//   four turn scores into weights, a row a thread (sv_prompt_tiles.cu says how);
//   eight load and split, and leave out values that are not finite, which rows
//   that see them get where results are written;
//   one issues the products; one finds the items.
// Three prompts of up to 4001 tokens under windows of 2048 (16 heads of 64
// float32 dims) take 435 us, 127 TFLOP/s, six times that in products.  A tile's
// 48 products, 50 cycles each one after the other, fill 0.7 of its 3300 cycles
// (their arithmetic, 32 cycles each, 0.5; ncu has the tensor core active for
// 0.38 of the kernel's time); the chain of a row's thread (scores, 64 weights in
// three parts each, sums) is about as long, with issue slots and instruction
// fetches that it shares with the loaders.  Which of these bounds it is not
// settled: less of one alone gained nothing.
// Above 128 float32 dims a block's queries do not fit shared memory: they come
// again with each tile of keys, 64 dims at a time, and tensor memory has room for
// the scores of one tile only.
#include "sv_prompt_items.cuh"

#include <algorithm>
#include <type_traits>

namespace sv {

namespace {

constexpr int kKeys = 64;
constexpr int kItems = 4;
constexpr float kLargeSum = 8192.0f;
constexpr int kSoftmaxWarps = 4, kLoadWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + kLoadWarps + 4);
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kSoftmaxRegisters = 208, kLoadRegisters = 112, kOtherRegisters = 64;
static_assert(kSoftmaxWarps * kSoftmaxRegisters + kLoadWarps * kLoadRegisters + 4 * kOtherRegisters <= 16 * 128, "registers of a block");

template <int DP, typename E> struct Config {
  static constexpr int kParts = sizeof(E) == 4 ? 3 : 1;           // bf16 values that make a value
  static constexpr bool kStream = DP == 256 && kParts == 3;       // queries come with each tile of keys
  static constexpr int kUnitDims = kStream || DP < 128 ? 64 : 128, kUnits = DP / kUnitDims;  // of a tile of keys or values
  static constexpr int kQueryPart = kRows * (kStream ? kUnitDims : DP) * 2;  // bytes of one part of a tile of queries (of a unit's)
  static constexpr int kPart = kKeys * kUnitDims * 2;  // and of keys or values
  static constexpr int kKeyAt = kStream ? kParts * kQueryPart : 0;  // of the keys in a stage
  static constexpr int kStageBytes = kKeyAt + kParts * kPart;
  static constexpr int kQueryBytes = kStream ? 0 : kParts * kQueryPart;
  static constexpr int kRoom = 224 * 1024 - kQueryBytes;
  static constexpr int kStages = kRoom / kStageBytes < 6 ? kRoom / kStageBytes : 6;
  static constexpr int kBytes = kQueryBytes + kStages * kStageBytes;
  // more than half of an SM's shared memory keeps it to one block
  static constexpr int kShared = (kBytes > 118 * 1024 ? kBytes : 118 * 1024) + 1024;
  // tensor memory, in columns: places for scores (large and small products' sums) and the weights they become, O, and the sums of a
  // unit of values
  static constexpr int kPlaces = kStream ? 1 : 2, kPlace = kParts == 1 ? kKeys : 2 * kKeys, kO = kPlaces * kPlace, kSums = kO + DP;
  static_assert(kPlace >= kParts * (kKeys / 2) && kSums + kUnitDims <= 512, "tensor memory");
};

struct Shared {
  uint64_t item_full[kItems], item_free[kItems];
  uint64_t q_full, q_free, full[6], free[6];
  uint64_t s_full[2], p_ready[2], sums_full, sums_free, last, answer;
  uint4 block;
  Item item[kItems];
  Sequences sequences;
  float rest[kSoftmaxWarps][SV_MAX_HEAD_DIM];  // see sum_rest
  uint32_t tmem;
  int gave_up;
  int claimed, finished[kSoftmaxWarps];
};

__device__ __forceinline__ bool warp_wait(Shared& sh, uint64_t& bar, int n) {
  return __all_sync(0xffffffffu, tc::barrier_wait(tc::smem_address(&bar), static_cast<uint32_t>(n & 1), &sh.gave_up));
}
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::barrier_arrive(tc::smem_address(&bar));
}

// ---- items ----

struct Plans {
  int answers;
  bool asked;
  long long next;
};

__device__ bool plan_role(const PromptView& a, int tpt, Shared& sh, Finder& finder, Plans& under) {
  const int lane = threadIdx.x & 31;
  int items = 0;
  const auto publish = [&](const Item& it) {
    if (items >= kItems && !warp_wait(sh, sh.item_free[items % kItems], items / kItems - 1)) return false;
    if (lane == 0) {
      sh.item[items % kItems] = it;
      if (it.tiles >= 0) sh.claimed = items + 1;
    }
    warp_arrive(sh.item_full[items % kItems]);
    ++items;
    return true;
  };
  Item it;
  for (int x = blockIdx.x; x >= 0;) {
    if (lane == 0) {
      const uint32_t bar = tc::smem_address(&sh.answer);
      tc::barrier_expect(bar, sizeof(sh.block));
      tc::ask_for_block(tc::smem_address(&sh.block), bar);
    }
    under.asked = true;
    for (under.next = x; finder.find<kKeys, 1>(a, sh.sequences, tpt, under.next, it); under.next += gridDim.x)
      if (!publish(it)) return false;
    if (!warp_wait(sh, sh.answer, under.answers)) return false;
    ++under.answers;
    under.asked = false;
    x = tc::taken_block(tc::smem_address(&sh.block));
    __syncwarp();
    tc::publish_shared();  // (read before the next answer is written)
  }
  it.tiles = -1;
  return publish(it);
}

// ---- loading and splitting ----

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }

// Two values in as many parts.
template <int PARTS>
__device__ __forceinline__ void split(float a, float b, uint32_t (&w)[PARTS]) {
#pragma unroll
  for (int p = 0; p < PARTS; ++p) {
    w[p] = floats_to_bf16x2(a, b);
    if (p + 1 < PARTS) {
      const float2 r = unpack_bf16x2(w[p]);
      a -= r.x;
      b -= r.y;
    }
  }
}

// The same of values whose first part may not be finite: it is taken towards
// zero where it would pass bf16's range, and infinities and NaN become NaN (or
// are left out, which the answer says): products of an infinity with the other
// side's parts would have their signs, which differ.
__device__ __noinline__ bool split_any(const float (&x)[8], bool leave_out, uint32_t (&w)[3][4]) {
  bool left = false;
  for (int p = 0; p < 3; ++p)
    for (int k = 0; k < 4; ++k) w[p][k] = 0;
  for (int k = 0; k < 8; ++k) {
    float v = x[k];
    const bool finite = fabsf(v) < CUDART_INF_F;
    if (!finite && leave_out) {
      left = true;
      continue;
    }
    const bool large = (__float_as_uint(v) & 0x7fffffffu) >= 0x7f7f8000u;
    for (int p = 0; p < (finite ? 3 : 1); ++p) {
      const uint32_t top = !finite ? 0x7fffu : large ? __float_as_uint(v) >> 16 : floats_to_bf16x2(v, 0.0f) & 0xffffu;
      w[p][k >> 1] |= top << (16 * (k & 1));
      v -= __uint_as_float(top << 16);
    }
  }
  return left;
}

// Eight values of a row; zeros behind its dims.
template <typename E>
__device__ __forceinline__ void fetch8(const E* at, bool there, bool vec, uint32_t (&raw)[2 * sizeof(E)]) {
  if constexpr (sizeof(E) == 4) {
    if (vec) {
      const uint4 u = there ? __ldg(reinterpret_cast<const uint4*>(at)) : make_uint4(0, 0, 0, 0);
      const uint4 v = there ? __ldg(reinterpret_cast<const uint4*>(at) + 1) : make_uint4(0, 0, 0, 0);
      raw[0] = u.x, raw[1] = u.y, raw[2] = u.z, raw[3] = u.w, raw[4] = v.x, raw[5] = v.y, raw[6] = v.z, raw[7] = v.w;
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) raw[k] = there ? __ldg(reinterpret_cast<const uint32_t*>(at) + k) : 0u;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) raw[k] = there ? __ldg(at + 2 * k) | static_cast<uint32_t>(__ldg(at + 2 * k + 1)) << 16 : 0u;
  }
}

// Writes them in their parts; true: some were left out.
template <typename E, int PARTS>
__device__ __forceinline__ bool store8(const uint32_t (&raw)[2 * sizeof(E)], bool leave_out, uint8_t* to, int part_bytes) {
  if constexpr (sizeof(E) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, raw[k] & 0x7fffffffu);
    uint32_t w[3][4];
    bool left = false;
    if (__builtin_expect(m < 0x7f7f8000u, 1)) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t two[3];
        split<3>(__uint_as_float(raw[2 * k]), __uint_as_float(raw[2 * k + 1]), two);
#pragma unroll
        for (int p = 0; p < 3; ++p) w[p][k] = two[p];
      }
    } else {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(raw[k]);
      left = split_any(x, leave_out, w);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(to + p * part_bytes) = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
    return left;
  } else {
    uint32_t w[4], drop = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t bad = leave_out ? __vcmpgeu2(raw[k] & 0x7fff7fffu, 0x7f807f80u) : 0u;
      drop |= bad;
      w[k] = raw[k] & ~bad;
    }
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    return drop != 0;
  }
}

// ROWS rows of DIMS dims from d0 on to shared memory, in their parts, in blocks of 64 dims of swizzled rows.  place(r): the row's
// offset, or -1.  MOST: eights of a thread under way.
template <typename E, int ROWS, int DIMS, int MOST, typename Place>
__device__ __forceinline__ bool load_rows(const E* from, Place place, int d0, int dim, bool vec, bool leave_out, uint8_t* to) {
  constexpr int kParts = sizeof(E) == 4 ? 3 : 1, kChunks = DIMS / 8, kAll = ROWS * kChunks / kLoadThreads, kOnce = kAll < MOST ? kAll : MOST;
  static_assert(ROWS * kChunks % kLoadThreads == 0 && kAll % kOnce == 0, "chunks of a thread");
  const int tid = threadIdx.x - 32 * kSoftmaxWarps;
  bool left = false;
#pragma unroll 1
  for (int n = 0; n < kAll; n += kOnce) {
    uint32_t raw[kOnce][2 * sizeof(E)];
#pragma unroll
    for (int k = 0; k < kOnce; ++k) {
      const int at = tid + (n + k) * kLoadThreads, r = at / kChunks, d = d0 + (at % kChunks) * 8;
      const int64_t offset = place(r);
      fetch8<E>(from + offset + d, offset >= 0 && d < dim, vec, raw[k]);
    }
#pragma unroll
    for (int k = 0; k < kOnce; ++k) {
      const int at = tid + (n + k) * kLoadThreads, r = at / kChunks, c = at % kChunks;
      left |= store8<E, kParts>(raw[k], leave_out, to + (c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), ROWS * DIMS * 2);
    }
  }
  return left;
}

template <int DP, typename E>
__device__ bool load_role(const PromptView& a, int tpt, Shared& sh, uint8_t* q_at, uint8_t* stages, bool vec) {
  using C = Config<DP, E>;
  int unit = 0, loaded = 0;
  for (int items = 0;; ++items) {
    if (!warp_wait(sh, sh.item_full[items % kItems], items / kItems)) return false;
    Item& it = sh.item[items % kItems];
    const int tiles = it.tiles;
    if (tiles < 0) return true;
    const E* q = static_cast<const E*>(a.q);
    const E* k = static_cast<const E*>(a.k) + static_cast<int64_t>(it.row0) * a.k_row + it.h * a.k_head;
    const E* v = static_cast<const E*>(a.v) + static_cast<int64_t>(it.row0) * a.v_row + it.h * a.v_head;
    const auto query = [&](int r) {
      const Place p = place_of(a, it, tpt, 0, r);
      return p.row >= 0 ? p.row * a.q_row + p.head * a.q_head : int64_t{-1};
    };
    const int n = it.n;
    const auto token = [&](int kb, int64_t stride) {
      return [=, &a](int r) { return kb + r < n && sv_in(static_cast<int64_t>(it.row0) + kb + r, a.total_new) ? (kb + r) * stride : int64_t{-1}; };
    };
    if constexpr (!C::kStream) {
      if (items > 0 && !warp_wait(sh, sh.q_free, items - 1)) return false;
      load_rows<E, kRows, DP, 2>(q, query, 0, a.dim, vec, false, q_at);
      tc::publish_shared();
      warp_arrive(sh.q_full);
    }
    // (keys and values by the same instructions, queries by few: they are fetched anew each time, and a copy for each took 446 us
    // for what now takes 435)
#pragma unroll 1
    for (int n = 0; n < 2 * tiles; ++n) {
      if (loaded++ == SV_PROMPT_LOST_TILE) return false;
      const Turn turn = turn_of<C::kPlaces == 2>(n, tiles);
      const int kb = key_of<kKeys>(it, turn.t);
#pragma unroll 1
      for (int u = 0; u < C::kUnits; ++u) {
        if (unit >= C::kStages && !warp_wait(sh, sh.free[unit % C::kStages], unit / C::kStages - 1)) return false;
        uint8_t* at = stages + unit % C::kStages * C::kStageBytes;
        if (C::kStream && turn.keys) load_rows<E, kRows, C::kUnitDims, 4>(q, query, u * C::kUnitDims, a.dim, vec, false, at);
        if (load_rows<E, kKeys, C::kUnitDims, 4>(turn.keys ? k : v, token(kb, turn.keys ? a.k_row : a.v_row), u * C::kUnitDims, a.dim, vec, !turn.keys,
                                              at + (turn.keys ? C::kKeyAt : 0)))
          atomicOr(&it.dirty, 1 << (turn.t & 31));
        tc::publish_shared();
        warp_arrive(sh.full[unit % C::kStages]);
        ++unit;
      }
    }
    warp_arrive(sh.item_free[items % kItems]);
  }
}

// ---- products ----

// Parts of the left and right side of the n-th product, the smallest first.
template <int PARTS>
__device__ __forceinline__ constexpr int left_part(int n) {
  return PARTS == 1 ? 0 : n == 0 ? 0 : n == 1 ? 1 : n == 2 ? 2 : n == 3 ? 0 : n == 4 ? 1 : 0;
}
template <int PARTS>
__device__ __forceinline__ constexpr int right_part(int n) {
  return PARTS == 1 ? 0 : n == 0 ? 2 : n == 1 ? 1 : n == 2 ? 0 : n == 3 ? 1 : n == 4 ? 0 : 0;
}

template <int DP, typename E>
__device__ bool product_role(Shared& sh, uint32_t q_at, uint32_t stages, uint32_t tmem) {
  using C = Config<DP, E>;
  constexpr int kProducts = C::kParts == 1 ? 1 : 6;
  constexpr uint32_t kScores = tc::product_kind_bf16(kKeys, false), kValues = tc::product_kind_bf16(C::kUnitDims, true);
  const auto wait = [&](uint64_t& bar, int n) {
    const bool ok = tc::barrier_wait(tc::smem_address(&bar), static_cast<uint32_t>(n & 1), &sh.gave_up);
    tc::fence_after();
    return ok;
  };
  const auto arrive = [&](uint64_t& bar) { tc::products_arrive(tc::smem_address(&bar)); };
  int unit = 0, tile = 0, sums = 0;
  for (int items = 0;; ++items) {
    if (!wait(sh.item_full[items % kItems], items / kItems)) return false;
    const int tiles = sh.item[items % kItems].tiles;
    tc::barrier_arrive(tc::smem_address(&sh.item_free[items % kItems]));
    if (tiles < 0) return true;
    const auto score = [&](int s) {
      for (int u = 0; u < C::kUnits; ++u, ++unit) {
        const int stage = unit % C::kStages;
        if (!wait(sh.full[stage], unit / C::kStages)) return false;
        const uint32_t at = stages + stage * C::kStageBytes, k = at + C::kKeyAt;
        const uint32_t q = C::kStream ? at : q_at + u * (C::kUnitDims / 64) * (kRows * 128);
#pragma unroll
        for (int n = 0; n < kProducts; ++n)
#pragma unroll
          for (int d = 0; d < C::kUnitDims / 16; ++d)
            tc::product_f16(tmem + s * C::kPlace + (n + 1 < kProducts ? kKeys : 0),
                            tc::tile_descriptor(q + left_part<C::kParts>(n) * C::kQueryPart + (d >> 2) * (kRows * 128) + (d & 3) * 32, 16, 1024),
                            tc::tile_descriptor(k + right_part<C::kParts>(n) * C::kPart + (d >> 2) * (kKeys * 128) + (d & 3) * 32, 16, 1024), kScores,
                            u > 0 || (n > 0 && n + 1 < kProducts) || d > 0);
        arrive(sh.free[stage]);
      }
      arrive(sh.s_full[s]);
      return true;
    };
    if (!C::kStream && !wait(sh.q_full, items)) return false;
    // the next tile's scores are formed before a tile's sums, where they have a place of their own
    const auto next = [&](int t) {
      if (t >= tiles) return true;
      if (!score((tile + (C::kPlaces == 2 && t > 0)) % C::kPlaces)) return false;
      if (!C::kStream && t + 1 == tiles) arrive(sh.q_free);
      return true;
    };
    if (!next(0)) return false;
    for (int t = 0; t < tiles; ++t, ++tile) {
      if (C::kPlaces == 2 && !next(t + 1)) return false;
      if (!wait(sh.p_ready[tile % C::kPlaces], tile / C::kPlaces)) return false;
      for (int u = 0; u < C::kUnits; ++u, ++unit, ++sums) {
        const int stage = unit % C::kStages;
        if (!wait(sh.full[stage], unit / C::kStages)) return false;
        if (sums > 0 && !wait(sh.sums_free, sums - 1)) return false;
        const uint32_t v = stages + stage * C::kStageBytes;
#pragma unroll
        for (int n = 0; n < kProducts; ++n)
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            tc::product_f16(tmem + C::kSums, tmem + tile % C::kPlaces * C::kPlace + left_part<C::kParts>(n) * (kKeys / 2) + k * 8,
                            tc::tile_descriptor(v + right_part<C::kParts>(n) * C::kPart + k * 2048, kKeys * 128, 1024), kValues,
                            n > 0 || k > 0);
        arrive(sh.free[stage]);
        arrive(sh.sums_full);
      }
      if (C::kPlaces == 1 && !next(t + 1)) return false;
    }
  }
}

// ---- scores to weights, and results ----

// 32 scores to weights 2^(x f + c), in their parts; their sum.
template <int PARTS>
__device__ __forceinline__ float weights32(const uint32_t (&x)[32], uint32_t seen, float f, float c, uint32_t (&w)[PARTS][16]) {
  float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    float a = ex2(fmaf(__uint_as_float(x[2 * k]), f, c)), b = ex2(fmaf(__uint_as_float(x[2 * k + 1]), f, c));
    a = seen >> (2 * k) & 1u ? a : 0.0f;
    b = seen >> (2 * k + 1) & 1u ? b : 0.0f;
    sum[2 * (k & 1)] += a;
    sum[2 * (k & 1) + 1] += b;
    uint32_t two[PARTS];
    split<PARTS>(a, b, two);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) w[p][k] = two[p];
  }
  return (sum[0] + sum[1]) + (sum[2] + sum[3]);
}

// Sums of the values that were left out of tiles that every row sees, by a warp; `dirty`: where there may be some.
template <typename E>
__device__ __noinline__ void sum_rest(const PromptView& a, const Item& it, int tpt, int dirty, float* sums) {
  const E* v = static_cast<const E*>(a.v) + static_cast<int64_t>(it.row0) * a.v_row + it.h * a.v_head;
  for (int d = threadIdx.x & 31; d < a.dim; d += 32) {
    float sum = 0.0f;
    for (int t = 0; t < it.tiles; ++t) {
      if (!(dirty >> (t & 31) & 1) || partly_seen<kKeys, 1>(a, it, tpt, t)) continue;
      const int kb = key_of<kKeys>(it, t);
#pragma unroll 8
      for (int j = kb; j < kb + kKeys; ++j) {
        const float y = sv_in(it.row0 + static_cast<int64_t>(j), a.total_new) ? value_of(v + j * a.v_row + d) : 0.0f;
        sum += fabsf(y) < CUDART_INF_F ? 0.0f : y;
      }
    }
    sums[d] = sum;
  }
  __syncwarp();
}

template <int DP, typename E>
__device__ bool softmax_role(const PromptView& a, int tpt, float f, Shared& sh, uint32_t tmem, bool out_vec32) {
  using C = Config<DP, E>;
  const int r = threadIdx.x, quarter = threadIdx.x >> 5;
  const uint32_t mine = tmem + (quarter << 21);  // the warp's 32 lanes
  const uint32_t own_o = mine + C::kO;
  const auto wait = [&](uint64_t& bar, int n) {
    const bool ok = warp_wait(sh, bar, n);
    tc::fence_after();
    return ok;
  };
  int tile = 0, sums = 0;
  // O = O fix + the sums of the next tile: these are formed by themselves, since what the products add to is cut off, not rounded,
  // each time (over 2048 tokens that came to 6e-6 of the result; here it is 2e-7).
  const auto gather = [&](bool first, float fix) {
    for (int u = 0; u < C::kUnits; ++u, ++sums) {
      if (!wait(sh.sums_full, sums)) return false;
#pragma unroll 1
      for (int d = 0; d < C::kUnitDims; d += 32) {
        uint32_t y[32], o[2][16];
        tc::tmem_load32(mine + C::kSums + d, y);
        if (!first) {
          tc::tmem_load16(own_o + u * C::kUnitDims + d, o[0]);
          tc::tmem_load16(own_o + u * C::kUnitDims + d + 16, o[1]);
          tc::wait_loads(o[0]);
          tc::wait_loads(o[1]);
        }
        tc::wait_loads(y);
#pragma unroll
        for (int k = 0; k < 32; ++k)
          o[k >> 4][k & 15] = first ? y[k] : __float_as_uint(fmaf(__uint_as_float(o[k >> 4][k & 15]), fix, __uint_as_float(y[k])));
        tc::tmem_store(own_o + u * C::kUnitDims + d, o[0]);
        tc::tmem_store(own_o + u * C::kUnitDims + d + 16, o[1]);
      }
      tc::wait_stores();
      tc::fence_before();
      warp_arrive(sh.sums_free);
    }
    return true;
  };
  for (int items = 0;; ++items) {
    if (!wait(sh.item_full[items % kItems], items / kItems)) return false;
    const Item& it = sh.item[items % kItems];
    const int tiles = it.tiles;
    if (tiles < 0) return true;
    const Place at = place_of(a, it, tpt, 0, r);
    const int token = at.token;
    const bool held = at.row >= 0;
    float m = held ? -CUDART_INF_F : 0.0f, l = 0.0f, fix = 1.0f, fix_before = 1.0f;  // fix: of what was summed before this tile
    for (int t = 0; t < tiles; ++t, ++tile) {
      const int s = tile % C::kPlaces, kb = key_of<kKeys>(it, t);
      const uint32_t scores = mine + s * C::kPlace;
      if (!wait(sh.s_full[s], tile / C::kPlaces)) return false;
      uint32_t x[2][32], w[C::kParts][16], seen[2];
      tc::tmem_load32(scores, x[0]);
      tc::tmem_load32(scores + 32, x[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        seen[c] = bits_below(token + 1 - kb - 32 * c);
        if (a.window) seen[c] = (seen[c] & ~bits_below(max(0, token - a.window + 1) - kb - 32 * c)) | bits_below(min(a.sinks, token + 1) - kb - 32 * c);
      }
      tc::wait_loads(x[0]);
      tc::wait_loads(x[1]);
      if constexpr (C::kParts == 3) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t y[32];
          tc::tmem_load32(scores + kKeys + 32 * c, y);
          tc::wait_loads(y);
#pragma unroll
          for (int k = 0; k < 32; ++k) x[c][k] = __float_as_uint(__uint_as_float(x[c][k]) + __uint_as_float(y[k]));
        }
      }
      bool raise = held && m == -CUDART_INF_F;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (__any_sync(0xffffffffu, raise)) {
          float top = m;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k) top = fmaxf(top, seen[c] >> k & 1u ? __uint_as_float(x[c][k]) * f : -CUDART_INF_F);
          if (raise && top > -CUDART_INF_F) {
            const float down = m == -CUDART_INF_F ? 1.0f : ex2(m - top);
            m = top;
            l *= down;
            fix *= down;
          }
        }
        const float base = m == -CUDART_INF_F ? 0.0f : m;
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          sum += weights32<C::kParts>(x[c], seen[c], f, -base, w);
#pragma unroll
          for (int p = 0; p < C::kParts; ++p) tc::tmem_store(scores + p * (kKeys / 2) + 16 * c, w[p]);
        }
        raise = pass == 0 && held && sum > kLargeSum;
        if (!__any_sync(0xffffffffu, raise)) {
          l += sum;
          break;
        }
      }
      tc::wait_stores();
      tc::fence_before();
      warp_arrive(sh.p_ready[s]);
      // (with two places the last tile's sums are formed while this one's weights are made)
      if (C::kPlaces == 2 ? t > 0 && !gather(t == 1, fix_before) : !gather(t == 0, fix)) return false;
      fix_before = fix;
      fix = 1.0f;
    }
    if (C::kPlaces == 2 && !gather(tiles == 1, fix_before)) return false;
    const float inv = 1.0f / l;  // (see sv_prompt_tiles.cu)
    E* out = static_cast<E*>(a.out) + at.row * a.out_row + at.head * a.out_head;
#pragma unroll 1
    for (int d = 0; d < DP; d += 16) {
      uint32_t o[16];
      tc::tmem_load16(own_o + d, o);
      tc::wait_loads(o);
      if (held && d < a.dim) {
        float x[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(o[k]) * inv;
        if (out_vec32) {
#pragma unroll
          for (int h = 0; h < static_cast<int>(sizeof(E)) / 2; ++h) {
            uint32_t y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = sizeof(E) == 4 ? __float_as_uint(x[(8 * h + k) & 15]) : floats_to_bf16x2(x[2 * k], x[2 * k + 1]);
            tc::store_32(out + d + 8 * h, y);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) put_value(out + d + k, x[k]);
        }
      }
      __syncwarp();
    }
    const int dirty = *const_cast<const volatile int*>(&it.dirty);
    if (dirty != 0) {
      sum_rest<E>(a, it, tpt, dirty, sh.rest[quarter]);
      if (held) add_rest<kKeys, E>(a, it, tpt, token, out, sh.rest[quarter]);
    }
    if (held && a.lse) a.lse[at.row * a.heads + at.head] = (m + log2f(l)) * 0.69314718055994530942f;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) sh.finished[quarter] = items + 1;
    warp_arrive(sh.item_free[items % kItems]);
  }
}

static_assert(Config<256, float>::kShared + sizeof(Shared) <= 227 * 1024, "shared memory of a block");

template <int DP, typename E>
__global__ void __launch_bounds__(kThreads, 1) prompt_split_kernel(const __grid_constant__ PromptView a, int tpt, float f, int vec, int out_vec32) {
  using C = Config<DP, E>;
  extern __shared__ uint8_t raw[];
  __shared__ Shared sh;
  const uint32_t at = tc::smem_address(raw);
  uint8_t* queries = raw + ((at + 1023u & ~1023u) - at);
  uint8_t* stages = queries + C::kQueryBytes;
  const int warp = threadIdx.x >> 5, tid = threadIdx.x;
  if (tid == 0) {
    sh.gave_up = 0;
    sh.claimed = 0;
    for (int i = 0; i < kSoftmaxWarps; ++i) sh.finished[i] = 0;
    for (int i = 0; i < kItems; ++i) {
      tc::barrier_init(tc::smem_address(&sh.item_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.item_free[i]), kSoftmaxWarps + kLoadWarps + 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      tc::barrier_init(tc::smem_address(&sh.full[i]), kLoadWarps);
      tc::barrier_init(tc::smem_address(&sh.free[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::barrier_init(tc::smem_address(&sh.s_full[i]), 1);
      tc::barrier_init(tc::smem_address(&sh.p_ready[i]), kSoftmaxWarps);
    }
    tc::barrier_init(tc::smem_address(&sh.q_full), kLoadWarps);
    tc::barrier_init(tc::smem_address(&sh.q_free), 1);
    tc::barrier_init(tc::smem_address(&sh.sums_full), 1);
    tc::barrier_init(tc::smem_address(&sh.sums_free), kSoftmaxWarps);
    tc::barrier_init(tc::smem_address(&sh.last), 1);
    tc::barrier_init(tc::smem_address(&sh.answer), 1);
    tc::publish_shared();
  }
  wait_for_stream();  // (before tensor memory is taken, which the launch before may still need)
  if (warp == 0) tc::tmem_alloc(tc::smem_address(&sh.tmem), 512);
  sort_sequences(a, sh.sequences, tpt, kThreads);
  if (blockIdx.x == 0) flag_lengths(a, kThreads);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = sh.tmem;
  if (warp < kSoftmaxWarps) {
    tc::registers_up<kSoftmaxRegisters>();
    softmax_role<DP, E>(a, tpt, f, sh, tmem, out_vec32);
  } else if (warp < kSoftmaxWarps + kLoadWarps) {
    tc::registers_down<kLoadRegisters>();
    load_role<DP, E>(a, tpt, sh, queries, stages, vec);
  } else {
    tc::registers_down<kOtherRegisters>();
    if (warp == kSoftmaxWarps + kLoadWarps) {
      if (tc::elected()) {
        product_role<DP, E>(sh, tc::smem_address(queries), tc::smem_address(stages), tmem);
        // products in flight end before the memory that they use is given up
        int unused = 0;
        tc::products_arrive(tc::smem_address(&sh.last));
        tc::barrier_wait(tc::smem_address(&sh.last), 0, &unused, tc::kEndCycles);
      }
      __syncwarp();
    } else if (warp == kSoftmaxWarps + kLoadWarps + 1) {
      Finder finder{0, 0};
      Plans under{};
      if (!plan_role(a, tpt, sh, finder, under)) {
        // items that no other role knows of are spoilt here, those of an answer that is under way among them
        Item it;
        for (; finder.find<kKeys, 1>(a, sh.sequences, tpt, under.next, it); under.next += gridDim.x) spoil<E>(a, it, tpt, 1, tid & 31, 32);
        if (under.asked) {
          int unused = 0;
          const bool answered = tc::barrier_wait(tc::smem_address(&sh.answer), under.answers & 1, &unused, tc::kEndCycles);
          const int x = __all_sync(0xffffffffu, answered) ? tc::taken_block(tc::smem_address(&sh.block)) : -1;
          if (x >= 0)
            for (long long index = x; finder.find<kKeys, 1>(a, sh.sequences, tpt, index, it); index += gridDim.x) spoil<E>(a, it, tpt, 1, tid & 31, 32);
        }
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (sh.gave_up) {
    int done = sh.finished[0];
    for (int i = 1; i < kSoftmaxWarps; ++i) done = min(done, sh.finished[i]);
    for (int k = done; k < sh.claimed; ++k) spoil<E>(a, sh.item[k % kItems], tpt, 1, tid, kThreads);
  }
  if (warp == 0) tc::tmem_free(tmem, 512);
}

template <int DP, typename E>
sv_status launch(const PromptView& a, cudaStream_t stream) {
  using C = Config<DP, E>;
  static FuncAttrCache attr;
  const auto kernel = prompt_split_kernel<DP, E>;
  if (!attr.ensure(reinterpret_cast<const void*>(kernel), C::kShared, false)) return SV_ERR_CUDA;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  const int64_t strides = a.q_row | a.q_head | a.k_row | a.k_head | a.v_row | a.v_head;
  const bool vec = at % 16 == 0 && strides % 4 == 0;
  const bool out_vec32 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && (a.out_row | a.out_head) * sizeof(E) % 32 == 0;
  const int tpt = kRows / a.group;
  if (launch_early(kernel, dim3(prompt_blocks(a, tpt)), dim3(kThreads), C::kShared, stream, a, tpt, a.scale * 1.44269504088896340736f, static_cast<int>(vec),
                   static_cast<int>(out_vec32)) != cudaSuccess)
    return SV_ERR_CUDA;
  note_launch(stream);
  return SV_OK;
}

template <typename E>
sv_status launch(const PromptView& a, cudaStream_t stream) {
  return a.dim <= 64 ? launch<64, E>(a, stream) : a.dim <= 128 ? launch<128, E>(a, stream) : launch<256, E>(a, stream);
}

}  // namespace

sv_status prompt_split(const PromptView& a, sv_dtype dtype, cudaStream_t stream) {
  return dtype == SV_BF16 ? launch<uint16_t>(a, stream) : launch<float>(a, stream);
}

}  // namespace sv
