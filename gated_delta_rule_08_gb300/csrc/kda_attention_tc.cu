// Attention over a paged cache for many rows a key head, on the tcgen05 tensor cores: prompts, and trees of drafted
// tokens of more rows than a warp MMA has.
//
// The mathematics is that of kda_attention.cu.  A work item is 256 rows of a request and key head, in two halves of 128
// (an MMA's rows: TMEM lanes), of whole tokens each.  For every tile of 128 keys
//   S_h [128 x 128] = Q_h K^T      Q, K in shared memory
//   P_h             = weights of S_h, bf16, written over S_h in TMEM
//   O_h [128 x d]  += P_h V        A operand P in TMEM, V as it lies in the cache (MN-major)
// The halves alternate: while one's four softmax warps work, the tensor cores multiply for the other.  A thread
// has a row of its own, so that maxima and sums need no exchange.  PV of a tile is issued before the next QK of
// its half: one commit tells a softmax warp that its scores are there and that O is at rest, so that it may rescale O
// itself in the rare case that a row's maximum has passed its reference by 2^8 (no warps of their own for that).
//
// Keys and values come by TMA, a box for each block of the cache (or 128 tokens of it), into one ring of tiles, K and V
// in turn.  A tile is made of boxes, not of 128 consecutive keys: the sinks' boxes and the window's lie in it side by
// side, which saves a tile for the sinks and most of one for a window that starts inside one.  Only tiles with a key
// that some row does not see look at masks.  Values that no row sees may be anything (unwritten memory, NaN) and meet
// weights of 0: a warp of its own clears them before such a tile is multiplied.
//
// Roles wait for phases of barriers by parity, so no phase may complete before all that wait for the one before it have
// seen that.  Rings and hand-overs that are answered see to it by themselves; `unclear` and `o_done` are told where it has to be.
//
// Warps: 0-3 and 4-7 softmax of the halves, 8 copies, 9 and 10 the halves' MMAs, 11 clears.  The two MMA warps take turns
// at the tensor cores (without turns both halves fall into step, and softmax and products no longer overlap: 2.2 ms
// instead of 1.5 for the first case below), and each passes its turn on before its QK, because that takes
// some 500 clocks.  A CTA an SM walks over items (a request's last tiles first, which have the most keys), which the
// copy warp looks up ahead and hands to the others; few items, and trees: a cluster of CTAs shares the keys of one and joins through distributed
// shared memory, cut by the request's own length, the longest first.
//
// Measured on GB300 (bf16, 32 heads of 8 key heads, d = 128): 16384 tokens, all keys: 1.57 ms by itself (1.38
// PFLOP/s of the pairs a token sees; 1.62 ms once the power limit takes hold); 8192 tokens, a window of 1024 and 4 sinks:
// 145 us (0.88 PFLOP/s); 32 trees of 64 drafted tokens over 500 to 16000: 185 us (3.5 TB/s).  Five parts of prompts, up to
// 2000 tokens over 9000, 20 heads of 4, d = 64, a window of 4096: 105 us.
// Bound in long prompts by a half's chain from scores to scores: softmax 1250 clocks (of them 700 exponentials, rounding and
// stores), PV 500 to 600, QK 650 to 700, two hand-overs of 150; the tensor cores are busy for 2300 of the 2800 clocks that
// the halves need for a tile.  A window's items have ten tiles and 6 to 8 thousand clocks between them (sums
// read and stored, the next queries).  Trees: a CTA starts and joins in 15 us, in which it reads nothing.
#include "kda_attention.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kThreads = 384;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kClearWarp = 11;  // (MMAs: two warps)
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;  // (208 and 88: 2 to 6 % slower)
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "registers of the launch");
constexpr int kHalf = 128, kKeys = 128;
constexpr float kLowest = -3.402823466e38f;  // below every score: a weight relative to it is 0 for a masked key
constexpr float kSlack = 8.f;
constexpr float kGone = -1.f;                 // for a sum of weights: the CTA has given up
constexpr uint32_t kTmS = 0, kTmO = 256;      // TMEM columns: S (and P) of the halves, O of the halves

template <int D>
struct Layout {
  static constexpr int kParts = D / 64;
  static constexpr uint32_t kPart = kKeys * 128;             // 64 values of 128 rows
  static constexpr uint32_t kTile = kParts * kPart;
  static constexpr int kStages = 5 * (2 / kParts);           // (four: long prompts 2 to 4 % slower)
  static constexpr uint32_t kRing = 2 * kTile;               // behind Q of the halves
  static constexpr uint32_t kBar = kRing + kStages * kTile;
  static constexpr uint32_t kItems = kBar + 512;
  static constexpr uint32_t kSmem = kItems + 1024 + 1024;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  static_assert((2 * kStages + 19 + 8) * 8 + kMostOrdered <= 512, "barriers");
  static_assert(256 * D * 4 <= kStages * kTile, "a split item's sums take the ring's place");
};

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rd, ra, rb;\n"
      " mov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void tma_load_rows(void* dst, const CUtensorMap* map, int x, int head, int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(head), "r"(token), "r"(smem_u32(bar))
      : "memory");
}
// 32 bytes of a row, at once where the output begins on 32 bytes (a sector of L2; its rows are multiples of that).
__device__ __forceinline__ void store32(void* p, const uint32_t (&u)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    static_cast<uint4*>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}
__device__ __forceinline__ void tma_prefetch_rows(const CUtensorMap* map, int x, int head, int token) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(head), "r"(token)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_box(const CUtensorMap* map, int x, int token, int head, int block) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(map), "r"(x), "r"(token), "r"(head),
               "r"(block)
               : "memory");
}
// Waits of a whole warp (branches are on votes, so that it stays together), with a limit of half a second to a second, or
// none at all in the variant that gives up.  hold() leaves the waiting to the hardware; poll() is for the MMA warp, which all
// others wait for (a suspended warp comes back some hundreds of clocks late).  Both are kept small: they are inlined many
// times, and the warps' loops share an instruction cache.
struct Waiter {
  volatile int* abort_flag;
  bool give_up;
  __device__ __forceinline__ bool hold(uint64_t* bar, uint32_t parity) const {
    const uint32_t tries = give_up ? 0u : kPausedTries;
#pragma unroll 1
    for (uint32_t i = 0; i < tries; ++i) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
      pause_after(i);
    }
    *abort_flag = 1;
    return false;
  }
  __device__ __forceinline__ bool poll(uint64_t* bar, uint32_t parity) const {
    const uint32_t tries = give_up ? 0u : kPolls;
#pragma unroll 1
    for (uint32_t i = 0; i < tries; ++i) {
      if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
      if (i >= kQuickPolls) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
        __nanosleep(1000);
      }
    }
    *abort_flag = 1;
    return false;
  }
  static constexpr uint32_t kQuickPolls = 16384, kPolls = kQuickPolls + 700000;
};

struct QMap {
  CUtensorMap q;
};

// The first key of 16-key group g of tile j, or -1 past the last box.
__device__ __forceinline__ int group_key(const Span& s, int j, int g, int box_shift) {
  const int key = j * kKeys + g * 16, box = key >> box_shift;
  return box < s.boxes ? box_key(s, box, box_shift) + (key & ((1 << box_shift) - 1)) : -1;
}
// Keys by their place in the item's tiles: the sinks' boxes come first, as they lie in the cache; from then on the place
// of a key is the key less this.
__device__ __forceinline__ int place_shift(const Span& s, int box_shift) { return (s.first_box - s.sink_boxes) << box_shift; }
// Whether some row of `rows` may see a key of tile j (a span's keys from lo to hi, and the sinks up to hi).
__device__ __forceinline__ bool tile_seen(const Params& p, const Span& boxes, const Span& rows, int j, int box_shift) {
  const int shift = place_shift(boxes, box_shift), first = j * kKeys;
  return (first < rows.hi + 1 - shift && first + kKeys > rows.lo - shift) || first < min(p.sinks, rows.hi + 1);
}
// Whether tile j may hold keys that no row of the item sees (of drafted tokens, those that no mask names).
template <bool TREES>
__device__ __forceinline__ bool unclean(const Params& p, const Tile& t, const Span& s, int j, int box_shift) {
  const int shift = place_shift(s, box_shift), first = j * kKeys;
  return first < s.lo - shift || first + kKeys > (TREES && p.mask ? t.before : s.hi + 1) - shift;
}
// Bits [a, b) of 32.
__device__ __forceinline__ uint32_t bits(int a, int b) {
  const uint32_t below_a = a <= 0 ? 0u : a >= 32 ? ~0u : (1u << a) - 1u, below_b = b <= 0 ? 0u : b >= 32 ? ~0u : (1u << b) - 1u;
  return below_b & ~below_a;
}
// Trees: whether some row of the tile sees one of the keys [key, key + n), a box of its span (one warp together, each lane a
// box of its own).
__device__ __forceinline__ bool box_used(const Params& p, const Tile& t, const Span& s, int key, int n) {
  const int a = p.by_G.div(t.first), b = a + p.by_G.div(t.rows);
  bool used = key < t.before && (s.lo < t.before || key < p.sinks);
#pragma unroll 1
  for (int w = 0; w * 64 < t.tokens; ++w) {
    const uint64_t named = named_word(p, t, a, b, w);
    const int x = key - t.before - 64 * w, y = min(x + n, t.tokens - 64 * w);
    used |= ((uint32_t)named & bits(x, y)) != 0 || ((uint32_t)(named >> 32) & bits(x - 32, y - 32)) != 0;
  }
  return used;
}
// Which keys of tile j a row sees, a bit each.
__device__ __forceinline__ uint4 row_mask(const Params& p, const Tile& t, const Span& s, const Row& r, int j, int box_shift) {
  const int shift = place_shift(s, box_shift), first = j * kKeys;
  const int sinks = min(p.sinks, r.hi + 1) - first, lo = r.lo - shift - first, hi = r.hi + 1 - shift - first;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bits(lo - 32 * i, hi - 32 * i) | bits(0, sinks - 32 * i);
  if (r.mask && first + kKeys > t.before - shift) {
#pragma unroll 1
    for (int g = 0; g < 8; ++g) {
      const int key = group_key(s, j, g, box_shift);
      const uint32_t see = key < 0 ? 0u : seen16(p, t, r, key) << (16 * (g & 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] |= i == g / 2 ? see : 0u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The tiles, if any, that hold 128 consecutive keys of which every row of the span sees all.
struct Plain {
  int first, end;
};
__device__ __forceinline__ Plain plain_tiles(const Span& boxes, const Span& rows, int box_shift) {
  // tile j's first key, from the first after the sinks' boxes on
  const int shift = place_shift(boxes, box_shift);
  const int first = max((boxes.sink_boxes << box_shift) + kKeys - 1, rows.all_lo - shift + kKeys - 1) / kKeys;
  return {first, max(first, (rows.all_hi + 1 - shift) / kKeys)};
}
// An item as every role sees it: the copy warp looks them up, one ahead, and hands them over in shared memory.
struct Item {
  int have;              // 0: there are no more
  Tile t;
  int tile0, tile1;      // this CTA's tiles
  Span span, half[2];    // of both halves (the boxes), and of each
  Plain plain, half_plain[2];
};
constexpr int kItems = 4;  // in shared memory, so that the copies need not wait for the other roles
static_assert(kItems * sizeof(Item) <= 1024, "items in shared memory");
// a value that is the same in all lanes, as one that the compiler knows to be
__device__ __forceinline__ int same(int x) { return __reduce_max_sync(0xffffffffu, x); }

// SPLIT: an item a cluster, whose p.split CTAs share its keys; else a CTA walks over items, which are not trees'.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
attention_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ QMap qmap, const Params p, const int box_shift) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = aligned_smem(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar);
  uint64_t* empty = full + L::kStages;
  uint64_t* q_full = empty + L::kStages;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_full + 2;   // [2] scores there, O at rest
  uint64_t* p_ready = q_full + 14;  // [2][2] weights of half the keys written
  uint64_t* o_done = q_full + 6;   // [2] the item's products complete (split: both halves')
  uint64_t* cleared = q_full + 8;  // a tile's values cleared
  uint64_t* unclear = q_full + 9;  // ... have landed, and both MMA warps know of the tile cleared before
  uint64_t* turn = q_full + 10;    // [2] the half's turn at the tensor cores
  uint64_t* bar_fin = q_full + 12;
  uint64_t* item_full = q_full + 18;   // [kItems] an item handed over
  uint64_t* item_empty = item_full + kItems;  // ... and done with, by the warps of the other roles
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(item_empty + kItems);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint8_t* order = reinterpret_cast<uint8_t*>(tmem_slot + 2);  // [kMostOrdered]
  Item* items = reinterpret_cast<Item*>(sm + L::kItems);
  // reference and sum of weights of 256 rows, in Q's place once the item's products are done (SPLIT)
  float2* sums = reinterpret_cast<float2*>(sm);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = SPLIT ? (int)(blockIdx.x % p.split) : 0;
  int split = 1;
  const int G = p.G, half_rows = p.half_rows, span_tokens = p.by_G.div(half_rows);  // of a half
  griddep_launch_dependents();
  griddep_wait();
  if (p.cu != nullptr && !offsets_within(p.cu, p.N, p.T)) {
    if (tid == 0) atomicOr(p.err, KDA_DEVERR_BAD_SEQLENS);
    return;
  }
  // Items of this CTA: all warps look up the first, the copy warp the others.
  Walk walk;
  if (SPLIT && p.ordered) {
    order_by_length(p.lengths, p.N, order);
    __syncthreads();
    walk.order = order;
  }
  int at = SPLIT ? blockIdx.x / p.split : blockIdx.x;
  const int step = SPLIT ? 0x40000000 : gridDim.x;
  auto next = [&](Item& it) {
    while (true) {
      if (at < 0 || !locate(p, 2 * half_rows, p.by_item, at, walk, it.t)) return false;
      at += step;  // (a second one of a split item's passes 2^31 or the last item)
      if (it.t.rows > 0) break;
    }
    const int a = p.by_G.div(it.t.first);
    it.span = span_of(p, it.t, a, a + p.by_G.div(it.t.rows), box_shift);
    const int tiles = ((it.span.boxes << box_shift) + kKeys - 1) / kKeys;
    if (SPLIT) split = parts_of(p, tiles);
    it.tile0 = SPLIT ? (int)((int64_t)tiles * rank / split) : 0;
    it.tile1 = SPLIT ? (int)((int64_t)tiles * (rank + 1) / split) : tiles;
    it.plain = plain_tiles(it.span, it.span, box_shift);
    for (int h = 0; h < 2; ++h) {
      const int first = a + h * span_tokens, last = min(first + span_tokens, a + p.by_G.div(it.t.rows));
      it.half[h] = first < last ? span_of(p, it.t, first, last, box_shift) : it.span;
      it.half_plain[h] = plain_tiles(it.span, it.half[h], box_shift);
    }
    return true;
  };
  Item coming;
  bool have = next(coming);
  if (SPLIT && (!have || rank >= split)) return;
  coming.have = have;
  if (warp == kCopyWarp && lane == 0) items[0] = coming;
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int h = 0; h < 2; ++h) {
      mbar_init(&s_full[h], 1);
      mbar_init(&p_ready[2 * h], 4);
      mbar_init(&p_ready[2 * h + 1], 4);
      mbar_init(&turn[h], 1);
      mbar_init(&o_done[h], SPLIT ? 2 : 1);
    }
    mbar_init(cleared, 1);
    mbar_init(unclear, 2);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], kThreads / 32 - 1);
    }
    mbar_init(bar_fin, 2);
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const Waiter w{abort_flag, p.waits == kWaitsGiveUp};
  bool ok = true;
  int64_t issued = 0, q_issued = 0;  // copies started (copy warp)
  // For the other roles: item n; done with it, on to the next.
  auto wait_item = [&](int n) { ok = w.hold(&item_full[n % kItems], (uint32_t)(n / kItems & 1)); };
  auto advance = [&](int& n) {
    warp_arrive(&item_empty[n % kItems]);
    wait_item(++n);
  };

  if (warp < 8) {
    // ======================== softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int h = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t ts = tmem_lane(tmem, warp) + kTmS + 128 * h, to = tmem_lane(tmem, warp) + kTmO + 128 * h;
    uint32_t seen = 0;  // scores so far: the barriers' phase
    int n = 0;
    wait_item(n);
    while (ok && items[n % kItems].have) {
      const Item& it = items[n % kItems];
      const int rows = min(half_rows, it.t.rows - h * half_rows);
      const bool live = row < rows;
      const int r = it.t.first + h * half_rows + (live ? row : 0);  // in the request
      float m = kLowest, l = 0.f;
      bool any = false;
      if (rows > 0) {
        const Span& span = it.half[h];
        const Row keys = row_keys(p, it.t, p.by_G.div(r));
        const Plain plain = it.half_plain[h];
        const int tile1 = it.tile1;
#pragma unroll 1
        for (int j = it.tile0; j < tile1; ++j) {
          const bool whole = j >= plain.first && j < plain.end;
          if (!whole && !tile_seen(p, it.span, span, j, box_shift)) continue;
          ok = w.hold(&s_full[h], seen & 1);
          if (!ok) break;
          ++seen;
          tc_fence_after();
          float s[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, s[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) tmem_landed(s[i]);
          if (!whole) {
            const uint4 see = row_mask(p, it.t, it.span, keys, j, box_shift);
            const uint32_t words[4] = {see.x, see.y, see.z, see.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(words[i] >> e & 1)) s[i][e] = -INFINITY;
          }
          float t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            t[i] = s[i][0];
#pragma unroll
            for (int e = 1; e < 31; e += 2) t[i] = fmaxf(t[i], fmaxf(s[i][e], s[i][e + 1]));
            t[i] = fmaxf(t[i], s[i][31]);
          }
          const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * p.c;
          if (__any_sync(0xffffffffu, live && top > m + kSlack)) {
            const float n = fmaxf(m, top), f = ex2(m - n);
            m = n;
            l *= f;
            if (any) {
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                float o[32];
                tmem_ld32(to + i, o);
                tmem_landed(o);
                uint32_t u[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
                tmem_st32u(to + i, u);
              }
            }
          }
          any = true;
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 c2 = make_float2(p.c, p.c), m2 = make_float2(-m, -m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 x = fma2(make_float2(s[i][2 * e], s[i][2 * e + 1]), c2, m2);
              x.x = ex2(x.x);
              x.y = ex2(x.y);
              sum[e & 1] = add2(sum[e & 1], x);
              // to bf16, what the tensor cores take: half a step, 2^-8 at most, of each weight, at random in a sum of many
              u[e] = pack_bf2(x.x, x.y);
            }
            tmem_st16u(ts + 16 * i, u);
            if (i == 1) {  // the first half of the keys can be multiplied
              tmem_wait_st();
              tc_fence_before();
              warp_arrive(&p_ready[2 * h]);
            }
          }
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(&p_ready[2 * h + 1]);
        }
      }
      if (!ok) break;
      ok = w.hold(&o_done[h], (uint32_t)(n & 1));
      if (!ok) break;
      tc_fence_after();
      if (SPLIT && split > 1) {
        // sums into the ring (all its tiles have been read), pieces of 16 bytes permuted by the row
        const int rr = h * kHalf + row;
        uint8_t* dst = sm + L::kRing + (uint32_t)rr * (D * 4);
#pragma unroll 1
        for (int i = 0; i < D; i += 32) {
          float o[32];
          if (any) {
            tmem_ld32(to + i, o);
            tmem_landed(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.f;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(dst + (((i + e) / 4 ^ (rr & (D / 4 - 1))) << 4)) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        sums[rr] = make_float2(m, l);
        break;  // one item
      }
      if (rows > 0) {
        const float inv = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing is zero (a NaN stays one)
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        const int tok = p.by_G.div(r);
        __nv_bfloat16* dst = p.out + ((int64_t)(it.t.t0 + tok) * p.H + (it.t.head * G + r - tok * G)) * D;
#pragma unroll
        for (int i = 0; i < D; i += 64) {
          float o[2][32];
          if (any) {
            tmem_ld32(to + i, o[0]);
            tmem_ld32(to + i + 32, o[1]);
            tmem_landed(o[0]);
            tmem_landed(o[1]);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[0][e] = o[1][e] = 0.f;
          }
          if (live) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float* x = &o[k / 2][k % 2 * 16];
              uint32_t u[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) u[e] = pack_bf2(x[2 * e] * inv, x[2 * e + 1] * inv);
              store32(dst + i + 16 * k, u, wide);
            }
          }
          __syncwarp();
        }
        tc_fence_before();  // O is read before the next item's weights are told
      }
      if (SPLIT) break;
      advance(n);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kCopyWarp) {
      // ======================== copies
      int n = 0;
      warp_arrive(&item_full[0]);
      while (ok && have) {
        const Item it = coming;
        auto copy_q = [&]() {
          if (q_issued > 0) ok = w.hold(q_empty, (uint32_t)((q_issued - 1) & 1));
          if (!ok) return;
          if (lane == 0) {
            const int halves = it.t.rows > half_rows ? 2 : 1;
            mbar_arrive_expect_tx(q_full, (uint32_t)(halves * L::kParts * half_rows * 128));
            for (int h = 0; h < halves; ++h)
              for (int i = 0; i < L::kParts; ++i)
                tma_load_rows(sm + h * L::kTile + i * L::kPart, &qmap.q, 64 * i, it.t.head * G,
                              it.t.t0 + p.by_G.div(it.t.first) + h * span_tokens, q_full);
          }
          __syncwarp();
          ++q_issued;
        };
        auto look_ahead = [&]() {
          have = next(coming);
          ++n;
          if (n >= kItems) ok = w.hold(&item_empty[n % kItems], (uint32_t)((n / kItems - 1) & 1));
          if (!ok) return;
          coming.have = have;
          if (lane == 0) items[n % kItems] = coming;
          warp_arrive(&item_full[n % kItems]);
          if (!have) return;
          // Towards L2, as all CTAs come to their next items at about the same time: its queries, and its last keys and
          // values (of a prompt: those that no item before it has read).
          const int part = lane % L::kParts, i = lane / L::kParts;
          if (i < 2 && i * half_rows < coming.t.rows)
            tma_prefetch_rows(&qmap.q, 64 * part, coming.t.head * G, coming.t.t0 + p.by_G.div(coming.t.first) + i * span_tokens);
          const int box = coming.span.boxes - 1 - i;
          if (i < kKeys >> box_shift && box >= 0) {
            const int key = box_key(coming.span, box, box_shift);
            const int id = p.tables[(int64_t)coming.t.n * p.max_blocks + (key >> p.shift)];
            if ((unsigned)id < (unsigned)p.num_blocks) {
              tma_prefetch_box(&maps.k, 64 * part, key & ((1 << p.shift) - 1), coming.t.head, id);
              tma_prefetch_box(&maps.v, 64 * part, key & ((1 << p.shift) - 1), coming.t.head, id);
            }
          }
          __syncwarp();
        };
        if (it.tile0 == it.tile1) {
          copy_q();
          look_ahead();
        }
        const int32_t* table = p.tables + (int64_t)it.t.n * p.max_blocks;
        const int per = kKeys >> box_shift;  // boxes of a tile, at most 8
        // a lane has a box of four tiles at a time
        auto block_ids = [&](int j) {
          const int box = j * per + lane, key = box_key(it.span, box, box_shift);
          const bool mine = lane < 4 * per && box < it.span.boxes && box < it.tile1 * per;
          int id = mine ? table[key >> p.shift] : 0;
          // by some row: of a tree's boxes, those that end before the drafted tokens are
          const bool used = !SPLIT || !p.mask || !__any_sync(0xffffffffu, mine && key + (1 << box_shift) > it.t.before) ||
                            box_used(p, it.t, it.span, key, 1 << box_shift);
          if (mine && (!used || (unsigned)id >= (unsigned)p.num_blocks)) {
            if (used) atomicOr(p.err, KDA_DEVERR_BAD_SLOT);
            id = p.num_blocks;  // reads as zeros
          }
          return id;
        };
        int ids = block_ids(it.tile0), next_ids = block_ids(it.tile0 + 4);
#pragma unroll 1
        for (int j = it.tile0; j < it.tile1 && ok; ++j) {
          const int in4 = (j - it.tile0) & 3;
          if (in4 == 0 && j > it.tile0) {
            ids = next_ids;
            next_ids = block_ids(j + 4);
          }
          const int mine = j * per + lane;  // box of this lane
          const int block = __shfl_sync(0xffffffffu, ids, (in4 * per + lane) & 31);
          const int boxes = min(per, it.span.boxes - j * per);
          const int token = box_key(it.span, mine, box_shift) & ((1 << p.shift) - 1);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (kv == 1 && j == it.tile0) {  // the first keys have not waited for the item before to leave Q
              copy_q();
              if (!ok) break;
            }
            const int s = (int)(issued % L::kStages);
            if (issued >= L::kStages) ok = w.hold(&empty[s], (uint32_t)((issued / L::kStages - 1) & 1));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)boxes * (uint32_t)(L::kParts * 128) << box_shift);
            __syncwarp();
            if (lane < boxes) {
              uint8_t* dst = sm + L::kRing + s * L::kTile + ((uint32_t)lane << box_shift) * 128u;
#pragma unroll
              for (int i = 0; i < L::kParts; ++i)
                tma_load_box(dst + i * L::kPart, kv ? &maps.v : &maps.k, 64 * i, token, it.t.head, block, &full[s]);
            }
            __syncwarp();
            ++issued;
          }
          if (ok && j == it.tile0) look_ahead();
        }
      }
    } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ======================== MMAs, a warp for each half
      // What the loops go by passes through votes and reductions, which the compiler knows to be the same in all lanes:
      // descriptors are then formed in uniform registers (from vector registers an MMA takes 100 clocks to issue).
      const bool leader = lane == 0;
      const int h = warp == kMmaWarp ? 0 : 1;
      constexpr uint32_t id_s = idesc_bf16_f32(128, kKeys, false, false), id_o = idesc_bf16_f32(128, D, false, true);
      const uint64_t d_q = smem_desc_sw128(smem_u32(sm + h * L::kTile), 16, 1024);
      const uint64_t d_k = smem_desc_sw128(smem_u32(sm + L::kRing), 16, 1024);
      const uint64_t d_v = smem_desc_sw128(smem_u32(sm + L::kRing), L::kPart, 1024);
      const uint32_t t_s = tmem + kTmS + 128 * h, t_o = tmem + kTmO + 128 * h;
      const bool works = !(p.waits == kFirstCtaStalls && blockIdx.x == 0);
      int stage = 0;  // of the next tile in the ring, and its phase
      uint32_t phase = 0, weights = 0, clears = 0, q_used = 0, turns = h ^ 1;  // (half 0 has the first turn)
      int n = 0;
      wait_item(n);
      while (works && ok && same(items[n % kItems].have)) {
        const Item& it = items[n % kItems];
        const int tile0 = same(it.tile0), tile1 = same(it.tile1);
        const bool rows = same(it.t.rows) > h * half_rows;
        const int plain0 = same(it.plain.first), plain1 = same(it.plain.end);
        const Span& span = it.half[h];
        ok = w.poll(q_full, q_used & 1);
        q_used ^= 1;
        bool pending = false, begun = false, clean = true, left = false;  // weights to come, O begun, V as it came, Q given up
        int v_stage = 0;
        uint32_t v_phase = 0;
#pragma unroll 1
        for (int j = tile0; j <= tile1; ++j) {
          if (!ok) break;
          const bool more = j < tile1;
          bool active = false, next_clean = true;
          if (more) {
            active = rows;
            if (j < plain0 || j >= plain1) {
              active = rows && __any_sync(0xffffffffu, tile_seen(p, it.span, span, j, box_shift));
              next_clean = !__any_sync(0xffffffffu, unclean<SPLIT>(p, it.t, it.span, j, box_shift));
            }
            ok = w.poll(&full[stage], phase);
            if (!ok) break;
          }
          if (j > tile0) {
            ok = clean ? w.poll(&full[v_stage], v_phase) : w.poll(cleared, clears);
            if (!ok) break;
            clears ^= clean ? 0 : 1;
          }
          ok = w.poll(&turn[h], turns);
          if (!ok) break;
          turns ^= 1;
          if (pending) {
            const uint64_t at = desc_add(d_v, v_stage * L::kTile);
            ok = w.poll(&p_ready[2 * h], weights);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kKeys / 32; ++i)
              mma_bf16_ts_by(leader, t_o, t_s + 8 * i, desc_add(at, i * 2048), id_o, i > 0 || begun);
            ok = w.poll(&p_ready[2 * h + 1], weights);
            if (!ok) break;
            weights ^= 1;
            tc_fence_after();
#pragma unroll
            for (int i = kKeys / 32; i < kKeys / 16; ++i)
              mma_bf16_ts_by(leader, t_o, t_s + 8 * i, desc_add(at, i * 2048), id_o, true);
            begun = true;
          }
          const uint64_t at = desc_add(d_k, stage * L::kTile);
          warp_arrive(&turn[h ^ 1]);  // with MMAs still to issue: the turn takes some 500 clocks to pass
          if (active) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              mma_bf16_ss_by(leader, t_s, desc_add(d_q, (i >> 2) * L::kPart + (i & 3) * 32),
                             desc_add(at, (i >> 2) * L::kPart + (i & 3) * 32), id_s, i > 0);
            mma_commit_by(leader, &s_full[h]);
          }
          if (j + 1 >= tile1 && !left) {  // Q has been read
            mma_commit_by(leader, q_empty);
            left = true;
          }
          if (j > tile0) mma_commit_by(leader, &empty[v_stage]);
          pending = active;
          clean = next_clean;
          if (more) {
            mma_commit_by(leader, &empty[stage]);
            if (++stage == L::kStages) {
              stage = 0;
              phase ^= 1;
            }
            v_stage = stage;
            v_phase = phase;
            if (++stage == L::kStages) {
              stage = 0;
              phase ^= 1;
            }
            if (!clean) {
              // Both warps tell of the tile, each past its wait for the tile cleared before: `cleared` is then never two
              // phases ahead of a warp, which would take it for the one that it waits for not to have come.
              if (h == 0) {
                ok = w.poll(&full[v_stage], v_phase);
                if (!ok) break;
              }
              warp_arrive(unclear);
            }
          }
        }
        if (!ok) break;
        if (!SPLIT && n > 0) {
          // All roles are done with the item before: its o_done has been seen, and does not move on by two phases.  (They
          // mostly have been for long; an item without keys, or without rows for this half, asks nothing of them.)
          ok = w.poll(&item_empty[(n - 1) % kItems], (uint32_t)((n - 1) / kItems & 1));
          if (!ok) break;
        }
        mma_commit_by(leader, &o_done[h]);
        if (SPLIT) {
          mma_commit_by(leader, &o_done[h ^ 1]);
          break;
        }
        advance(n);
      }
    } else if (warp == kClearWarp) {
      // ======================== values that no row sees
      // (told of a tile's arrival by the MMA warps, which follow the ring; a wait that skips phases would mistake them)
      uint32_t used = 0, tiles = 0;
      int n = 0;
      wait_item(n);
      while (ok && items[n % kItems].have) {
        const Item& it = items[n % kItems];
        const bool drafted = SPLIT && p.mask && it.tile1 * kKeys > it.t.before - place_shift(it.span, box_shift);  // in its tiles
        const int a = p.by_G.div(it.t.first);
        const uint64_t named = drafted ? named_by(p, it.t, a, a + p.by_G.div(it.t.rows)) : 0;
#pragma unroll 1
        for (int j = it.tile0; j < it.tile1 && ok; ++j, used += 2) {
          if (!unclean<SPLIT>(p, it.t, it.span, j, box_shift)) continue;
          const int s = (int)((used + 1) % L::kStages);
          ok = w.hold(unclear, tiles & 1);
          if (!ok) break;
          ++tiles;
          uint8_t* st = sm + L::kRing + s * L::kTile;
          // (lane g looks at group g)
          const int base = group_key(it.span, j, lane & 7, box_shift);
          const uint32_t seen = used16<SPLIT>(p, it.t, it.span, named, base < 0 ? 0 : base), keeps = base < 0 ? 0u : seen;
          for (int g = 0; g < 8; ++g) {
            const uint32_t keep = __shfl_sync(0xffffffffu, keeps, g);
            if (keep == 0xffffu) continue;
            for (int i = lane; i < 16 * 8 * L::kParts; i += 32) {
              const int r = i & 15, c = i >> 4;
              if (!(keep >> r & 1))
                *reinterpret_cast<uint4*>(st + (c >> 3) * L::kPart + row_chunk(16 * g + r, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_proxy_async_smem();
          warp_arrive(cleared);
        }
        if (SPLIT) break;
        advance(n);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // copies and MMAs that may still be under way are waited for, with a limit
    if (tid == kCopyWarp * 32) {
      if (q_issued > 0) mbar_wait(q_full, (uint32_t)((q_issued - 1) & 1));
      for (int64_t i = issued > L::kStages ? issued - L::kStages : 0; i < issued; ++i)
        mbar_wait(&full[i % L::kStages], (uint32_t)((i / L::kStages) & 1));
      atomicOr(p.err, KDA_DEVERR_WAIT_TIMEOUT);
    }
    if (tid == kMmaWarp * 32 || tid == (kMmaWarp + 1) * 32) {
      mma_commit(bar_fin);
      mbar_wait(bar_fin, 0);
    }
    __syncthreads();
  }
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  if (!SPLIT || split == 1) return;

  // the cluster's CTAs join: each a part of the rows
  if (*abort_flag && tid < 256) sums[tid] = make_float2(kLowest, kGone);
  cluster_sync();
  {
    const Tile& t = items[0].t;
    constexpr int kPieces = D / 8;  // a thread's eight values
    const int each = 256 / split;
    for (int i = tid; i < each * kPieces; i += kThreads) {
      const int rr = rank * each + i / kPieces, x = i % kPieces * 8;
      const int h = rr / kHalf, row = rr % kHalf, q = h * half_rows + row;
      if (row >= half_rows || q >= t.rows) continue;
      float m = kLowest, l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
      const uint8_t* src = sm + L::kRing + (uint32_t)rr * (D * 4);
      const uint32_t pa = (uint32_t)(x / 4 ^ (rr & (D / 4 - 1))) << 4, pb = (uint32_t)((x / 4 + 1) ^ (rr & (D / 4 - 1))) << 4;
      bool lost = false;
#pragma unroll 2
      for (int k = 0; k < split; k += 2) {  // (the loads of several parts under way at a time)
        const float2 s0 = ld_peer2(peer(sums + rr, k)), s1 = ld_peer2(peer(sums + rr, min(k + 1, split - 1)));
        const float4 a0 = ld_peer4(peer(src + pa, k)), b0 = ld_peer4(peer(src + pb, k));
        const float4 a1 = ld_peer4(peer(src + pa, min(k + 1, split - 1))), b1 = ld_peer4(peer(src + pb, min(k + 1, split - 1)));
        lost |= s0.y == kGone || s1.y == kGone;
        const float n = fmaxf(m, fmaxf(s0.x, s1.x)), f = ex2(m - n), f0 = ex2(s0.x - n), f1 = k + 1 < split ? ex2(s1.x - n) : 0.f;
        m = n;
        l = fmaf(f, l, fmaf(f0, s0.y, f1 * s1.y));
        a = f4_fma(f0, a0, f4_fma(f1, a1, make_float4(f * a.x, f * a.y, f * a.z, f * a.w)));
        b = f4_fma(f0, b0, f4_fma(f1, b1, make_float4(f * b.x, f * b.y, f * b.z, f * b.w)));
      }
      if (lost) continue;
      const float inv = l != 0.f ? 1.f / l : 0.f;
      const int r = t.first + q;
      *reinterpret_cast<uint4*>(p.out + ((int64_t)(t.t0 + p.by_G.div(r)) * p.H + t.head * G + p.by_G.mod(r)) * D + x) =
          make_uint4(pack_bf2(a.x * inv, a.y * inv), pack_bf2(a.z * inv, a.w * inv), pack_bf2(b.x * inv, b.y * inv),
                     pack_bf2(b.z * inv, b.w * inv));
    }
  }
  cluster_sync();  // no CTA leaves while another reads its memory
}

// CTAs that may share an item's keys, and the tiles for each at least: where items leave SMs idle, as many as there are SMs
// for, with two tiles each; else (trees: lengths differ from request to request) a few, with kMostTiles each (32 requests of 500
// to 16000 tokens, 16 / 32 / 64 tiles: 189 / 193 / 262 us; 8 of them: 110 / 77 / 123 us).
constexpr int kMaxSplit = 8, kMostTiles = 32, kMostCtas = 1024;
void split_of(int64_t items, int64_t keys, int sms, int* split, int* least) {
  *split = 1;
  *least = 2;
  while (*split < kMaxSplit && items * *split * 2 <= sms && keys > *split * 2 * kKeys) *split *= 2;
  if (items * 2 <= sms) return;
  *least = kMostTiles;
  while (*split < kMaxSplit && items * *split * 2 <= kMostCtas && keys > *split * kMostTiles * kKeys) *split *= 2;
}

template <int D, bool SPLIT>
cudaError_t launch_one(const Maps& maps, const QMap& qmap, const Params& p, int box_shift, unsigned grid, cudaStream_t st) {
  static DeviceOnce once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const cudaError_t e = once.run(dev, [] {
    cudaError_t f = cudaFuncSetAttribute(attention_tc_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::kSmem);
    if (f == cudaSuccess) f = cudaFuncSetAttribute(attention_tc_kernel<D, SPLIT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return f;
  });
  if (e != cudaSuccess) return e;
  TraceScope ts("kda_attention_tc", st);
  return launch_overlapped(attention_tc_kernel<D, SPLIT>, grid, kThreads, Layout<D>::kSmem, (unsigned)p.split, st, maps, qmap, p, box_shift);
}

template <int D>
cudaError_t launch(const AttentionArgs& a, Params p, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int box_shift = a.shift < 7 ? a.shift : 7, tokens = kHalf / p.G;
  p.half_rows = tokens * p.G;
  p.by_item = divisor(2 * p.half_rows);
  p.by_each = divisor((p.G + 2 * p.half_rows - 1) / (2 * p.half_rows));
  Maps maps;
  QMap qmap;
  if (!tensor_map_cache(&maps.k, a.k_cache, a.num_blocks, 1u << a.shift, a.Hkv, D, a.block_stride, a.token_stride, a.head_stride, 1u << box_shift) ||
      !tensor_map_cache(&maps.v, a.v_cache, a.num_blocks, 1u << a.shift, a.Hkv, D, a.block_stride, a.token_stride, a.head_stride, 1u << box_shift) ||
      !tensor_map_rows(&qmap.q, a.q, a.T, a.H, D, a.q_stride, (uint32_t)tokens, (uint32_t)p.G))
    return cudaErrorInvalidValue;
  const int64_t items = most_tiles(a, 2 * p.half_rows) * a.Hkv;
  if (a.tree_mask == nullptr && items > sms / 2) return launch_one<D, false>(maps, qmap, p, box_shift, (unsigned)(items < sms ? items : sms), st);
  split_of(items, most_keys(a, 2 * tokens), sms, &p.split, &p.least);
  p.ordered = a.N > 1 && a.N <= kMostOrdered && items * p.split > sms;
  return launch_one<D, true>(maps, qmap, p, box_shift, (unsigned)(items * p.split), st);
}

}  // namespace

cudaError_t attention_tc_launch(const AttentionArgs& a, cudaStream_t st) {
  return a.d == 64 ? launch<64>(a, params_of(a), st) : launch<128>(a, params_of(a), st);
}

}  // namespace kda
