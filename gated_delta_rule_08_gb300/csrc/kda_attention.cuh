// What the two attention kernels over a paged cache share: which request and rows a CTA works on, which keys its
// rows see, and the copies of the cache's boxes.
//
// The rows of a request and a key head are its (token, query head) pairs, row r = token r / G and head r % G of
// the G query heads that share the key head, so that a tile of rows reads each key once for all of them.
#pragma once

#include "kda_internal.h"
#include "kda_tc_common.cuh"
#include "kda_tma.h"

namespace kda {
namespace attn {

using namespace tcx;

struct Maps {
  CUtensorMap k, v;
};
// n / d for 0 <= n < 2^31 by a multiplication (d fixed by the launch): with 2^s >= d and m = floor(2^32 (2^s - d) / d) + 1
// it is (n + floor(n m / 2^32)) / 2^s, and the sum stays below 2^32.
struct Divisor {
  uint32_t m, s, d;
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi((uint32_t)n, m) + (uint32_t)n) >> s); }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * (int)d; }
};
inline Divisor divisor(int d) {
  uint32_t s = 0;
  while ((1u << s) < (uint32_t)d) ++s;
  return {(uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - (uint64_t)d)) / (uint64_t)d + 1), s, (uint32_t)d};
}
struct Params {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const int32_t* tables;
  const int32_t* lengths;
  const int32_t* cu;         // null: one token of each request
  const uint64_t* mask;      // null: causal
  int mask_words;
  __nv_bfloat16* out;
  int N;
  int64_t T;
  int H, Hkv, G;
  Divisor by_G, by_Hkv, by_each;  // by_each: tiles of a request of one token
  int half_rows;             // rows of half an item, and of an item (kda_attention_tc.cu)
  Divisor by_item;
  int shift, max_blocks, num_blocks, window, sinks;
  float c;                   // scale log2(e): scores are kept in log2
  unsigned int* err;
  int waits;                 // enum Waits
  int split;                 // CTAs (a cluster) that may share a tile's keys: those past parts_of() leave at once
  int ordered;               // take the requests by falling length
  int least;                 // boxes (tc: tiles) for each of them at least
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
// 4-D tiled copy of a box of the cache: 64 values from `x` on, tokens from `token` on, of a head and a block.
__device__ __forceinline__ void tma_load_box(void* dst, const CUtensorMap* map, int x, int token, int head, int block, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(token), "r"(head), "r"(block), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the same shared address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
// Loads and stores there.  (Between the cluster's barriers, which the compiler moves no memory access over; the loads
// themselves may overlap.)
__device__ __forceinline__ float2 ld_peer2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void st_peer2(uint32_t a, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(a), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st_peer4(uint32_t a, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Into how many parts (CTAs) a tile's keys are cut: a power of two that the host bounds and the request's length decides.
__device__ __forceinline__ int parts_of(const Params& p, int boxes) {
  int parts = 1;
  while (parts < p.split && boxes > parts * p.least) parts *= 2;
  return parts;
}

// Whether the offsets rise from 0 to at most T (all threads of the CTA).
__device__ __forceinline__ bool offsets_within(const int32_t* __restrict__ cu, int N, int64_t T) {
  bool bad = cu[0] != 0 || cu[N] > T;
  for (int i = threadIdx.x; i < N; i += blockDim.x) bad |= cu[i + 1] < cu[i];
  return !__syncthreads_or(bad);
}

// Tokens of a request: its tiles take some 0.2 s of a CTA of the kernel for many rows, and a role may wait for another one that
// long, out of half a second.  (The kernel for few rows has no such wait, but sizes decide between the two, and a request
// is not to be refused by one and answered by the other.)
constexpr int kMaxLength = 1 << 24;
// A tile of rows of one request and key head.
struct Tile {
  int n, head;         // request, key head
  int len, before;     // tokens in the cache; those before the new ones
  int t0, tokens;      // first new token in q, number of new tokens
  int first, rows;     // first row and number of rows of the tile (0: nothing to do)
};

// Walks the tiles of all requests in order, `per` rows a tile: item = (tile, key head).  A warp calls it
// with rising items; `base` and `tiles` keep its place.
struct Walk {
  int base = 0;     // request of lane 0
  int tiles = 0;    // tiles of the requests before it
  const uint8_t* order = nullptr;  // requests in the order to take them in, or null
};
// The requests by falling length, for tiles that start in order and take as long as their requests (all threads of the CTA,
// at most kMostOrdered requests; a barrier before the order is read).
constexpr int kMostOrdered = 64;
__device__ __forceinline__ void order_by_length(const int32_t* __restrict__ lengths, int N, uint8_t* order) {
  const int i = threadIdx.x;
  if (i >= N) return;
  const int n = lengths[i];
  int rank = 0;
  for (int j = 0; j < N; ++j) {
    const int m = lengths[j];
    rank += m > n || (m == n && j < i);
  }
  order[rank] = (uint8_t)i;
}
__device__ __forceinline__ bool locate(const Params& p, int per, Divisor by_per, int item, Walk& w, Tile& t) {
  const int lane = threadIdx.x & 31;
  const int tile = p.by_Hkv.div(item);
  t.head = item - tile * p.Hkv;
  int k;
  if (p.cu == nullptr) {
    const int i = p.by_each.div(tile);
    if (i >= p.N) return false;
    t.n = w.order ? w.order[i] : i;
    t.t0 = t.n;
    t.tokens = 1;
    k = tile - i * (int)p.by_each.d;
  } else {
    while (true) {
      if (w.base >= p.N) return false;
      const int i = w.base + lane, n = i < p.N && w.order ? w.order[i] : i;
      const int a = i < p.N ? p.cu[n] : 0, b = i < p.N ? p.cu[n + 1] : 0;
      int sum = by_per.div((b - a) * p.G + per - 1);  // (T H and a tile's rows are below 2^31 together)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      const int all = __shfl_sync(0xffffffffu, sum, 31);
      if (tile < w.tiles + all) {
        const unsigned over = __ballot_sync(0xffffffffu, w.tiles + sum > tile);
        const int src = __ffs(over) - 1;
        t.n = __shfl_sync(0xffffffffu, n, src);
        t.t0 = __shfl_sync(0xffffffffu, a, src);
        t.tokens = __shfl_sync(0xffffffffu, b - a, src);
        // a request's last tile first: it sees the most keys
        k = __shfl_sync(0xffffffffu, w.tiles + sum, src) - 1 - tile;
        break;
      }
      w.tiles += all;
      w.base += 32;
    }
  }
  t.len = p.lengths[t.n];
  t.before = t.len - t.tokens;
  t.first = k * per;
  t.rows = min(t.tokens * p.G - t.first, per);
  bool bad = t.len < 0 || t.len > kMaxLength || (int64_t)t.len > ((int64_t)p.max_blocks << p.shift);
  if (p.cu == nullptr) {
    if (t.len == 0) t.before = 0;  // no key: a row of zeros
  } else {
    bad |= t.tokens > t.len;
  }
  if (bad) {
    if (lane == 0) atomicOr(p.err, KDA_DEVERR_BAD_SEQLENS);
    t.rows = 0;
  }
  if (p.mask && t.tokens > 64 * p.mask_words) {
    if (lane == 0) atomicOr(p.err, KDA_DEVERR_BAD_COUNT);
    t.rows = 0;
  }
  return true;
}

// Drafted tokens that a row sees (those of its request that the mask names).
__device__ __forceinline__ int mask_count(const Params& p, const Tile& t, int token) {
  const uint64_t* m = p.mask + (int64_t)(t.t0 + token) * p.mask_words;
  int n = 0;
  for (int w = 0; w * 64 < t.tokens; ++w) {
    const int left = t.tokens - 64 * w;
    n += __popcll(m[w] & (left < 64 ? (1ull << left) - 1 : ~0ull));
  }
  return n;
}

// The keys that a row sees: [lo, hi] and those below `sinks` up to hi; a drafted token also what its mask names.
struct Row {
  int lo, hi;
  const uint64_t* mask;  // null: causal
};
__device__ __forceinline__ Row row_keys(const Params& p, const Tile& t, int token) {
  Row r;
  int pos = t.before + token;
  r.mask = nullptr;
  r.hi = p.cu == nullptr ? t.len - 1 : pos;
  if (p.mask) {
    r.mask = p.mask + (int64_t)(t.t0 + token) * p.mask_words;
    if (p.window > 0) pos = t.before + mask_count(p, t, token) - 1;
    r.hi = t.before - 1;
  }
  const int64_t lo = p.window > 0 ? (int64_t)pos + 1 - p.window : 0;
  r.lo = lo > 0 ? (int)lo : 0;
  return r;
}

// The keys that any row, and every row, of a span of tokens sees, and the boxes of B keys that hold them: the sinks'
// boxes, then those from the first key of a window on.
struct Span {
  int lo, hi;          // some row sees them, as it sees the sinks up to hi
  int all_lo, all_hi;  // every row sees these
  int sink_boxes, first_box, boxes;
};
// (one warp together; tokens [a, b) of the tile's request)
__device__ __forceinline__ Span span_of(const Params& p, const Tile& t, int a, int b, int box_shift) {
  Span s;
  int64_t lo, all_lo;
  if (p.mask) {
    int least = 1 << 30, most = 0;
    if (p.window > 0) {
      for (int i = a + (threadIdx.x & 31); i < b; i += 32) {
        const int m = mask_count(p, t, i);
        least = min(least, m);
        most = max(most, m);
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
    }
    s.hi = t.len - 1;
    s.all_hi = t.before - 1;
    lo = p.window > 0 ? (int64_t)t.before + least - p.window : 0;
    all_lo = p.window > 0 ? (int64_t)t.before + most - p.window : 0;
    if (lo > t.before) lo = t.before;  // the window says nothing of drafted tokens
  } else {
    s.hi = p.cu == nullptr ? t.len - 1 : t.before + b - 1;
    s.all_hi = p.cu == nullptr ? t.len - 1 : t.before + a;
    lo = p.window > 0 ? (int64_t)(p.cu == nullptr ? t.len - 1 : t.before + a) + 1 - p.window : 0;
    all_lo = p.window > 0 ? (int64_t)s.hi + 1 - p.window : 0;
  }
  s.lo = lo > 0 ? (int)lo : 0;
  s.all_lo = all_lo > 0 ? (int)all_lo : 0;
  s.first_box = s.lo >> box_shift;
  const int sinks = p.sinks < s.lo ? p.sinks : s.lo;  // below the window
  const int sink_boxes = (sinks + (1 << box_shift) - 1) >> box_shift;
  s.sink_boxes = sink_boxes < s.first_box ? sink_boxes : s.first_box;
  const int last = s.hi < 0 ? -1 : s.hi >> box_shift;
  s.boxes = s.sink_boxes + (last >= s.first_box ? last - s.first_box + 1 : 0);
  return s;
}
// the first key of the span's box i
__device__ __forceinline__ int box_key(const Span& s, int i, int box_shift) {
  return (i < s.sink_boxes ? i : i - s.sink_boxes + s.first_box) << box_shift;
}

// Bits a .. b of 16 (bit i: key `base` + i lies in [a, b]).
__device__ __forceinline__ uint32_t bits_between(int base, int a, int b) {
  const int x = a - base, y = b - base;  // keys are below 2^31, so these do not wrap
  if (y < 0 || x > 15 || y < x) return 0;
  const uint32_t up = y >= 15 ? 0xffffu : (2u << y) - 1u;
  return x > 0 ? up & ~((1u << x) - 1u) : up;
}
// Which of the 16 keys from `base` on a row sees.
__device__ __forceinline__ uint32_t seen16(const Params& p, const Tile& t, const Row& r, int base) {
  uint32_t m = bits_between(base, r.lo, r.hi);
  if (p.sinks > 0) m |= bits_between(base, 0, min(p.sinks - 1, r.hi));
  if (r.mask && base + 15 >= t.before) {
    const int off = base - t.before;  // drafted token of bit 0, above -16
    uint64_t w;
    if (off < 0) {
      w = r.mask[0] << -off;
    } else {
      const int i = off >> 6, sh = off & 63;
      w = i < p.mask_words ? r.mask[i] >> sh : 0;
      if (sh > 48 && i + 1 < p.mask_words) w |= r.mask[i + 1] << (64 - sh);
    }
    m |= (uint32_t)w & bits_between(base, t.before, t.len - 1);
  }
  return m;
}
// Trees: 64 drafted tokens from 64 w on, those of them that some row of tokens [a, b) of the request sees (one warp together).
__device__ __forceinline__ uint64_t named_word(const Params& p, const Tile& t, int a, int b, int w) {
  uint32_t lo = 0, hi = 0;
  for (int i = a + (int)(threadIdx.x & 31); i < b; i += 32) {
    const uint64_t m = p.mask[(int64_t)(t.t0 + i) * p.mask_words + w];
    lo |= (uint32_t)m;
    hi |= (uint32_t)(m >> 32);
  }
  return (uint64_t)__reduce_or_sync(0xffffffffu, hi) << 32 | __reduce_or_sync(0xffffffffu, lo);
}
// All of them, word w in lane w.
__device__ __forceinline__ uint64_t named_by(const Params& p, const Tile& t, int a, int b) {
  uint64_t mine = 0;
#pragma unroll 1
  for (int w = 0; w * 64 < t.tokens; ++w) {
    const uint64_t word = named_word(p, t, a, b, w);
    if ((int)(threadIdx.x & 31) == w) mine = word;
  }
  return mine;
}
// Which of the 16 keys from `base` on some row of the span sees.  Trees: `named` as above for the span's tokens, one warp
// together (each lane may have a base of its own).  TREES says that there may be masks.
template <bool TREES>
__device__ __forceinline__ uint32_t used16(const Params& p, const Tile& t, const Span& s, uint64_t named, int base) {
  const int hi = TREES && p.mask ? t.before - 1 : s.hi;
  uint32_t m = bits_between(base, s.lo, hi) | (p.sinks > 0 ? bits_between(base, 0, min(p.sinks - 1, hi)) : 0u);
  if (TREES && p.mask) {
    const int off = base - t.before, i = off > 0 ? off >> 6 : 0, sh = off & 63;
    const uint64_t w = __shfl_sync(0xffffffffu, named, i & 31), next = __shfl_sync(0xffffffffu, named, (i + 1) & 31);
    const uint64_t drafted = off <= -16 ? 0 : off < 0 ? w << -off : sh > 48 ? w >> sh | next << (64 - sh) : w >> sh;
    m |= (uint32_t)drafted & bits_between(base, t.before, t.len - 1);
  }
  return m;
}
// Whether every row of the span sees all keys of [base, base + n).
__device__ __forceinline__ bool all_seen(const Params& p, const Span& s, int base, int n) {
  return base + n - 1 <= s.all_hi && (base >= s.all_lo || base + n <= p.sinks);
}

// Tiles of `per` rows that the requests' new tokens can make at most (their lengths are on the device).
inline int64_t most_tiles(const AttentionArgs& a, int per) {
  const int64_t G = a.H / a.Hkv;
  return a.cu_seqlens ? a.T * G / per + a.N : a.N * ((G + per - 1) / per);
}
inline Params params_of(const AttentionArgs& a) {
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q); p.q_stride = a.q_stride; p.tables = a.block_tables; p.lengths = a.lengths;
  p.cu = a.cu_seqlens; p.mask = a.tree_mask; p.mask_words = a.mask_words; p.out = static_cast<__nv_bfloat16*>(a.out);
  p.N = a.N; p.T = a.T; p.H = a.H; p.Hkv = a.Hkv; p.G = a.H / a.Hkv; p.shift = a.shift; p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks; p.window = a.window; p.sinks = a.sinks; p.c = a.scale * 1.4426950408889634f; p.err = a.err;
  p.waits = a.waits; p.split = 1; p.by_G = divisor(p.G); p.by_Hkv = divisor(p.Hkv);
  return p;
}
// Keys that a tile sees at most, as far as the host knows.
inline int64_t most_keys(const AttentionArgs& a, int64_t tokens) {
  const int64_t seen = a.window > 0 ? (int64_t)a.window + a.sinks + tokens : a.max_length;
  return seen < a.max_length ? seen : a.max_length;
}

}  // namespace attn
}  // namespace kda
