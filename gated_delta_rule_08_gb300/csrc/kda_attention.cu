// Attention over a paged cache for few rows a key head: single tokens, and small trees of drafted tokens.
//
//   out_r = sum_j e^{s_rj - m_r} v_j / sum_j e^{s_rj - m_r},  s_rj = scale q_r . k_j,  m_r = max_j s_rj
//
// One pass over the keys with a running m and sum per row.  The weights are kept relative to a reference that follows
// the running maximum only when that passes it by 2^8, so that the sums are rarely rescaled: every weight is then
// at most 2^8, and nothing is lost, since sums and weights are floating point.
//
// A CTA has 16 rows of a request and key head (the rows of an m16n8k16 MMA; both products are MMAs, the weights go
// from one to the other in registers) and its four warps take boxes of 16 keys in turn.  Each warp copies its own
// boxes with TMA into a ring of its own, so that nothing but the end joins the warps; 107 KB a CTA and two
// CTAs an SM keep some 190 KB under way, which is what HBM's latency asks for.  Legacy MMAs are enough here:
// a box takes about 120 instructions and 32 MMAs of a scheduler, and its 8 KB some 350 clocks of an SM's share of HBM.
//
// Few requests leave SMs idle, so up to 16 CTAs, a cluster, share a tile's boxes; they join through distributed
// shared memory, each a part of the output, and no second launch or workspace is needed.
#include "kda_attention.cuh"

namespace kda {
namespace {

using namespace attn;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStages = 3;
constexpr int kRows = 16, kBox = 16, kBoxShift = 4;
constexpr int kMaxSplit = 16;
constexpr float kGone = -1.f;                // for a sum of weights: the CTA has given up
constexpr float kLowest = -3.402823466e38f;  // below every score: a weight relative to it is 0 for a masked key
constexpr float kSlack = 8.f;

template <int D>
struct Layout {
  static constexpr int kParts = D / 64;                    // 128-byte pieces of a token
  static constexpr uint32_t kPart = kBox * 128;            // a piece of all 16 tokens
  static constexpr uint32_t kStage = 2 * kParts * kPart;   // K, then V
  static constexpr uint32_t kRing = kStages * kStage;      // of a warp; at the end its sums [16][kPitch] fp32
  static constexpr int kPitch = D + 8;                     // (the rows of a quad's store in banks of their own)
  static constexpr uint32_t kIn = kWarps * kRing;          // [split][16 D / split]: this CTA's part of every CTA's sums
  static constexpr uint32_t kSums = kIn + kRows * D * 4;   // [kWarps][16] references and sums of weights of the warps,
  static constexpr uint32_t kAll = kSums + kWarps * kRows * 8;  // [kMaxSplit][16] of the CTAs
  static constexpr uint32_t kBar = kAll + kMaxSplit * kRows * 8;
  static constexpr uint32_t kSmem = kBar + kWarps * kStages * 8 + 8 + 1024;
  static_assert(kRows * kPitch * 4 <= kRing, "a warp's sums take its ring's place");
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool TREES>
__global__ void __launch_bounds__(kThreads)
attention_rows_kernel(const __grid_constant__ Maps maps, const Params p) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = aligned_smem(smem_raw);
  float2* sums = reinterpret_cast<float2*>(sm + L::kSums);  // reference, sum of weights
  float2* all = reinterpret_cast<float2*>(sm + L::kAll);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::kBar);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + kWarps * kStages);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.split > 1 ? (int)(blockIdx.x % p.split) : 0;

  griddep_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(&full[i], 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  griddep_wait();
  if (p.cu != nullptr && !offsets_within(p.cu, p.N, p.T)) {
    if (tid == 0) atomicOr(p.err, KDA_DEVERR_BAD_SEQLENS);
    return;
  }
  Walk walk;
  Tile t;
  if (!locate(p, kRows, Divisor{1, 4, kRows}, blockIdx.x / p.split, walk, t) || t.rows == 0) return;
  const int token0 = p.by_G.div(t.first), token1 = p.by_G.div(t.first + t.rows + p.G - 1);
  const Span span = span_of(p, t, token0, token1, kBoxShift);
  const int split = parts_of(p, span.boxes);
  if (rank >= split) return;
  if (split > 1) cluster_arrive();  // this CTA has begun: others may write to its memory
  __syncthreads();
  const int box0 = split > 1 ? (int)((int64_t)span.boxes * rank / split) : 0;
  const int box1 = split > 1 ? (int)((int64_t)span.boxes * (rank + 1) / split) : span.boxes;

  float O[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) O[i][j] = 0.f;
  float m0 = kLowest, m1 = kLowest, l0 = 0.f, l1 = 0.f;

  uint8_t* ring = sm + warp * L::kRing;
  uint64_t* bars = full + warp * kStages;
  const int count = box1 > box0 + warp ? (box1 - box0 - warp + kWarps - 1) / kWarps : 0;  // boxes of this warp
  const int32_t* table = p.tables + (int64_t)t.n * p.max_blocks;
  // trees: which drafted tokens the CTA's rows see, from the first box on that holds some
  uint64_t named = 0;
  bool drafted = false;
  // the blocks of boxes [32 i, 32 i + 32) of this warp, one a lane
  auto block_ids = [&](int i) {
    const int at = 32 * i + lane;
    int id = 0, key = 0;
    auto check = [&](bool used) {  // by some row
      if (used && (unsigned)id < (unsigned)p.num_blocks) return;
      if (used) atomicOr(p.err, KDA_DEVERR_BAD_SLOT);
      id = p.num_blocks;  // reads as zeros
    };
    if (at < count) {
      key = box_key(span, box0 + warp + at * kWarps, kBoxShift);
      id = table[key >> p.shift];
      if (!TREES) check(true);  // (here: below, with the trees', a single token over 8000 keys takes 15.6 us instead of 14.5)
    }
    if (TREES) {
      bool used = true;
      if (__any_sync(0xffffffffu, at < count && key + kBox > t.before)) {
        if (!drafted) named = named_by(p, t, token0, token1);
        drafted = true;
        used = used16<TREES>(p, t, span, named, key) != 0;
      }
      if (at < count) check(used);
    }
    return id;
  };
  int ids = block_ids(0), next_ids = block_ids(1), ids_of = 0;
  const bool copies = !(p.waits == kFirstCtaStalls && blockIdx.x == 0);
  int issued = 0;
  auto issue = [&]() {
    if (issued >> 5 != ids_of) {
      ids = next_ids;
      ++ids_of;
      next_ids = block_ids(ids_of + 1);
    }
    const int block = __shfl_sync(0xffffffffu, ids, issued & 31), s = issued % kStages;
    const int token = box_key(span, box0 + warp + issued * kWarps, kBoxShift) & ((1 << p.shift) - 1);
    if (lane == 0) {
      mbar_arrive_expect_tx(&bars[s], L::kStage);
      uint8_t* st = ring + s * L::kStage;
#pragma unroll
      for (int i = 0; i < L::kParts; ++i) {
        tma_load_box(st + i * L::kPart, &maps.k, 64 * i, token, t.head, block, &bars[s]);
        tma_load_box(st + (L::kParts + i) * L::kPart, &maps.v, 64 * i, token, t.head, block, &bars[s]);
      }
    }
    __syncwarp();
    ++issued;
  };
  if (copies) {
#pragma unroll 1
    while (issued < count && issued < kStages) issue();
  }

  // Q as the MMA's A operand: rows g and g + 8 of the lane's quad
  const int g = lane >> 2, c2 = (lane & 3) * 2;
  const int row0 = g, row1 = g + 8;
  const bool live0 = row0 < t.rows, live1 = row1 < t.rows;
  const int r0 = t.first + (live0 ? row0 : 0), r1 = t.first + (live1 ? row1 : 0);
  const int tok0 = p.by_G.div(r0), tok1 = p.by_G.div(r1);
  uint32_t Q[D / 16][4];
  {
    const int h0 = t.head * p.G + p.by_G.mod(r0), h1 = t.head * p.G + p.by_G.mod(r1);
    const uint32_t* q0 = reinterpret_cast<const uint32_t*>(p.q + (int64_t)(t.t0 + tok0) * p.q_stride + (int64_t)h0 * D + c2);
    const uint32_t* q1 = reinterpret_cast<const uint32_t*>(p.q + (int64_t)(t.t0 + tok1) * p.q_stride + (int64_t)h1 * D + c2);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      Q[i][0] = live0 ? q0[8 * i] : 0u;
      Q[i][1] = live1 ? q1[8 * i] : 0u;
      Q[i][2] = live0 ? q0[8 * i + 4] : 0u;
      Q[i][3] = live1 ? q1[8 * i + 4] : 0u;
    }
  }
  const Row keys0 = row_keys(p, t, tok0), keys1 = row_keys(p, t, tok1);

  const uint32_t key_row = (uint32_t)(((lane >> 4) << 3) + (lane & 7)), k_chunk = (uint32_t)(lane >> 3) & 1u;
  const uint32_t val_row = (uint32_t)(lane & 15), v_chunk = (uint32_t)lane >> 4;
  bool ok = true;
#pragma unroll 1
  for (int it = 0; it < count; ++it) {
    const int s = it % kStages;
    ok = p.waits == kWaitsGiveUp ? warp_wait<true>(&bars[s], 0, abort_flag)
                                 : warp_wait<false>(&bars[s], (uint32_t)((it / kStages) & 1), abort_flag);
    if (!ok) break;
    uint8_t* st = ring + s * L::kStage;
    const uint32_t sk = smem_u32(st), sv = sk + L::kParts * L::kPart;
    const int base = box_key(span, box0 + warp + it * kWarps, kBoxShift);
    const bool whole = all_seen(p, span, base, kBox);
    if (!whole) {
      // values that no row sees may be anything, and meet weights of 0 in the product: cleared
      const uint32_t used = used16<TREES>(p, t, span, named, base);
      if (used != 0xffffu) {
        for (int i = lane; i < kBox * 8 * L::kParts; i += 32) {
          const int r = i & 15, j = i >> 4;
          if (!(used >> r & 1))
            *reinterpret_cast<uint4*>(st + (L::kParts + (j >> 3)) * L::kPart + row_chunk(r, j & 7)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
    }
    float S[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t j = 2 * i + k_chunk;
      uint32_t b[4];
      ldsm4(sk + (j >> 3) * L::kPart + key_row * 128u + (((j & 7u) ^ (key_row & 7u)) << 4), b);
      mma16816(S[0], Q[i], b[0], b[1]);
      mma16816(S[1], Q[i], b[2], b[3]);
    }
    if (!whole) {
      const uint32_t see0 = seen16(p, t, keys0, base) >> c2, see1 = seen16(p, t, keys1, base) >> c2;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!(see0 >> (8 * n + j) & 1)) S[n][j] = -INFINITY;
          if (!(see1 >> (8 * n + j) & 1)) S[n][2 + j] = -INFINITY;
        }
    }
    const float top0 = fmaxf(fmaxf(S[0][0], S[0][1]), fmaxf(S[1][0], S[1][1])) * p.c;
    const float top1 = fmaxf(fmaxf(S[0][2], S[0][3]), fmaxf(S[1][2], S[1][3])) * p.c;
    if (__any_sync(0xffffffffu, top0 > m0 + kSlack || top1 > m1 + kSlack)) {
      float n0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, 1)), n1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, 1));
      n0 = fmaxf(m0, fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, 2)));
      n1 = fmaxf(m1, fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, 2)));
      const float f0 = ex2(m0 - n0), f1 = ex2(m1 - n1);
      m0 = n0;
      m1 = n1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        O[i][0] *= f0;
        O[i][1] *= f0;
        O[i][2] *= f1;
        O[i][3] *= f1;
      }
    }
    uint32_t P[4];
    float w[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) w[n][j] = ex2(fmaf(S[n][j], p.c, j < 2 ? -m0 : -m1));
    l0 += (w[0][0] + w[0][1]) + (w[1][0] + w[1][1]);
    l1 += (w[0][2] + w[0][3]) + (w[1][2] + w[1][3]);
    // to bf16, what the tensor cores take: half a step, 2^-8 at most, of each weight, at random in a sum of many
    P[0] = pack_bf2(w[0][0], w[0][1]);
    P[1] = pack_bf2(w[0][2], w[0][3]);
    P[2] = pack_bf2(w[1][0], w[1][1]);
    P[3] = pack_bf2(w[1][2], w[1][3]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t j = 2 * i + v_chunk;
      uint32_t b[4];
      ldsm4_t(sv + (j >> 3) * L::kPart + val_row * 128u + (((j & 7u) ^ (val_row & 7u)) << 4), b);
      mma16816(O[2 * i], P, b[0], b[1]);
      mma16816(O[2 * i + 1], P, b[2], b[3]);
    }
    __syncwarp();  // all lanes have read the stage
    if (copies && issued < count) issue();
  }
  if (!ok) {  // copies that are still under way land before the memory is given back
    for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
      if (lane == 0) mbar_wait(&bars[i % kStages], (uint32_t)((i / kStages) & 1));
    if (lane == 0) atomicOr(p.err, KDA_DEVERR_WAIT_TIMEOUT);
    __syncwarp();
  }

  // join: the warps' sums, then the CTAs'
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    *reinterpret_cast<float2*>(mine + row0 * L::kPitch + 8 * i + c2) = make_float2(O[i][0], O[i][1]);
    *reinterpret_cast<float2*>(mine + row1 * L::kPitch + 8 * i + c2) = make_float2(O[i][2], O[i][3]);
  }
  if ((lane & 3) == 0) {
    sums[warp * kRows + row0] = make_float2(m0, l0);
    sums[warp * kRows + row1] = make_float2(m1, l1);
  }
  __syncthreads();
  const bool gone = *abort_flag != 0;
  if (split > 1) cluster_wait();  // every CTA of the cluster has begun
  constexpr int kPieces = kRows * D / 4;  // of four values
  const int part = split == 1 ? kPieces : kPieces / split;
#pragma unroll
  for (int k = 0; k < kPieces / kThreads; ++k) {
    const int at = tid + k * kThreads, r = at / (D / 4), x = at % (D / 4) * 4;
    float m = kLowest, l = 0.f;
    float2 s[kWarps];
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      s[i] = sums[i * kRows + r];
      m = fmaxf(m, s[i].x);
    }
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float f = ex2(s[i].x - m);
      l = fmaf(f, s[i].y, l);
      a = f4_fma(f, *reinterpret_cast<const float4*>(sm + i * L::kRing + (r * L::kPitch + x) * 4), a);
    }
    if (gone) l = kGone;
    if (split == 1) {
      *reinterpret_cast<float4*>(sm + L::kIn + at * 16) = a;
      if (x == 0) all[r] = make_float2(m, l);
    } else {
      const int to = at / part;  // the CTA that writes these values; and everyone wants the sums
      st_peer4(peer(sm + L::kIn + (rank * part + at - to * part) * 16, to), a);
      if (x / 4 < split) st_peer2(peer(all + rank * kRows + r, x / 4), make_float2(m, l));
    }
  }
  if (split > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // this CTA's part of the rows (nobody writes to its memory any more, and it reads no one else's)
  for (int i = tid; i < part; i += kThreads) {
    const int at = rank * part + i, r = at / (D / 4), x = at % (D / 4) * 4;
    float m = kLowest, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    bool lost = false;
#pragma unroll 4
    for (int k = 0; k < split; ++k) m = fmaxf(m, all[k * kRows + r].x);
#pragma unroll 4
    for (int k = 0; k < split; ++k) {
      const float2 s = all[k * kRows + r];
      const float f = ex2(s.x - m);
      lost |= s.y == kGone;
      l = fmaf(f, s.y, l);
      a = f4_fma(f, *reinterpret_cast<const float4*>(sm + L::kIn + (k * part + i) * 16), a);
    }
    if (r >= t.rows || lost) continue;
    const float inv = l != 0.f ? 1.f / l : 0.f;  // a row that sees nothing is zero (a NaN stays one)
    const int tok = p.by_G.div(t.first + r), h = t.head * p.G + p.by_G.mod(t.first + r);
    *reinterpret_cast<uint2*>(p.out + ((int64_t)(t.t0 + tok) * p.H + h) * D + x) =
        make_uint2(pack_bf2(a.x * inv, a.y * inv), pack_bf2(a.z * inv, a.w * inv));
  }
}

// CTAs that may share a tile's keys, and the boxes for each at least: few tiles leave SMs idle, and are cut down to 256
// keys; many are cut to about kMostKeys, so that no long request is left over at the end, as far as CTAs that find nothing
// to do (of the others) remain cheap (256 requests with a window of 1024, 1024 / 2048 keys: 149 / 115 us; 16 requests of 20
// to 16000 tokens, 512 / 1024 / 2048 keys: 64 / 65 / 46 us).
constexpr int kMostKeys = 2048, kMostCtas = 4096;
void split_of(int64_t tiles, int64_t keys, int sms, int* split, int* least) {
  *split = 1;
  while (*split < kMaxSplit && tiles * *split * 2 <= 2 * sms && keys > 256 * *split) *split *= 2;
  *least = 256 / kBox;
  if (tiles * 4 <= 2 * sms) return;
  *least = kMostKeys / kBox;
  while (*split < kMaxSplit && tiles * *split * 2 <= kMostCtas && keys > kMostKeys * *split) *split *= 2;
}

template <int D, bool TREES>
cudaError_t launch(const AttentionArgs& a, Params p, cudaStream_t st) {
  Maps maps;
  if (!tensor_map_cache(&maps.k, a.k_cache, a.num_blocks, 1u << a.shift, a.Hkv, D, a.block_stride, a.token_stride, a.head_stride, kBox) ||
      !tensor_map_cache(&maps.v, a.v_cache, a.num_blocks, 1u << a.shift, a.Hkv, D, a.block_stride, a.token_stride, a.head_stride, kBox))
    return cudaErrorInvalidValue;
  static DeviceOnce once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  cudaError_t e = once.run(dev, [] {
    cudaError_t f = cudaFuncSetAttribute(attention_rows_kernel<D, TREES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<D>::kSmem);
    if (f == cudaSuccess) f = cudaFuncSetAttribute(attention_rows_kernel<D, TREES>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return f;
  });
  if (e != cudaSuccess) return e;
  const int64_t tiles = most_tiles(a, kRows) * a.Hkv;
  p.by_each = divisor((p.G + kRows - 1) / kRows);
  split_of(tiles, most_keys(a, kRows), sms, &p.split, &p.least);
  TraceScope ts("kda_attention_rows", st);
  return launch_overlapped(attention_rows_kernel<D, TREES>, (unsigned)(tiles * p.split), kThreads, Layout<D>::kSmem, (unsigned)p.split, st, maps, p);
}

}  // namespace

cudaError_t attention_rows_launch(const AttentionArgs& a, cudaStream_t st) {
  if (a.tree_mask) return a.d == 64 ? launch<64, true>(a, params_of(a), st) : launch<128, true>(a, params_of(a), st);
  return a.d == 64 ? launch<64, false>(a, params_of(a), st) : launch<128, false>(a, params_of(a), st);
}

}  // namespace kda
