// Matrix product of e4m3 rows with a scale for each block of 128 values, on the tcgen05 tensor cores.
//
//   out[m][n] = sum_kb a_scale[m][kb] b_scale[n / 128][kb] P_kb[m][n],  P_kb = sum_{k in block kb} a[m][k] b[n][k]
//
// The scales are free fp32 numbers, so each block's product P_kb (four MMAs of K = 32 into a fresh
// TMEM accumulator) is read back and added in fp32 registers with its scale: the tensor cores sum 128
// terms, registers the blocks.  TMEM holds several accumulators, so that the MMAs of a block run while
// earlier ones are read.  A block of 128 e4m3 values is one 128-byte row: exactly one swizzle atom, one
// stage of the ring that the TMA copies fill.  Rows and columns past the edges read as zeros.
//
// Two orientations:
//  matmul_fp8_tall: 128 activation rows x 256 weight rows per tile, one CTA per SM walking over tiles;
//    a thread owns part of one activation row, whose scale for a block of K is one number.
//  matmul_fp8_flat: 128 weight rows x BN activation rows per tile, for few rows: the weight is then the
//    operand with 128 rows and nothing is padded but the activations (to BN).  Bound by the weight's
//    bytes, so the K blocks of a tile are split over the CTAs of a cluster, which add their partial
//    sums through distributed shared memory in a fixed order.
//
// Measured: 8192 x 12288 x 4096 342 to 370 us from run to run, 2.2 to 2.4 PFLOP/s (900-960 clocks a block of K, of
// which the MMAs need 524: 48 KB a block into each SM bound it); 64 x 12288 x 4096 15.4 us, 3.3 TB/s of weight;
// 16 x 12288 x 4096 12.6 us, 4.0 TB/s.
#include "kda_device.cuh"
#include "kda_internal.h"
#include "kda_tc_common.cuh"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace tcx;

constexpr int kK = 128;  // values of a scale block = bytes of a stage's row

// kind::f8f6f4: D fp32 (bit 4), A and B e4m3 (0), both K-major
constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// One block of 128: P = A B^T, K = 32 bytes per MMA.
__device__ __forceinline__ void mma_block(bool leader, uint32_t d, const uint8_t* a, const uint8_t* b, uint32_t idesc) {
  const uint64_t da = smem_desc_sw128(smem_u32(a), 16, 1024), db = smem_desc_sw128(smem_u32(b), 16, 1024);
#pragma unroll
  for (int i = 0; i < 4; ++i) mma_f8_ss_by(leader, d, desc_add(da, 32 * i), desc_add(db, 32 * i), idesc, i > 0);
}

// acc (two fp32 lanes) += s * d
__device__ __forceinline__ void acc_fma2(uint64_t& acc, float s0, float s1, float d0, float d1) {
  asm("{\n .reg .b64 rs, rd;\n mov.b64 rs, {%1, %2};\n mov.b64 rd, {%3, %4};\n fma.rn.f32x2 %0, rs, rd, %0;\n}"
      : "+l"(acc)
      : "f"(s0), "f"(s1), "f"(d0), "f"(d1));
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// four fp32 at the same shared-memory offset of CTA `rank` of the cluster
__device__ __forceinline__ float4 load_peer(const float* p, uint32_t rank) {
  uint32_t a;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// the word at the same shared-memory offset of CTA `rank` of the cluster
__device__ __forceinline__ int load_peer(const volatile int* p, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(const_cast<const int*>(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

struct Maps {
  CUtensorMap a, b;
};

// ------------------------------------------------------------------------------ many rows
constexpr int kTallM = 128, kTallN = 256, kTallStages = 4;
// The tile's two halves of 128 columns are worked on apart, each with two accumulators: while one set of four
// warps adds a block's half, the other half's MMAs and the next block's run, and the two sets stay out of step, so
// that one's TMEM loads lie beside the other's arithmetic.
// Warps 0-3 and 4-7 read accumulators, scale, add and store: a thread owns 128 columns of a row.  Warp 8 copies,
// warp 9 fetches the scales.  Warps 12-15 issue the MMAs, one warp to an accumulator: a commit takes 70 clocks of the
// thread that issues it and a wait behind it 150, so one thread alone would leave the tensor pipe idle in between.
// Warps 10 and 11 only complete their group of four; the groups hand their registers to the first eight warps.
constexpr int kPromoteWarps = 8, kTallCopyWarp = 8, kTallScaleWarp = 9, kTallMmaWarp = 12, kTallThreads = 512;
constexpr int kPromoteRegs = 208, kOtherRegs = 48;
static_assert(kPromoteWarps * 32 * kPromoteRegs + 8 * 32 * kOtherRegs <= kTallThreads * 128, "registers of the launch");
constexpr uint32_t kTallA = kTallM * kK, kTallStage = (kTallM + kTallN) * kK;
// Each promoting warp's 16 rows x 128 bytes of output, so that rows are stored as whole lines: a thread's own row,
// 16 bytes at a time, took 8400 clocks a tile.
constexpr uint32_t kTallOut = kTallStages * kTallStage, kTallOutWarp = 16 * 128;
// The activations' scales of a tile's rows, for groups of eight blocks: [2][8][132], and the weights' [2][8][2].
constexpr int kGroup = 8, kScaleLd = kTallM + 4;
constexpr uint32_t kTallSa = kTallOut + kPromoteWarps * kTallOutWarp, kTallSb = kTallSa + 2 * kGroup * kScaleLd * 4;
constexpr uint32_t kTallBar = kTallSb + 2 * kGroup * 2 * 4;
constexpr uint32_t kTallSmem = kTallBar + 256 + 1024;
static_assert(kTallSmem <= 232448, "shared memory of a CTA");

// PAIR: two CTAs of a cluster share a tile, each with half of the K blocks (so few tiles that every pair is resident).
template <typename Tout, bool PAIR, int WAITS>
__global__ void __launch_bounds__(kTallThreads, 1)
matmul_fp8_tall(const __grid_constant__ Maps maps, const float* __restrict__ a_scale, const float* __restrict__ b_scale,
                Tout* __restrict__ out, int M, int N, int nkb, int tiles_m, int tiles, unsigned int* __restrict__ err) {
  constexpr bool GIVEUP = WAITS == kWaitsGiveUp;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = aligned_smem(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kTallBar);  // [stages] tiles landed
  uint64_t* mma_done = full + kTallStages;                      // [half][stages] accumulator complete, stage read
  uint64_t* acc_empty = mma_done + 2 * kTallStages;             // [half][2] accumulator read
  uint64_t* sc_full = acc_empty + 4;                            // [2] group of scales there
  uint64_t* sc_empty = sc_full + 2;                             // [2] group of scales read
  uint64_t* bar_fin = sc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* s_sa = reinterpret_cast<float*>(sm + kTallSa);
  float* s_sb = reinterpret_cast<float*>(sm + kTallSb);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int tile0 = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x, step = PAIR ? tiles : (int)gridDim.x;
  const int kb0 = PAIR && rank == 1 ? nkb / 2 : 0, kb1 = PAIR && rank == 0 ? nkb / 2 : nkb;  // this CTA's blocks

  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < kTallStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&mma_done[i], 1);
      mbar_init(&mma_done[kTallStages + i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&acc_empty[i], kPromoteWarps / 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sc_full[i], 1);
      mbar_init(&sc_empty[i], kPromoteWarps);
    }
    mbar_init(bar_fin, 4);
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int64_t issued = 0;  // stages whose copies have been started

  if (warp >= kPromoteWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kTallCopyWarp && lane == 0) {
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += step) {
        const int m0 = tile % tiles_m * kTallM, n0 = tile / tiles_m * kTallN;
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++issued) {
          const int s = (int)(issued % kTallStages);
          if (issued >= kTallStages) {
            const uint32_t ph = (uint32_t)((issued / kTallStages - 1) & 1);
            ok = spin_or_abort<GIVEUP>(&mma_done[s], ph, abort_flag) &&
                 spin_or_abort<GIVEUP>(&mma_done[kTallStages + s], ph, abort_flag);
          }
          if (!ok) break;
          uint8_t* st = sm + s * kTallStage;
          mbar_arrive_expect_tx(&full[s], kTallStage);
          tma_load_2d(st, &maps.a, kb * kK, m0, &full[s]);
          tma_load_2d(st + kTallA, &maps.b, kb * kK, n0, &full[s]);
        }
      }
    } else if (warp >= kTallMmaWarp) {
      const bool leader = lane == 0;
      const int half = (warp - kTallMmaWarp) >> 1, buf = warp & 1;
      int64_t it = 0;
      bool ok = !(WAITS == kFirstCtaStalls && blockIdx.x == 0);
      for (int tile = tile0; tile < tiles && ok; tile += step) {
        for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
          if ((it & 1) != buf) continue;
          const int s = (int)(it % kTallStages);
          ok = warp_wait<GIVEUP>(&full[s], (uint32_t)((it / kTallStages) & 1), abort_flag);
          if (ok && it >= 2)
            ok = warp_wait<GIVEUP>(&acc_empty[2 * half + buf], (uint32_t)((it / 2 - 1) & 1), abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint8_t* st = sm + s * kTallStage;
          mma_block(leader, tmem + 256 * buf + 128 * half, st, st + kTallA + half * 128 * kK, idesc_e4m3(kTallM, kTallN / 2));
          mma_commit_by(leader, &mma_done[half * kTallStages + s]);
        }
      }
    } else if (warp == kTallScaleWarp) {
      int64_t grp = 0;
      bool ok = true;
      for (int tile = tile0; tile < tiles && ok; tile += step) {
        // rows and blocks past the edges take another's scale; their products are zero
        const int m0 = tile % tiles_m * kTallM, nb0 = tile / tiles_m * (kTallN / 128), nb = (N + 127) / 128;
        for (int k0 = kb0; k0 < kb1; k0 += kGroup, ++grp) {
          const int slot = (int)(grp & 1), kb = k0 + (lane & 7);
          if (grp >= 2) ok = warp_wait<GIVEUP>(&sc_empty[slot], (uint32_t)((grp / 2 - 1) & 1), abort_flag);
          if (!ok) break;
          float* d = s_sa + slot * kGroup * kScaleLd + (lane & 7) * kScaleLd;
          if (kb < kb1) {
#pragma unroll 8
            for (int r = lane >> 3; r < kTallM; r += 4) {
              const int m = m0 + r;
              d[r] = __ldg(a_scale + (int64_t)(m < M ? m : M - 1) * nkb + kb);
            }
            if (lane < 16) {
              const int j = nb0 + (lane >> 3);
              s_sb[(slot * kGroup + (lane & 7)) * 2 + (lane >> 3)] = __ldg(b_scale + (int64_t)(j < nb ? j : nb - 1) * nkb + kb);
            }
          }
          warp_arrive(&sc_full[slot]);
        }
      }
    }
    if constexpr (PAIR) {  // the joins of the promoting warps
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPromoteRegs));
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem_lane(tmem, warp) + 128 * half;
    uint64_t* my_done = mma_done + kTallStages * half;
    uint64_t* my_empty = acc_empty + 2 * half;
    int64_t it = 0, grp = 0;
    bool ok = true;
    for (int tile = tile0; tile < tiles && ok; tile += step) {
      const int m = tile % tiles_m * kTallM + row, n0 = tile / tiles_m * kTallN + 128 * half;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      // In steps of 32 columns: the next step's load is under way while this one is added, across blocks too
      // (a barrier that is already complete still takes some 250 clocks to be seen).
      float v[32], w[32];
      auto add = [&](const float (&x)[32], int c, float s) {
#pragma unroll
        for (int i = 0; i < 16; ++i) acc_fma2(acc[16 * c + i], s, s, x[2 * i], x[2 * i + 1]);
      };
      auto wait_block = [&](int64_t i) {  // the loads are collective: a warp leaves together
        return warp_wait<GIVEUP>(&my_done[i % kTallStages], (uint32_t)((i / kTallStages) & 1), abort_flag);
      };
      ok = wait_block(it);
      if (ok) {
        tc_fence_after();
        tmem_ld32(tl + 256 * (uint32_t)(it & 1), v);
      }
#pragma unroll 1
      for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
        const uint32_t ta = tl + 256 * (uint32_t)(it & 1);
        const bool more = kb + 1 < kb1;
        const int slot = (int)(grp & 1), kg = (kb - kb0) % kGroup;
        if (kg == 0) {
          ok = warp_wait<GIVEUP>(&sc_full[slot], (uint32_t)((grp / 2) & 1), abort_flag);
          if (!ok) break;
        }
        const float s = s_sa[(slot * kGroup + kg) * kScaleLd + row] * s_sb[(slot * kGroup + kg) * 2 + half];
        tmem_landed(v);
        tmem_ld32(ta + 32, w);
        add(v, 0, s);
        tmem_landed(w);
        tmem_ld32(ta + 64, v);
        add(w, 1, s);
        tmem_landed(v);
        tmem_ld32(ta + 96, w);
        const bool seen = !GIVEUP && more && mbar_test_wait(&my_done[(it + 1) % kTallStages], (uint32_t)(((it + 1) / kTallStages) & 1));
        add(v, 2, s);
        tmem_landed(w);
        tc_fence_before();
        warp_arrive(&my_empty[it & 1]);
        if (kg == kGroup - 1 || !more) {
          warp_arrive(&sc_empty[slot]);
          ++grp;
        }
        if (more) {
          if (!__all_sync(0xffffffffu, seen)) ok = wait_block(it + 1);
          if (!ok) break;
          tc_fence_after();
          tmem_ld32(tl + 256 * (uint32_t)((it + 1) & 1), v);
        }
        add(w, 3, s);
      }
      if constexpr (PAIR) {
        // CTA r finishes columns 64 r to 64 r + 63 of each half; the others' sums go to the peer by way of the
        // stages.  All MMAs have read those once both halves' last accumulators are complete.
        float* part = reinterpret_cast<float*>(sm) + 4 * tid;
        ok = group_and(1, kPromoteWarps * 32, ok && !*abort_flag);
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (ok && r != rank)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = split2(acc[32 * r + 2 * i]), y = split2(acc[32 * r + 2 * i + 1]);
              *reinterpret_cast<float4*>(part + i * kPromoteWarps * 128) = make_float4(x.x, x.y, y.x, y.y);
            }
        cluster_sync();
        // a peer that has given up has no sums to add: neither CTA stores
        const bool peer_ok = load_peer(abort_flag, (uint32_t)(rank ^ 1)) == 0;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (ok && r == rank)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 x = load_peer(part + i * kPromoteWarps * 128, (uint32_t)(rank ^ 1));
              acc_fma2(acc[32 * r + 2 * i], 1.f, 1.f, x.x, x.y);
              acc_fma2(acc[32 * r + 2 * i + 1], 1.f, 1.f, x.z, x.w);
            }
        cluster_sync();  // the peer's sums have been read
        ok = ok && peer_ok;
      }
      if (!ok) break;
      // by 128 bytes of columns: to shared memory with the row's 16-byte pieces permuted, then out by rows
      constexpr int kCols = 128 / sizeof(Tout), kPiece = 16 / sizeof(Tout);
      uint8_t* stage = sm + kTallOut + warp * kTallOutWarp;
      const int m_warp = m - lane;
#pragma unroll
      for (int c = 0; c < 128 / kCols; ++c) {
        if (PAIR && c * kCols / 64 != rank) continue;
        const int nc = n0 + c * kCols;
        for (int h = 0; h < 2; ++h) {  // rows 0-15, then 16-31 of the warp
          if ((lane >> 4) == h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint4 w4;
              if constexpr (sizeof(Tout) == 4) {
                const float2 x = split2(acc[(c * kCols + 4 * i) / 2]), y = split2(acc[(c * kCols + 4 * i) / 2 + 1]);
                w4 = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
              } else {
                uint32_t q[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 x = split2(acc[(c * kCols + 8 * i) / 2 + e]);
                  const __nv_bfloat162 hh = __floats2bfloat162_rn(x.x, x.y);
                  q[e] = *reinterpret_cast<const uint32_t*>(&hh);
                }
                w4 = make_uint4(q[0], q[1], q[2], q[3]);
              }
              *reinterpret_cast<uint4*>(stage + row_chunk(lane & 15, i)) = w4;
            }
          }
          __syncwarp();
          const int m_half = m_warp + 16 * h;
          if (N % kPiece == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 4 * i + (lane >> 3), n = nc + (lane & 7) * kPiece;
              if (m_half + r < M && n < N)
                *reinterpret_cast<uint4*>(out + (int64_t)(m_half + r) * N + n) =
                    *reinterpret_cast<const uint4*>(stage + row_chunk(r, lane & 7));
            }
          } else {  // rows off the 16-byte boundaries: value by value
            for (int r = 0; r < 16 && m_half + r < M; ++r)
#pragma unroll
              for (int e = lane; e < kCols; e += 32)
                if (nc + e < N)
                  out[(int64_t)(m_half + r) * N + nc + e] =
                      *reinterpret_cast<const Tout*>(stage + row_chunk(r, e / kPiece) + e % kPiece * sizeof(Tout));
          }
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  drain_after_abort<kTallStages>(abort_flag, tid == kTallCopyWarp * 32, warp >= kTallMmaWarp && lane == 0, full, issued, bar_fin, err);
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------------------ few rows
constexpr int kFlatRows = 128;  // weight rows of a tile
// Warps 0-3 read accumulators, scale, add up: a thread owns a weight row; 4 copies, 5 multiplies, 6 makes the factors.
constexpr int kFlatCopyWarp = 4, kFlatMmaWarp = 5, kFlatScaleWarp = 6, kFlatThreads = 224;

template <int BN>
struct Flat {
  static constexpr int kBufs = 4;  // accumulators; two CTAs share an SM's 512 columns
  static constexpr uint32_t kCols = kBufs * BN;
  static constexpr uint32_t kW = kFlatRows * kK, kStage = kW + BN * kK;
  static constexpr int kStages = 98304 / kStage;  // 96 KB: two CTAs per SM
  static constexpr int kLd = BN + 4;              // factors of a block: one for each activation row
  static constexpr uint32_t kPart = BN * kFlatRows * 4;  // partial sums, over the stages once they are read
  static constexpr uint32_t kScale = kStages * kStage;
  static constexpr uint32_t kBar = kScale + 2 * kGroup * kLd * 4;
  static constexpr uint32_t kSmem = kBar + 256 + 1024;
  static_assert(kPart <= kScale && kStages >= kBufs, "an accumulator is read before its stage's next MMAs");
};

constexpr int kMaxSplit = 8;

template <int BN, typename Tout, int WAITS>
__global__ void __launch_bounds__(kFlatThreads)
matmul_fp8_flat(const __grid_constant__ Maps maps, const float* __restrict__ a_scale, const float* __restrict__ b_scale,
                Tout* __restrict__ out, int M, int N, int nkb, int split, unsigned int* __restrict__ err) {
  using F = Flat<BN>;
  constexpr bool GIVEUP = WAITS == kWaitsGiveUp;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = aligned_smem(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + F::kBar);  // [stages] tiles landed
  uint64_t* mma_done = full + F::kStages;                      // [stages] accumulator complete, stage read
  uint64_t* acc_empty = mma_done + F::kStages;                 // [bufs] accumulator read
  uint64_t* sc_full = acc_empty + F::kBufs;                    // [2] group of factors there
  uint64_t* sc_empty = sc_full + 2;                            // [2] group of factors read
  uint64_t* bar_fin = sc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* part = reinterpret_cast<float*>(sm);
  float* fac = reinterpret_cast<float*>(sm + F::kScale);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = split > 1 ? (int)cluster_rank() : 0;
  const int n0 = blockIdx.x / split * kFlatRows, m0 = blockIdx.y * BN;
  // this CTA's blocks: [kb0, kb0 + cnt), as even as they get
  const int kb0 = (int)((int64_t)nkb * rank / split), cnt = (int)((int64_t)nkb * (rank + 1) / split) - kb0;

  if (warp == 0) {
    tmem_alloc(tmem_slot, F::kCols);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < F::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&mma_done[i], 1);
    }
    for (int i = 0; i < F::kBufs; ++i) mbar_init(&acc_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sc_full[i], 1);
      mbar_init(&sc_empty[i], 4);
    }
    mbar_init(bar_fin, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int issued = 0;  // stages whose copies have been started

  if (warp == kFlatCopyWarp) {
    if (lane == 0) {
      bool ok = true;
      for (; issued < cnt; ++issued) {
        const int it = issued, s = it % F::kStages;
        if (it >= F::kStages) ok = spin_or_abort<GIVEUP>(&mma_done[s], (uint32_t)((it / F::kStages - 1) & 1), abort_flag);
        if (!ok) break;
        uint8_t* st = sm + s * F::kStage;
        mbar_arrive_expect_tx(&full[s], F::kStage);
        tma_load_2d(st, &maps.b, (kb0 + it) * kK, n0, &full[s]);
        tma_load_2d(st + F::kW, &maps.a, (kb0 + it) * kK, m0, &full[s]);
      }
    }
  } else if (warp == kFlatMmaWarp) {
    {
      const bool leader = lane == 0;
      bool ok = !(WAITS == kFirstCtaStalls && blockIdx.x == 0 && blockIdx.y == 0);
      for (int it = 0; it < cnt && ok; ++it) {
        const int s = it % F::kStages, buf = it % F::kBufs;
        ok = warp_spin<GIVEUP>(&full[s], (uint32_t)((it / F::kStages) & 1), abort_flag);
        if (ok && it >= F::kBufs)
          ok = warp_spin<GIVEUP>(&acc_empty[buf], (uint32_t)((it / F::kBufs - 1) & 1), abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint8_t* st = sm + s * F::kStage;
        mma_block(leader, tmem + BN * buf, st, st + F::kW, idesc_e4m3(kFlatRows, BN));
        mma_commit_by(leader, &mma_done[s]);
      }
    }
  } else if (warp == kFlatScaleWarp) {
    bool ok = true;
    const float* pb = b_scale + (int64_t)(n0 / 128) * nkb + kb0;
    for (int k0 = 0, grp = 0; k0 < cnt; k0 += kGroup, ++grp) {
      const int slot = grp & 1, kb = k0 + (lane & 7);
      if (grp >= 2) ok = warp_wait<GIVEUP>(&sc_empty[slot], (uint32_t)((grp / 2 - 1) & 1), abort_flag);
      if (!ok) break;
      if (kb < cnt) {
        float* d = fac + (slot * kGroup + (lane & 7)) * F::kLd;
        const float sb = __ldg(pb + kb);
        float sa[BN / 4];
#pragma unroll
        for (int i = 0; i < BN / 4; ++i) {
          const int m = m0 + (lane >> 3) + 4 * i;
          sa[i] = m < M ? __ldg(a_scale + (int64_t)m * nkb + kb0 + kb) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < BN / 4; ++i) d[(lane >> 3) + 4 * i] = sa[i] * sb;
      }
      warp_arrive(&sc_full[slot]);
    }
  } else {
    const uint32_t tl = tmem_lane(tmem, warp);
    uint64_t acc[BN / 2];
#pragma unroll
    for (int i = 0; i < BN / 2; ++i) acc[i] = 0;
    bool ok = true;
#pragma unroll 1
    for (int it = 0; it < cnt; ++it) {
      const int s = it % F::kStages, buf = it % F::kBufs, slot = (it / kGroup) & 1, kg = it % kGroup;
      if (kg == 0) ok = warp_wait<GIVEUP>(&sc_full[slot], (uint32_t)((it / kGroup / 2) & 1), abort_flag);
      ok = ok && warp_wait<GIVEUP>(&mma_done[s], (uint32_t)((it / F::kStages) & 1), abort_flag);
      if (!ok) break;
      tc_fence_after();
      const float* f = fac + (slot * kGroup + kg) * F::kLd;
#pragma unroll
      for (int c = 0; c < BN / 16; ++c) {
        float v[16];
        tmem_ld16(tl + BN * buf + 16 * c, v);
        tmem_landed(v);
        if (c == BN / 16 - 1) {
          tc_fence_before();
          warp_arrive(&acc_empty[buf]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(f + 16 * c + 4 * i);
          acc_fma2(acc[8 * c + 2 * i], w.x, w.y, v[4 * i], v[4 * i + 1]);
          acc_fma2(acc[8 * c + 2 * i + 1], w.z, w.w, v[4 * i + 2], v[4 * i + 3]);
        }
      }
      if (kg == kGroup - 1) warp_arrive(&sc_empty[slot]);
    }
    // Every copy has landed and every MMA has read its stage once the last accumulator is complete (the
    // MMAs complete in order), so the partial sums may lie over the stages.  After a wait that ran out the
    // copies may still be on their way: nothing is written there.  All four warps decide together.
    if (group_and(1, 128, ok && !*abort_flag)) {
      const int n = (warp & 3) * 32 + lane;
#pragma unroll
      for (int i = 0; i < BN / 2; ++i) {
        const float2 x = split2(acc[i]);
        part[(2 * i) * kFlatRows + n] = x.x;
        part[(2 * i + 1) * kFlatRows + n] = x.y;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  drain_after_abort<F::kStages>(abort_flag, tid == kFlatCopyWarp * 32, tid == kFlatMmaWarp * 32, full, issued, bar_fin, err);
  if (split > 1) cluster_sync();
  tc_fence_after();
  // The activation rows are dealt to the warps of the cluster's CTAs; each sums the partial sums in rank order, four
  // columns a thread.  A CTA that has given up has no partial sums: then nobody stores (lane r asks CTA r, beside the
  // sums' loads).
  const int rows = M - m0 < BN ? M - m0 : BN, n = n0 + 4 * lane;
  for (int j = rank + split * warp; j < rows; j += split * (kFlatThreads / 32)) {
    const float* p = part + j * kFlatRows + 4 * lane;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    int gave_up = *abort_flag;
    if (split == 1) {
      x = *reinterpret_cast<const float4*>(p);
    } else {
      float4 y[kMaxSplit];
      if (lane < split) gave_up = load_peer(abort_flag, lane);
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < split) y[r] = load_peer(p, r);
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        if (r < split) x = make_float4(x.x + y[r].x, x.y + y[r].y, x.z + y[r].z, x.w + y[r].w);
    }
    if (__any_sync(0xffffffffu, gave_up)) break;
    Tout* dst = out + (int64_t)(m0 + j) * N + n;
    if (N % 4 == 0) {
      if (n < N) {
        if constexpr (sizeof(Tout) == 4) {
          *reinterpret_cast<float4*>(dst) = x;
        } else {
          const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(x.z, x.w)};
          *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(h);
        }
      }
    } else {
      const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < N) dst[e] = from_f32<Tout>(v[e]);
    }
  }
  if (split > 1) cluster_sync();  // the peers' partial sums stay until they are read
  if (warp == 0) tmem_dealloc(tmem, F::kCols);
}

// ------------------------------------------------------------------------------ host side
struct DeviceState {
  DeviceOnce once;
  int sms[kMaxDevices] = {};
};
DeviceState g_state;

// The kernels' variants, indexed by test_wait_timeout().
template <int BN, typename Tout>
auto* flat_kernel(int waits) {
  return waits == kWaits ? matmul_fp8_flat<BN, Tout, kWaits>
                         : (waits == kWaitsGiveUp ? matmul_fp8_flat<BN, Tout, kWaitsGiveUp> : matmul_fp8_flat<BN, Tout, kFirstCtaStalls>);
}
template <typename Tout, bool PAIR>
auto* tall_kernel(int waits) {
  return waits == kWaits ? matmul_fp8_tall<Tout, PAIR, kWaits>
                         : (waits == kWaitsGiveUp ? matmul_fp8_tall<Tout, PAIR, kWaitsGiveUp> : matmul_fp8_tall<Tout, PAIR, kFirstCtaStalls>);
}
template <typename Kernel>
cudaError_t allow_smem(Kernel* k, uint32_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}
template <int BN>
cudaError_t allow_flat() {
  cudaError_t e = cudaSuccess;
  for (int w = kWaits; w <= kFirstCtaStalls; ++w) {
    if (e == cudaSuccess) e = allow_smem(flat_kernel<BN, __nv_bfloat16>(w), Flat<BN>::kSmem);
    if (e == cudaSuccess) e = allow_smem(flat_kernel<BN, float>(w), Flat<BN>::kSmem);
  }
  return e;
}
template <typename Tout>
cudaError_t allow_tall() {
  cudaError_t e = cudaSuccess;
  for (int w = kWaits; w <= kFirstCtaStalls; ++w) {
    if (e == cudaSuccess) e = allow_smem(tall_kernel<Tout, false>(w), kTallSmem);
    if (e == cudaSuccess) e = allow_smem(tall_kernel<Tout, true>(w), kTallSmem);
  }
  return e;
}
cudaError_t prepare_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const cudaError_t e = g_state.once.run(dev, [dev] {
    cudaError_t e = allow_tall<__nv_bfloat16>();
    if (e == cudaSuccess) e = allow_tall<float>();
    if (e == cudaSuccess) e = allow_flat<16>();
    if (e == cudaSuccess) e = allow_flat<32>();
    if (e == cudaSuccess) e = allow_flat<64>();
    if (e != cudaSuccess) return e;
    return cudaDeviceGetAttribute(&g_state.sms[dev], cudaDevAttrMultiProcessorCount, dev);
  });
  if (e == cudaSuccess) *sms = g_state.sms[dev];
  return e;
}

template <int BN, typename Tout>
cudaError_t launch_flat(const MatmulArgs& a, int sms, cudaStream_t st) {
  using F = Flat<BN>;
  const int nkb = (a.K + kK - 1) / kK, tiles = (a.N + kFlatRows - 1) / kFlatRows;
  const int64_t rows = (a.M + BN - 1) / BN;
  Maps maps;
  if (!tensor_map_2d(&maps.a, a.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.M, a.K, a.K, BN, kK) ||
      !tensor_map_2d(&maps.b, a.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.N, a.K, a.K, kFlatRows, kK))
    return cudaErrorInvalidValue;
  // as many CTAs as fit two to an SM, with two blocks each at least
  int64_t split = 2 * (int64_t)sms / (tiles * rows);
  if (split > nkb / 2) split = nkb / 2;
  if (split > kMaxSplit) split = kMaxSplit;
  if (split < 1) split = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * split), (unsigned)rows);
  cfg.blockDim = dim3(kFlatThreads);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  TraceScope ts("kda_matmul_fp8_flat", st);
  return cudaLaunchKernelEx(&cfg, flat_kernel<BN, Tout>(a.waits), maps, a.a_scale, a.b_scale, static_cast<Tout*>(a.out), (int)a.M, a.N, nkb,
                            (int)split, a.err);
}

template <typename Tout>
cudaError_t launch(const MatmulArgs& a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = prepare_device(&sms);
  if (e != cudaSuccess) return e;
  const int64_t tiles_m = (a.M + kTallM - 1) / kTallM, tiles = tiles_m * ((a.N + kTallN - 1) / kTallN);
  // Few rows, or so few tiles that most SMs would have none.  flat against tall: 64 x 12288 x 4096 15.4 against
  // 21.0 us; 256 x 4096 x 4096, 32 tiles of 152 SMs, 17.0 against 21.7; 128 x 12288 x 4096, 48 tiles, 23.1 against
  // 21.2 (17.1 in pairs).  As narrow as the rows allow: 16 x 12288 x 4096 12.6 us with 16, 16.9 with 64; 32 rows 13.1 and 14.8.
  if (a.M <= 16) return launch_flat<16, Tout>(a, sms, st);
  if (a.M <= 32) return launch_flat<32, Tout>(a, sms, st);
  if (a.M <= 64 || tiles * 4 < sms) return launch_flat<64, Tout>(a, sms, st);
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  Maps maps;
  if (!tensor_map_2d(&maps.a, a.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.M, a.K, a.K, kTallM, kK) ||
      !tensor_map_2d(&maps.b, a.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.N, a.K, a.K, kTallN, kK))
    return cudaErrorInvalidValue;
  const int nkb = (a.K + kK - 1) / kK;
  // Two CTAs to a tile where every pair is resident and each has eight blocks: 128 x 12288 x 4096, 48 tiles, 17.1
  // against 21.4 us; 512 x 4096 x 4096, 64 tiles, 18.2 against 21.4; four blocks, 512 x 4096 x 512, 15.2 against 12.8.
  const bool pair = 2 * tiles <= sms && nkb >= 16;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(pair ? 2 * tiles : tiles < sms ? tiles : sms));
  cfg.blockDim = dim3(kTallThreads);
  cfg.dynamicSmemBytes = kTallSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 1 : 0;
  TraceScope ts("kda_matmul_fp8_tall", st);
  auto* kernel = pair ? tall_kernel<Tout, true>(a.waits) : tall_kernel<Tout, false>(a.waits);
  return cudaLaunchKernelEx(&cfg, kernel, maps, a.a_scale, a.b_scale, static_cast<Tout*>(a.out), (int)a.M, a.N, nkb,
                            (int)tiles_m, (int)tiles, a.err);
}

}  // namespace

cudaError_t matmul_fp8_launch(const MatmulArgs& a, cudaStream_t st) {
  return a.out_bf16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}

}  // namespace kda
