// Shared definitions of the tensor-core prefill kernels: the per-(chunk, head) record
// exchanged between the chunk-parallel kernel and the scan, swizzled shared-memory
// addressing, and thin wrappers over tcgen05 / TMEM / named barriers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kda_device.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace tcx {

using namespace tc;

// ----------------------------------------------------------------- record layout (bytes)
// Every operand block is fp16 in "row format": 128-byte rows of 64 values, 8-row atoms with the
// 128-byte swizzle (row_chunk below).  The scan feeds two fused products from the staged part:
//   [D_U | D_O] = S^T [W^T | Q_hat^T]  (B MN-major: two 64-column blocks 16 KB apart)
//   [D_O | S^T] += U^T [M ; K_bar^T]^T (B K-major: 192 rows, M directly followed by K_bar^T)
constexpr uint32_t kRecWT = 0;          // W^T     [128 dk][64 r]
constexpr uint32_t kRecQT = 16384;      // Q_hat^T [128 dk][64 r]
constexpr uint32_t kRecMM = 32768;      // M       [64 r][64 s]
constexpr uint32_t kRecKT = 40960;      // K_bar^T [128 dk][64 r]
constexpr uint32_t kRecGC = 57344;      // e^{G_C} [128] fp32
constexpr uint32_t kRecStage = 57856;   // bytes the scan kernel stages in shared memory
constexpr uint32_t kRecUT = 59392;      // U_hat^T [128 dv][64 r] (read from global)
constexpr uint32_t kRecBytes = 75776;   // 74 KB

// ----------------------------------------------------------------- swizzled addressing
// fp16 [R rows][64 cols] row format: chunk j (cols 8j..8j+7) of row r.
__device__ __forceinline__ uint32_t row_chunk(int r, int j) {
  return (uint32_t)r * 128u + ((((uint32_t)j ^ (uint32_t)r) & 7u) << 4);
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h2(uint32_t u) {
  __half2 h = *reinterpret_cast<__half2*>(&u);
  return __half22float2(h);
}
__device__ __forceinline__ float2 unpack_bf2(uint32_t u) {
  __nv_bfloat162 h = *reinterpret_cast<__nv_bfloat162*>(&u);
  return __bfloat1622float2(h);
}
__device__ __forceinline__ uint4 pack8_h(const float* v) {
  uint4 w;
  w.x = pack_h2(v[0], v[1]);
  w.y = pack_h2(v[2], v[3]);
  w.z = pack_h2(v[4], v[5]);
  w.w = pack_h2(v[6], v[7]);
  return w;
}

constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (0u << 7) | (0u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  mma_bf16_ss(d, a, b, idesc, acc);  // same instruction form; the descriptor selects f16
}
// A shared-memory descriptor advanced by `bytes` (start-address field, 16-byte units;
// shared addresses stay below 256 KB, so the 14-bit field never carries).
__device__ __forceinline__ uint64_t desc_add(uint64_t d, uint32_t bytes) { return d + (uint64_t)(bytes >> 4); }

__device__ __forceinline__ uint32_t tmem_lane(uint32_t base, int warp) {
  return base + ((uint32_t)((warp & 3) * 32) << 16);
}
// Named barrier over `n` threads returning the AND of `v` across them.
__device__ __forceinline__ bool group_and(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}


// MMA with the A operand in TMEM (lane = row, fp16 pairs packed two per 32-bit column, the
// even K index in the low half) and B from a shared-memory descriptor.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st32u(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
// Bounded mbarrier wait that also gives up once another role has raised the CTA's abort flag;
// a wait that runs out raises the flag itself.
__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              uint32_t max_spins = kWaitTries) {
  for (uint32_t i = 0; i < max_spins; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 63u && *abort_flag) return false;
  }
  *abort_flag = 1;
  return false;
}
// The same wait in a kernel variant built to test the abort path: with kGiveUp it gives up at
// once (raises the abort flag without polling), which is what a wait that runs out does.
template <bool kGiveUp>
__device__ __forceinline__ bool wait_or_abort_t(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if constexpr (kGiveUp) {
    *abort_flag = 1;
    return false;
  } else {
    return wait_or_abort(bar, parity, abort_flag);
  }
}

__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// What a kernel's waits do: the product's; the variant whose waits give up at once; and the one whose first CTA
// starts no MMA, so that its waits run out by themselves while the other CTAs go on (both for tests).
enum Waits : int { kWaits = 0, kWaitsGiveUp = 1, kFirstCtaStalls = 2 };

// Where other warps of a CTA are at a cluster barrier, a try_wait returns at once instead of blocking.  The waits
// below, which clusters use, therefore keep late tries at least 4 us apart: half a second to a second in all.  (In
// wait_or_abort the pause costs the KDA prefill 337 -> 348 us without being reached.)
constexpr uint32_t kPausedTries = 130000u, kQuickTries = 4096u;
__device__ __forceinline__ void pause_after(uint32_t tries) {
  if (tries >= kQuickTries) __nanosleep(4000);
}
// wait_or_abort_t for hand-overs that take less than a microsecond: polls first (a poll takes 15 clocks),
// because a thread that try_wait has suspended comes back some hundreds of clocks late.
template <bool kGiveUp>
__device__ __forceinline__ bool spin_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if constexpr (!kGiveUp) {
    for (int i = 0; i < 2048; ++i) {
      if (mbar_test_wait(bar, parity)) return true;
      if ((i & 63) == 63 && *abort_flag) return false;
    }
    for (uint32_t i = 0; i < kPausedTries; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
      if (*abort_flag) return false;
      pause_after(i);
    }
  }
  *abort_flag = 1;
  return false;
}
// The start of dynamic shared memory, rounded up to the swizzle's 1024 bytes, as a pointer that the compiler
// still knows to be shared memory.
__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* raw) { return raw + ((0u - smem_u32(raw)) & 1023u); }

// The same for a whole warp, which stays together: every branch is on a vote.  (Lanes that leave a polling
// loop one by one, or one lane that polls for the others, stay apart afterwards, and the warp then runs the
// work that follows once for each group.)
template <bool kGiveUp, bool kSpin = false>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  if constexpr (kGiveUp) {
    *abort_flag = 1;
    return false;
  } else {
    if constexpr (kSpin) {
#pragma unroll 1
      for (uint32_t i = 0; i < 512u; ++i)
        if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    }
#pragma unroll 1
    for (uint32_t i = 0; i < kPausedTries; ++i) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
      pause_after(i);
    }
    *abort_flag = 1;
    return false;
  }
}
// ... for the warps that issue the MMAs, which everything waits for: polls at first (a suspended warp comes back
// some hundreds of clocks late), at the price of issue slots.
template <bool kGiveUp>
__device__ __forceinline__ bool warp_spin(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return warp_wait<kGiveUp, true>(bar, parity, abort_flag);
}

// One arrival for a whole warp, after all its lanes' work (each has executed the fence that work needs).
// Predicated, not branched, for the same reason.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 st;\n setp.eq.u32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 st, [%0];\n}" ::"r"(
          smem_u32(bar)),
      "r"(threadIdx.x & 31u)
      : "memory");
}

// MMAs and commits that a whole warp runs through and one lane (`leader`) issues: with warp-uniform control
// flow the descriptors stay in uniform registers, where the instruction wants them (in a branch of one lane
// every one of them is moved there first, at some 200 clocks an MMA in a busy SM).
__device__ __forceinline__ void mma_bf16_ss_by(bool leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts_by(bool leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_f8_ss_by(bool leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(leader ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit_by(bool leader, uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_u32(bar)),
      "r"(leader ? 1u : 0u)
      : "memory");
}

// Two fp32 lanes per instruction (each lane rounded as the scalar operation).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mul.rn.f32x2 rd, ra, rb;\n"
      " mov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n sub.rn.f32x2 rd, ra, rb;\n"
      " mov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
      " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Waits for this thread's TMEM loads; the values pass through, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_landed(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_landed(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
// 8 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// 8 consecutive columns of this thread's TMEM lane; valid on return.
__device__ __forceinline__ void tmem_ld8_wait(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
// The same columns of two accumulators.
__device__ __forceinline__ void tmem_ld8x2_wait(uint32_t ta, uint32_t tb, float (&v)[8], float (&w)[8]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n"
      " tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [%17];\n tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = __uint_as_float(r[i]);
    w[i] = __uint_as_float(r[8 + i]);
  }
}

// At the end of a CTA (all threads, after a barrier, so that the flag is final): if a wait ran out, the
// copies and MMAs that may still be in flight are waited for, with a limit, before shared memory and TMEM
// are given back.  Without an abort every MMA, and with it every copy, was waited for by its readers.
template <int STAGES>
__device__ __forceinline__ void drain_after_abort(volatile int* abort_flag, bool copier, bool multiplier, uint64_t* full,
                                                  int64_t issued, uint64_t* bar_fin, unsigned int* err) {
  if (!*abort_flag) return;
  if (copier) {
    for (int64_t l = issued > STAGES ? issued - STAGES : 0; l < issued; ++l)
      mbar_wait(&full[l % STAGES], (uint32_t)((l / STAGES) & 1));
    atomicOr(err, KDA_DEVERR_WAIT_TIMEOUT);
  }
  if (multiplier) {
    mma_commit(bar_fin);
    mbar_wait(bar_fin, 0);
  }
  __syncthreads();
}

}  // namespace tcx
}  // namespace kda
