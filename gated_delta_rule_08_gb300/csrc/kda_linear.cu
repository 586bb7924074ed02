// Linear attention with one decay per head: the recurrent forms.
//
// Per (sequence or request, head), state S in R^{dk x dv} (rows = key channels):
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// the KDA recurrence (section 2.2 Eq. 1) without the delta rule's erase and with a scalar decay.
//
// linear_recurrent_kernel: whole sequences of fp32 inputs, token by token (bf16: kda_linear_tc.cu), so that fp32
// inputs are multiplied as fp32.  Value columns are independent of one another, so a CTA takes 16 of them for the
// whole sequence and keeps its dk x 16 slice of the state in registers; a thread owns dk / 8 rows of one column.
// Decays come in two parts (decay_low), by a fifth warp that works a stage ahead: with e^g as one fp32 number the
// states were off by 1.3e-5 at g = -2^-8 and by 2e-4 over 8192 tokens at -1e-5, with two by 2.9e-7 and 1.6e-6, which
// is what rounding the state once a token leaves.
// Bound by the chain of tokens: ~110 ns a token at dk = 64 and ~138 ns at 128 (1024 tokens of one sequence: 112 and
// 141 us; with single decays 96 and 134); with every SM busy by the instructions (8 x 1024 tokens, H = 32, d = 128:
// 1.15 ms).
//
// linear_step_kernel: one token per request on a pool of states, in place (section 13.9's pooled
// layout).  It streams each state in and out once.
#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

// ------------------------------------------------------------------------------ sequences
constexpr int kCols = 16;  // value columns of a CTA
constexpr int kTile = 8;   // tokens of a stage
constexpr int kRecStages = 6;  // the copies run five stages ahead: a token takes less time than a load
constexpr int kRecThreads = 128;  // and a warp that makes the decays

template <int DK>
struct RecStage {
  float k[kTile][DK], q[kTile][DK], v[kTile][kCols];
};

// 16 bytes of global memory to shared memory without registers; zeros if not `in`
__device__ __forceinline__ void cp_async_zero(void* dst, const void* src, bool in) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(in ? 16 : 0) : "memory");
}

// Two fp32 lanes an instruction, each rounded as the scalar operation.
__device__ __forceinline__ uint64_t pair2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

template <int DK, typename Tout>
__global__ void __launch_bounds__(kRecThreads + 32)
linear_recurrent_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v,
                        int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* __restrict__ g,
                        int g_per_token, const float* h0, const int32_t* __restrict__ cu, Tout* __restrict__ out,
                        float* hT, int B, int64_t T, int64_t T_tot, int H, int dv, float scale,
                        unsigned int* __restrict__ err) {
  constexpr int NI = DK / 32;  // groups of four rows of a thread
  extern __shared__ __align__(16) uint8_t rec_smem[];
  RecStage<DK>* stages = reinterpret_cast<RecStage<DK>*>(rec_smem);
  __shared__ float so[kTile][kCols];
  __shared__ float2 se[2][kTile];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slices = dv / kCols;
  const int slice = blockIdx.x % slices, bh = blockIdx.x / slices, h = bh % H, b = bh / H;
  int64_t t0 = (int64_t)b * T;
  int n = (int)T;  // token counts fit 32 bits
  if (cu != nullptr) {
    if (!offsets_ok(cu, B, T_tot)) {
      if (tid == 0) atomicOr(err, KDA_DEVERR_BAD_SEQLENS);
      return;
    }
    t0 = cu[b];
    n = cu[b + 1] - cu[b];
  }
  if (warp == kRecThreads / 32) {
    // The decays of a stage, in two parts: made while the stage before is worked on, from values loaded while the
    // one before that was.  Tokens past the sequence have none.
    const float* pg = g + (g_per_token ? (t0 + lane) * H + h : h);
    const int64_t g_step = g_per_token ? (int64_t)kTile * H : 0;
    auto decays = [&](float x) {
      const float e = expf(x);
      return make_float2(e, decay_low(x, e));
    };
    float g_next = lane < kTile && lane < n ? *pg : 0.f;
    int par = 0;
#pragma unroll 1
    for (int c = 0; c < n; c += kTile) {
      const float x = g_next;
      pg += g_step;
      g_next = lane < kTile && c + kTile + lane < n ? *pg : 0.f;
      if (lane < kTile) se[par][lane] = decays(x);
      par ^= 1;
      __syncthreads();
      __syncthreads();
    }
    return;
  }
  const int rg = lane & 7, col = warp * 4 + (lane >> 3);
  const int64_t soff = ((int64_t)b * H + h) * DK * dv + slice * kCols + col;
  uint64_t s[NI][2];  // pairs of rows
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float* at = h0 + soff + (int64_t)(32 * i + 4 * rg + 2 * j) * dv;
      s[i][j] = h0 ? pair2(at[0], at[dv]) : 0;
    }

  // This thread's pieces of a stage: a row of k and q every kRowStep tokens, a piece of v, a decay.  Tokens past
  // the sequence come as zeros with no decay (read from the sequence's first, of size 0).
  constexpr int kRowStep = kRecThreads / (DK / 4), kRows = kTile / kRowStep;
  const int r0 = tid / (DK / 4), d0 = tid % (DK / 4) * 4, rv = tid / (kCols / 4), dv0 = tid % (kCols / 4) * 4;
  const float* pk = k + (t0 + r0) * k_stride + h * DK + d0;
  const float* pq = q + (t0 + r0) * q_stride + h * DK + d0;
  const float* pv = v + (t0 + rv) * v_stride + (int64_t)h * dv + slice * kCols + dv0;
  int fetched = 0, put = 0;
  auto fetch = [&] {
    if (fetched < n) {
      RecStage<DK>& st = stages[put];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i * kRowStep;
        const bool in = fetched + r < n;
        cp_async_zero(&st.k[r][d0], in ? pk + i * kRowStep * k_stride : k, in);
        cp_async_zero(&st.q[r][d0], in ? pq + i * kRowStep * q_stride : q, in);
      }
      if (tid < kTile * kCols / 4) cp_async_zero(&st.v[rv][dv0], fetched + rv < n ? pv : v, fetched + rv < n);
      pk += kTile * k_stride;
      pq += kTile * q_stride;
      pv += kTile * v_stride;
      fetched += kTile;
      put = put + 1 < kRecStages ? put + 1 : 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kRecStages - 1; ++i) fetch();
  Tout* po = out + ((t0 + tid / kCols) * H + h) * dv + slice * kCols + tid % kCols;
  int get = 0, par = 0;
#pragma unroll 1
  for (int c = 0; c < n; c += kTile) {
    const int m = n - c < kTile ? n - c : kTile;
    asm volatile("cp.async.wait_group %0;" ::"n"(kRecStages - 2) : "memory");
    __syncthreads();  // this stage has landed, and the one before has been read and its outputs stored
    fetch();
    const RecStage<DK>& st = stages[get];
    get = get + 1 < kRecStages ? get + 1 : 0;
    // Four tokens at a time: their states follow one another, but nothing else does, so the loads and the
    // read-outs of one run beside the others'.
#pragma unroll 1
    for (int t = 0; t < kTile; t += 4) {
      float acc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 e = se[par][t + u];
        const float x = st.v[t + u][col];
        const uint64_t e2 = pair2(e.x, e.x), low2 = pair2(e.y, e.y), x2 = pair2(x, x);
        uint64_t a = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const ulonglong2 k4 = *reinterpret_cast<const ulonglong2*>(&st.k[t + u][32 * i + 4 * rg]);
          const ulonglong2 q4 = *reinterpret_cast<const ulonglong2*>(&st.q[t + u][32 * i + 4 * rg]);
          s[i][0] = fma2(e2, s[i][0], fma2(k4.x, x2, mul2(low2, s[i][0])));
          s[i][1] = fma2(e2, s[i][1], fma2(k4.y, x2, mul2(low2, s[i][1])));
          a = fma2(q4.x, s[i][0], a);
          a = fma2(q4.y, s[i][1], a);
        }
        acc[u] = split2(a).x + split2(a).y;
      }
      // sums over the eight row groups; lane rg keeps token t + (rg & 3)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float give = rg & 1 ? acc[2 * u] : acc[2 * u + 1];
        acc[u] = (rg & 1 ? acc[2 * u + 1] : acc[2 * u]) + __shfl_xor_sync(0xffffffffu, give, 1);
      }
      float o = (rg & 2 ? acc[1] : acc[0]) + __shfl_xor_sync(0xffffffffu, rg & 2 ? acc[0] : acc[1], 2);
      o += __shfl_xor_sync(0xffffffffu, o, 4);
      if (rg < 4) so[t + rg][col] = o;
    }
    __syncthreads();
    static_assert(kTile * kCols == kRecThreads, "one output a thread");
    if (tid < m * kCols) *po = from_f32<Tout>(scale * (&so[0][0])[tid]);
    po += (int64_t)kTile * H * dv;
    par ^= 1;
  }
  if (hT) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float* at = hT + soff + (int64_t)(32 * i + 4 * rg + 2 * j) * dv;
        at[0] = split2(s[i][j]).x;
        at[dv] = split2(s[i][j]).y;
      }
  }
}

template <typename Tout>
cudaError_t recurrent_typed(const LinearArgs& a, cudaStream_t st) {
  const int64_t grid = (int64_t)a.B * a.H * (a.dv / kCols);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  static DeviceOnce once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  constexpr int kSmem = kRecStages * (int)sizeof(RecStage<128>);
  const cudaError_t e = once.run(dev, [] {
    return cudaFuncSetAttribute(linear_recurrent_kernel<128, Tout>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  auto* kernel = a.dk == 64 ? linear_recurrent_kernel<64, Tout> : linear_recurrent_kernel<128, Tout>;
  TraceScope ts("kda_linear_recurrent", st);
  kernel<<<(unsigned)grid, kRecThreads + 32, a.dk == 64 ? kRecStages * sizeof(RecStage<64>) : kSmem, st>>>(
      static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v), a.q_stride,
      a.k_stride, a.v_stride, a.g, a.g_per_token, a.h0, a.cu_seqlens, static_cast<Tout*>(a.out), a.hT, a.B, a.T, a.T_tot, a.H,
      a.dv, a.scale, a.err);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------------ one token
constexpr int kStepThreads = 256;

// CTA = (request, head).  A thread owns four columns of DK / NG consecutive rows, so a warp's state accesses are
// whole 128-bit pieces of a row; the state stays in registers between load and store.
//
// Bound by the states' bytes, read once and written once: 256 requests x 32 heads of 128 x 128 take 156 us,
// 6.8 TB/s (the rate of a plain copy).  Few requests are bound by the latency of a load, a product and a store:
// 32 states 2.9 us, 128 states 3.1 us.
template <int DK, int DV, typename Tin, typename Tout>
__global__ void __launch_bounds__(kStepThreads)
linear_step_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v, int64_t q_stride,
                   int64_t k_stride, int64_t v_stride, const float* __restrict__ g, int g_per_token,
                   float* __restrict__ pool, const int32_t* __restrict__ slot_idx, Tout* __restrict__ out, int H,
                   int num_slots, float scale, unsigned int* __restrict__ err) {
  constexpr int TPR = DV / 4;               // threads per row
  constexpr int NG = kStepThreads / TPR;    // row groups
  constexpr int RPG = DK / NG;              // rows per thread
  static_assert(DK % NG == 0, "rows must split evenly");
  __shared__ __align__(16) float sk[DK], sq[DK];
  __shared__ __align__(16) float4 part[NG][TPR];

  const int nh = blockIdx.x, n = nh / H, h = nh - n * H;
  const int tid = threadIdx.x, cg = tid % TPR, rg = tid / TPR;
  const int slot = slot_idx[n];
  if (slot < 0 || slot >= num_slots) {
    if (tid == 0 && h == 0) atomicOr(err, KDA_DEVERR_BAD_SLOT);
    return;
  }
  float* S = pool + ((int64_t)slot * H + h) * (DK * DV) + 4 * cg;
  float4 s[RPG];
#pragma unroll
  for (int i = 0; i < RPG; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(S + (rg * RPG + i) * DV));

  const float log_decay = g[g_per_token ? (int64_t)nh : h];
  float2 e;
  e.x = expf(log_decay);
  e.y = decay_low(log_decay, e.x);
  for (int i = tid; i < DK; i += kStepThreads) {
    sk[i] = to_f32(k[n * k_stride + h * DK + i]);
    sq[i] = to_f32(q[n * q_stride + h * DK + i]);
  }
  float4 x;
  {
    const Tin* vp = v + n * v_stride + h * DV + 4 * cg;
    x = make_float4(to_f32(vp[0]), to_f32(vp[1]), to_f32(vp[2]), to_f32(vp[3]));
  }
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < RPG; ++i) {
    const float kk = sk[rg * RPG + i], qq = sq[rg * RPG + i];
    s[i] = make_float4(decay_add(e, s[i].x, kk, x.x), decay_add(e, s[i].y, kk, x.y), decay_add(e, s[i].z, kk, x.z),
                       decay_add(e, s[i].w, kk, x.w));
    __stcs(reinterpret_cast<float4*>(S + (rg * RPG + i) * DV), s[i]);
    acc = f4_fma(qq, s[i], acc);
  }
  part[rg][cg] = acc;
  __syncthreads();
  if (tid < DV) {
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) o += reinterpret_cast<const float*>(part[i])[tid];
    out[(int64_t)nh * DV + tid] = from_f32<Tout>(scale * o);
  }
}

template <int DK, int DV, typename Tin, typename Tout>
cudaError_t step_sized(const LinearStepArgs& a, cudaStream_t st) {
  TraceScope ts("kda_linear_step", st);
  linear_step_kernel<DK, DV, Tin, Tout><<<(unsigned)(a.N * a.H), kStepThreads, 0, st>>>(
      static_cast<const Tin*>(a.q), static_cast<const Tin*>(a.k), static_cast<const Tin*>(a.v), a.q_stride, a.k_stride,
      a.v_stride, a.g, a.g_per_token, a.state_pool, a.slot_idx, static_cast<Tout*>(a.out), a.H, a.num_slots, a.scale,
      a.err);
  return cudaGetLastError();
}
template <typename Tin, typename Tout>
cudaError_t step_typed(const LinearStepArgs& a, cudaStream_t st) {
  if (a.dk == 64) return a.dv == 64 ? step_sized<64, 64, Tin, Tout>(a, st) : step_sized<64, 128, Tin, Tout>(a, st);
  return a.dv == 64 ? step_sized<128, 64, Tin, Tout>(a, st) : step_sized<128, 128, Tin, Tout>(a, st);
}

}  // namespace

cudaError_t linear_recurrent_launch(const LinearArgs& a, cudaStream_t st) {
  return a.out_bf16 ? recurrent_typed<__nv_bfloat16>(a, st) : recurrent_typed<float>(a, st);
}

cudaError_t linear_step_launch(const LinearStepArgs& a, cudaStream_t st) {
  if (a.bf16) return a.out_bf16 ? step_typed<__nv_bfloat16, __nv_bfloat16>(a, st) : step_typed<__nv_bfloat16, float>(a, st);
  return a.out_bf16 ? step_typed<float, __nv_bfloat16>(a, st) : step_typed<float, float>(a, st);
}

}  // namespace kda
