// RMS norm with the residual's addition and an 8-bit output with scales.
//
//   z = x + r (fp32),  y = z / sqrt(mean z^2 + eps) w
//   per block of 128 values of a row (the last may be shorter): s = max(max|y|, 1e-30) / 448,
//   q = e4m3(y / s), so that the block's largest value becomes 448, the largest e4m3 number.
// The norm and the scales come from the unrounded fp32 sum z; the stored z is rounded once to its
// type, and each y / s once to e4m3 (by way of one reciprocal a block, so the quotient is off by a step of
// fp32 at most before it is rounded to 4 bits; sixteen divisions a thread cost 4 of 47 us at 8192 x 4096).
// A block of zeros keeps the scale 1e-30 / 448.
//
// A thread keeps 16 consecutive values of a row in registers between the two reductions, so the data
// are read once; eight neighbouring lanes hold one block of 128.  Bound by HBM: 7 bytes per value for
// bf16 with a residual.
#include <cuda_fp8.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kBlock = 128;
constexpr float kFp8Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;

__device__ __forceinline__ void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
      w[j] = *reinterpret_cast<const uint32_t*>(&t);
    }
    reinterpret_cast<uint4*>(p)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// TR threads share a row (a power of two, at least 8), each with UNITS pieces of 16 values, TR pieces
// apart; a CTA of max(TR, 128) threads holds 128 / TR rows when TR < 128.
template <int TR, int UNITS, typename T>
__global__ void __launch_bounds__(TR > 128 ? TR : 128)
rmsnorm_quant_kernel(const T* x, const T* residual, const float* __restrict__ weight, T* residual_out,
                     uint8_t* __restrict__ y, float* __restrict__ y_scale, int64_t rows, int D, float eps) {
  constexpr int kThreads = TR > 128 ? TR : 128;
  constexpr int kRows = kThreads / TR;
  const int tid = threadIdx.x, t = tid % TR;
  const int64_t row = (int64_t)blockIdx.x * kRows + tid / TR;
  const bool live = row < rows;
  const int64_t base = (live ? row : 0) * D;
  float z[UNITS][16];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = (u * TR + t) * 16;
    const bool in = live && c < D;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[u][i] = 0.f;
    if (in) {
      load16(x + base + c, z[u]);
      if (residual != nullptr) {
        float r[16];
        load16(residual + base + c, r);
#pragma unroll
        for (int i = 0; i < 16; ++i) z[u][i] += r[i];
        if (residual_out != nullptr) store16(residual_out + base + c, z[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(z[u][i], z[u][i], sum);
  }
#pragma unroll
  for (int o = (TR < 32 ? TR : 32) / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (TR > 32) {
    constexpr int kWarps = TR / 32;
    __shared__ float red[kThreads / 32];
    if ((tid & 31) == 0) red[tid / 32] = sum;
    __syncthreads();
    const float* r = red + (tid / TR) * kWarps;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += r[i];
  }
  const float inv = rsqrtf(sum / (float)D + eps);
  const int nblk = (D + kBlock - 1) / kBlock;
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = (u * TR + t) * 16;
    const bool in = live && c < D;
    float amax = 0.f;
    float w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = 1.f;
    if (in && weight != nullptr) load16(weight + c, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      z[u][i] = z[u][i] * inv * w[i];
      // not fmaxf, which would drop a NaN: the block's scale must show it
      const float m = fabsf(z[u][i]);
      amax = (m > amax || isnan(m)) ? m : amax;
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, amax, o);
      amax = (m > amax || isnan(m)) ? m : amax;
    }
    const float s = (amax < kAmaxFloor ? kAmaxFloor : amax) / kFp8Max;
    const float rs = 1.f / s;
    if (in) {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_fp8x4_e4m3 f(make_float4(z[u][4 * i] * rs, z[u][4 * i + 1] * rs, z[u][4 * i + 2] * rs, z[u][4 * i + 3] * rs));
        p[i] = f.__x;
      }
      *reinterpret_cast<uint4*>(y + base + c) = make_uint4(p[0], p[1], p[2], p[3]);
      if ((t & 7) == 0) y_scale[row * nblk + c / kBlock] = s;
    }
  }
}

template <int TR, int UNITS, typename T>
cudaError_t launch(const NormQuantArgs& a, cudaStream_t st) {
  constexpr int kThreads = TR > 128 ? TR : 128;
  const int64_t grid = (a.rows + kThreads / TR - 1) / (kThreads / TR);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  TraceScope ts("kda_rmsnorm_quant", st);
  rmsnorm_quant_kernel<TR, UNITS, T><<<(unsigned)grid, kThreads, 0, st>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual), a.weight, static_cast<T*>(a.residual_out), a.y,
      a.y_scale, a.rows, a.D, a.eps);
  return cudaGetLastError();
}
template <typename T>
cudaError_t dispatch(const NormQuantArgs& a, cudaStream_t st) {
  const int units = (a.D + 15) / 16;  // the smallest power of two of threads that covers a row
  if (units <= 8) return launch<8, 1, T>(a, st);
  if (units <= 16) return launch<16, 1, T>(a, st);
  if (units <= 32) return launch<32, 1, T>(a, st);
  if (units <= 64) return launch<64, 1, T>(a, st);
  if (units <= 128) return launch<128, 1, T>(a, st);
  // Many long rows: half the threads with twice the values each (8192 x 4096: 41.5 against 43.5 us); few rows are
  // done sooner with more threads (1 x 4096: 2.8 against 2.4 us).
  const bool many = a.rows >= 2048;
  if (units <= 256) return many ? launch<128, 2, T>(a, st) : launch<256, 1, T>(a, st);
  if (units <= 512) return many ? launch<256, 2, T>(a, st) : launch<512, 1, T>(a, st);
  if (units <= 1024) return many ? launch<512, 2, T>(a, st) : launch<1024, 1, T>(a, st);
  return launch<1024, 2, T>(a, st);
}

}  // namespace

cudaError_t rmsnorm_quant_launch(const NormQuantArgs& a, cudaStream_t st) {
  return a.bf16 ? dispatch<__nv_bfloat16>(a, st) : dispatch<float>(a, st);
}

}  // namespace kda
