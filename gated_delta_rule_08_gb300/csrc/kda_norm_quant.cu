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
// A thread keeps pieces of consecutive values of a row in registers between the two reductions, so the data are
// read once.  A piece is 8 values of fp32, 16 of bf16 (32 bytes each): neighbouring lanes hold one block of 128, and
// longer pieces save shuffles (bf16, 8192 x 4096: 41.7 against 46.6 us with pieces of 8; fp32, 1237 x 2000: 4.5
// against 3.8 us with pieces of 16).  Bound by HBM: 7 bytes per value for
// bf16 with a residual (8192 x 4096: 41.6 us, 5.7 TB/s, 84 % of a plain copy's rate; one row of 4096: 2.4 us).
#include <cuda_fp8.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kBlock = 128;
constexpr float kFp8Max = 448.f;
constexpr float kAmaxFloor = 1e-30f;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 a = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = a.x; v[4 * i + 1] = a.y; v[4 * i + 2] = a.z; v[4 * i + 3] = a.w;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&t);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// P values, eight at a time
template <int P, typename T>
__device__ __forceinline__ void load(const T* p, float (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 8) {
    float a[8];
    load8(p + i, a);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i + j] = a[j];
  }
}
template <int P, typename T>
__device__ __forceinline__ void store(T* p, const float (&v)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 8) {
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = v[i + j];
    store8(p + i, a);
  }
}

// TR threads share a row (a power of two, at least a block's 128 / P), each with UNITS pieces of P values, TR pieces
// apart; a CTA of max(TR, 128) threads holds 128 / TR rows when TR < 128.
template <typename T>
constexpr int kPiece = sizeof(T) == 2 ? 16 : 8;

template <int TR, int UNITS, typename T>
__global__ void __launch_bounds__(TR > 128 ? TR : 128)
rmsnorm_quant_kernel(const T* x, const T* residual, const float* __restrict__ weight, T* residual_out,
                     uint8_t* __restrict__ y, float* __restrict__ y_scale, int64_t rows, int D, float eps) {
  constexpr int kThreads = TR > 128 ? TR : 128;
  constexpr int kRows = kThreads / TR;
  constexpr int P = kPiece<T>, kLanes = kBlock / P;
  static_assert(TR >= kLanes, "a block lies within a row's threads");
  const int tid = threadIdx.x, t = tid % TR;
  const int64_t row = (int64_t)blockIdx.x * kRows + tid / TR;
  const bool live = row < rows;
  const int64_t base = (live ? row : 0) * D;
  float z[UNITS][P];
  float sum = 0.f;
#pragma unroll
  for (int u = 0; u < UNITS; ++u) {
    const int c = (u * TR + t) * P;
#pragma unroll
    for (int i = 0; i < P; ++i) z[u][i] = 0.f;
    if (live && c < D) {
      load(x + base + c, z[u]);
      if (residual != nullptr) {
        float r[P];
        load(residual + base + c, r);
#pragma unroll
        for (int i = 0; i < P; ++i) z[u][i] += r[i];
        if (residual_out != nullptr) store(residual_out + base + c, z[u]);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i) sum = fmaf(z[u][i], z[u][i], sum);
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
    const int c = (u * TR + t) * P;
    const bool in = live && c < D;
    float amax = 0.f;
    float w[P];
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = 1.f;
    if (in && weight != nullptr) load(weight + c, w);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      z[u][i] = z[u][i] * inv * w[i];
      // not fmaxf, which would drop a NaN: the block's scale must show it
      const float m = fabsf(z[u][i]);
      amax = (m > amax || isnan(m)) ? m : amax;
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      const float m = __shfl_xor_sync(0xffffffffu, amax, o);
      amax = (m > amax || isnan(m)) ? m : amax;
    }
    const float s = (amax < kAmaxFloor ? kAmaxFloor : amax) / kFp8Max;
    const float rs = 1.f / s;
    if (in) {
      uint32_t p[P / 4];
#pragma unroll
      for (int i = 0; i < P / 4; ++i) {
        const __nv_fp8x4_e4m3 f(make_float4(z[u][4 * i] * rs, z[u][4 * i + 1] * rs, z[u][4 * i + 2] * rs, z[u][4 * i + 3] * rs));
        p[i] = f.__x;
      }
      if constexpr (P == 16) *reinterpret_cast<uint4*>(y + base + c) = make_uint4(p[0], p[1], p[2], p[3]);
      else *reinterpret_cast<uint2*>(y + base + c) = make_uint2(p[0], p[1]);
      if (t % kLanes == 0) y_scale[row * nblk + c / kBlock] = s;
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
  constexpr int kLanes = kBlock / kPiece<T>, kUnits = 32768 / kPiece<T> / 1024;
  const int units = a.D / kPiece<T>;
  if (units <= kLanes) return launch<kLanes, 1, T>(a, st);
  if (units <= 16) return launch<16, 1, T>(a, st);
  if (units <= 32) return launch<32, 1, T>(a, st);
  if (units <= 64) return launch<64, 1, T>(a, st);
  if (units <= 128) return launch<128, 1, T>(a, st);
  // Many long rows: half the threads with twice the values each (bf16, 8192 x 4096: 41.7 against 43.5 us; fp32,
  // 1237 x 2000: 3.8 against 4.2 us); few rows are done sooner with more threads (1 x 4096: 2.8 against 2.4 us).
  const bool many = a.rows >= (sizeof(T) == 2 ? 2048 : 1024);
  if (units <= 256) return many ? launch<128, 2, T>(a, st) : launch<256, 1, T>(a, st);
  if (units <= 512) return many ? launch<256, 2, T>(a, st) : launch<512, 1, T>(a, st);
  if (units <= 1024) return many ? launch<512, 2, T>(a, st) : launch<1024, 1, T>(a, st);
  return launch<1024, kUnits, T>(a, st);
}

}  // namespace

cudaError_t rmsnorm_quant_launch(const NormQuantArgs& a, cudaStream_t st) {
  return a.bf16 ? dispatch<__nv_bfloat16>(a, st) : dispatch<float>(a, st);
}

}  // namespace kda
