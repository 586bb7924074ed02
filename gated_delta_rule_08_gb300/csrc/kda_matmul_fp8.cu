// Matrix product of e4m3 rows with a scale for each block of 128 values.
//
//   out[m][n] = sum_kb a_scale[m][kb] b_scale[n / 128][kb] sum_{k in block kb} a[m][k] b[n][k]
#include <cuda_fp8.h>

#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kTile = 64, kKs = 16;

template <typename Tout>
__global__ void __launch_bounds__(256)
matmul_fp8_kernel(const __nv_fp8_e4m3* __restrict__ a, const float* __restrict__ a_scale,
                  const __nv_fp8_e4m3* __restrict__ b, const float* __restrict__ b_scale, Tout* __restrict__ out,
                  int64_t M, int N, int K) {
  __shared__ float sa[kKs][kTile + 1], sb[kKs][kTile + 1];
  const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
  const int64_t m0 = (int64_t)blockIdx.y * kTile;
  const int n0 = blockIdx.x * kTile, kb = (K + 127) / 128;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += kKs) {  // K is a multiple of 16
    for (int i = tid; i < kTile * kKs; i += 256) {
      const int r = i / kKs, c = i % kKs, blk = (k0 + c) / 128;
      const int64_t m = m0 + r;
      const int n = n0 + r;
      sa[c][r] = m < M ? float(a[m * K + k0 + c]) * a_scale[m * kb + blk] : 0.f;
      sb[c][r] = n < N ? float(b[(int64_t)n * K + k0 + c]) * b_scale[(int64_t)(n / 128) * kb + blk] : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kKs; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[c][ty + 16 * i], sb[c][tx + 16 * j], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i;
      const int n = n0 + tx + 16 * j;
      if (m < M && n < N) out[m * N + n] = from_f32<Tout>(acc[i][j]);
    }
}

}  // namespace

cudaError_t matmul_fp8_launch(const MatmulArgs& a, cudaStream_t st) {
  const int64_t gy = (a.M + kTile - 1) / kTile;
  if (gy > 65535) return cudaErrorInvalidValue;
  const dim3 grid((a.N + kTile - 1) / kTile, (unsigned)gy);
  TraceScope ts("kda_matmul_fp8", st);
  const auto* pa = reinterpret_cast<const __nv_fp8_e4m3*>(a.a);
  const auto* pb = reinterpret_cast<const __nv_fp8_e4m3*>(a.b);
  if (a.out_bf16)
    matmul_fp8_kernel<<<grid, 256, 0, st>>>(pa, a.a_scale, pb, a.b_scale, static_cast<__nv_bfloat16*>(a.out), a.M, a.N, a.K);
  else
    matmul_fp8_kernel<<<grid, 256, 0, st>>>(pa, a.a_scale, pb, a.b_scale, static_cast<float*>(a.out), a.M, a.N, a.K);
  return cudaGetLastError();
}

}  // namespace kda
