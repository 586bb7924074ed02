// C-ABI entry points of the operators around a recurrent layer: argument validation and dispatch.
// The public contract is include/kda.h.
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_internal.h"

#define KDA_API extern "C" __attribute__((visibility("default")))

using namespace kda;

namespace {

bool dims_ok(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }
bool dtype_ok(kda_dtype d) { return d == KDA_DTYPE_BF16 || d == KDA_DTYPE_FP32; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Sequences, tokens and heads of a linear attention call (32-bit token numbers and grids).
bool counts_ok(int B, int64_t T_tot, int H) { return T_tot <= kMaxTokens && B <= 16384 && (int64_t)B * H <= 0x7fffffff / 64; }

// Row strides of q, k, v (elements): rows may not overlap, and each must start on a 16-byte boundary.
bool stride_ok(int64_t stride, int64_t row, kda_dtype d) {
  return stride >= row && stride < ((int64_t)1 << 32) && stride % (d == KDA_DTYPE_BF16 ? 8 : 4) == 0;
}

kda_status ready(unsigned int** err) {
  bool supported = false;
  if (!device_ready(err, &supported)) return KDA_ERR_CUDA;
  return supported ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

}  // namespace

KDA_API size_t kda_linear_chunk_fwd_workspace_size(int B, int64_t T, int H, int dk, int dv, kda_dtype dtype) {
  if (B <= 0 || T < 0 || H <= 0 || !dims_ok(dk, dv) || !dtype_ok(dtype) || !counts_ok(B, T, H)) return 0;
  return 256 + (dtype == KDA_DTYPE_BF16 ? linear_tc_workspace(B, T, H, dk, dv) : 0);
}

KDA_API kda_status kda_linear_chunk_fwd(const void* q, const void* k, const void* v, const float* g, int g_per_token,
                                        const float* h0, const int32_t* cu_seqlens, void* out, float* hT, int B,
                                        int64_t T, int H, int dk, int dv, int64_t q_stride, int64_t k_stride,
                                        int64_t v_stride, float scale, kda_dtype dtype, kda_dtype out_dtype,
                                        void* workspace, size_t workspace_bytes, void* stream) {
  if (B <= 0 || T < 0 || H <= 0) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype) || !dims_ok(dk, dv)) return KDA_ERR_UNSUPPORTED;
  if (!cu_seqlens && T > ((int64_t)1 << 40) / B) return KDA_ERR_UNSUPPORTED;
  const int64_t T_tot = cu_seqlens ? T : (int64_t)B * T;
  if (!counts_ok(B, T_tot, H)) return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(q_stride, (int64_t)H * dk, dtype) || !stride_ok(k_stride, (int64_t)H * dk, dtype) ||
      !stride_ok(v_stride, (int64_t)H * dv, dtype))
    return KDA_ERR_INVALID_ARG;
  if (T_tot > 0 && (!q || !k || !v || !g || !out)) return KDA_ERR_INVALID_ARG;
  if (out && (out == q || out == k || out == v || out == (const void*)g)) return KDA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(h0) || !aligned16(hT) ||
      !aligned4(g) || !aligned4(cu_seqlens))
    return KDA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kda_linear_chunk_fwd_workspace_size(B, T, H, dk, dv, dtype) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return KDA_ERR_WORKSPACE;
  unsigned int* err = nullptr;
  const kda_status st = ready(&err);
  if (st != KDA_OK) return st;
  LinearArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.g = g; a.g_per_token = g_per_token != 0; a.h0 = h0; a.cu_seqlens = cu_seqlens; a.out = out; a.hT = hT;
  a.B = B; a.T = T; a.T_tot = T_tot; a.H = H; a.dk = dk; a.dv = dv; a.scale = scale;
  a.bf16 = dtype == KDA_DTYPE_BF16; a.out_bf16 = out_dtype == KDA_DTYPE_BF16;
  a.workspace = workspace; a.err = err; a.waits = test_wait_timeout();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(a.bf16 ? linear_tc_launch(a, s) : linear_recurrent_launch(a, s));
}

KDA_API kda_status kda_linear_decode_step(const void* q, const void* k, const void* v, const float* g, int g_per_token,
                                          float* state_pool, const int32_t* slot_idx, void* out, int N, int H, int dk,
                                          int dv, int num_slots, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                          float scale, kda_dtype dtype, kda_dtype out_dtype, void* stream) {
  if (N < 0 || H <= 0 || num_slots < 0) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype) || !dims_ok(dk, dv)) return KDA_ERR_UNSUPPORTED;
  if ((int64_t)N * H > 0x7fffffff / 8) return KDA_ERR_UNSUPPORTED;
  if (!stride_ok(q_stride, (int64_t)H * dk, dtype) || !stride_ok(k_stride, (int64_t)H * dk, dtype) ||
      !stride_ok(v_stride, (int64_t)H * dv, dtype))
    return KDA_ERR_INVALID_ARG;
  if (N > 0 && (!q || !k || !v || !g || !state_pool || !slot_idx || !out)) return KDA_ERR_INVALID_ARG;
  if (!aligned16(state_pool) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4(g) ||
      !aligned4(slot_idx))
    return KDA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  const kda_status st = ready(&err);
  if (st != KDA_OK) return st;
  if (N == 0) return KDA_OK;
  LinearStepArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.g = g; a.g_per_token = g_per_token != 0; a.state_pool = state_pool; a.slot_idx = slot_idx; a.out = out;
  a.N = N; a.H = H; a.dk = dk; a.dv = dv; a.num_slots = num_slots; a.scale = scale;
  a.bf16 = dtype == KDA_DTYPE_BF16; a.out_bf16 = out_dtype == KDA_DTYPE_BF16; a.err = err;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (debug_checks() && check_slots(slot_idx, N, num_slots, err, s) != cudaSuccess) return KDA_ERR_CUDA;
  return done(linear_step_launch(a, s));
}

KDA_API kda_status kda_rmsnorm_quant(const void* x, const void* residual, const float* weight, void* residual_out,
                                     void* y, float* y_scale, int64_t rows, int D, float eps, kda_dtype dtype,
                                     void* stream) {
  if (rows < 0 || D <= 0 || !(eps >= 0.f)) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(dtype) || D % 16 != 0 || D > 32768 || rows > 0x7fffffff) return KDA_ERR_UNSUPPORTED;
  if (rows > 0 && (!x || !y || !y_scale)) return KDA_ERR_INVALID_ARG;
  if (residual_out && !residual) return KDA_ERR_INVALID_ARG;
  if (y && (y == x || y == residual || y == residual_out)) return KDA_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned4(y_scale))
    return KDA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  const kda_status st = ready(&err);
  if (st != KDA_OK) return st;
  if (rows == 0) return KDA_OK;
  NormQuantArgs a{};
  a.x = x; a.residual = residual; a.weight = weight; a.residual_out = residual_out;
  a.y = static_cast<uint8_t*>(y); a.y_scale = y_scale; a.rows = rows; a.D = D; a.eps = eps;
  a.bf16 = dtype == KDA_DTYPE_BF16;
  return done(rmsnorm_quant_launch(a, static_cast<cudaStream_t>(stream)));
}

KDA_API kda_status kda_matmul_fp8(const void* a, const float* a_scale, const void* b, const float* b_scale, void* out,
                                  int64_t M, int N, int K, kda_dtype out_dtype, void* stream) {
  if (M < 0 || N <= 0 || K <= 0) return KDA_ERR_INVALID_ARG;
  if (!dtype_ok(out_dtype) || K % 16 != 0 || M > (1 << 22) || N > (1 << 22) || K > (1 << 22)) return KDA_ERR_UNSUPPORTED;
  if (M > 0 && (!a || !a_scale || !b || !b_scale || !out)) return KDA_ERR_INVALID_ARG;
  if (out && (out == a || out == b || out == (const void*)a_scale || out == (const void*)b_scale)) return KDA_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned4(a_scale) || !aligned4(b_scale))
    return KDA_ERR_INVALID_ARG;
  unsigned int* err = nullptr;
  const kda_status st = ready(&err);
  if (st != KDA_OK) return st;
  if (M == 0) return KDA_OK;
  MatmulArgs m{};
  m.a = static_cast<const uint8_t*>(a); m.a_scale = a_scale; m.b = static_cast<const uint8_t*>(b); m.b_scale = b_scale;
  m.out = out; m.M = M; m.N = N; m.K = K; m.out_bf16 = out_dtype == KDA_DTYPE_BF16; m.err = err;
  m.waits = test_wait_timeout();
  return done(matmul_fp8_launch(m, static_cast<cudaStream_t>(stream)));
}
