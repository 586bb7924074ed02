// Rotary positions with one or several axes, fused with the write of keys and values to a paged cache.
//
//   angle = pos f,  (a, b) -> (a cos - b sin, b cos + a sin)  for each pair of a head's first rot values
//
// A position times a frequency has more whole turns than fp32 can hold fractions of, so the angle is taken in
// fixed point: F = f / (2 pi) 2^64 modulo 2^64 once for each pair, and pos F modulo 2^64, which wraps at whole turns by
// itself.  Its top 32 bits, as a signed fraction of a turn, go to sincospi.  That is exact to 2^-32 of a turn for every
// 32-bit position (F's own rounding, 2^-53 of it, adds at most |pos f| 2^-53).
//
// A unit of work is 16 values of one head of one token (two pieces of 16 bytes in bf16): eight pairs, or 16 values
// to copy.  A block holds the cosines and sines of its tokens in shared memory, for all their heads; each thread
// loads several units before it needs the first cosine.  Few tokens: a block has one, and its heads are spread
// over several blocks, which all make the 64 cosines (a quarter of a microsecond) rather than wait for one another.
//
// Bound by HBM for many tokens: every value read once and written once.
#include "kda_device.cuh"
#include "kda_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 3;  // units a thread has under way

struct Values {
  float x[16];
};
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}

// A unit's two pieces: eight values at `lo` and at `hi` of its head, and its first pair (-1: values to copy).
struct Unit {
  int lo, hi, pair;
};
template <bool ADJ>
__device__ __forceinline__ Unit unit_of(int u, int rot, bool rotated) {
  if (!rotated || 16 * u >= rot) return {16 * u, 16 * u + 8, -1};
  return ADJ ? Unit{16 * u, 16 * u + 8, 8 * u} : Unit{8 * u, rot / 2 + 8 * u, 8 * u};
}

// TOK tokens a block; blockIdx.y: its part of their units
template <typename Tin, int TOK, bool ADJ>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(const RopeArgs p) {
  __shared__ float cs[TOK][64], sn[TOK][64];
  __shared__ int slots[TOK];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;
  const int per_head = p.d / 16, heads = p.H + 2 * p.Hkv, units = per_head * heads;
  const int part = (units * TOK + gridDim.y - 1) / gridDim.y;  // units of this block
  const int first = blockIdx.y * part, last = min(first + part, units * TOK);

  Values v[kAhead];
  // Every thread passes the barrier below, so the loads before it need no more than their own bounds.
  auto fetch = [&](int at, Values& x) {
    const int tok = at / units, r = at - tok * units, head = r / per_head, u = r - head * per_head;
    const int64_t t = t0 + tok;
    if (at >= last || t >= p.T) return;
    const Unit w = unit_of<ADJ>(u, p.rot, head < p.H + p.Hkv);
    const Tin* src = head < p.H ? static_cast<const Tin*>(p.q) + t * p.q_stride + (int64_t)head * p.d
                     : head < p.H + p.Hkv ? static_cast<const Tin*>(p.k) + t * p.k_stride + (int64_t)(head - p.H) * p.d
                                          : static_cast<const Tin*>(p.v) + t * p.v_stride + (int64_t)(head - p.H - p.Hkv) * p.d;
    load8(src + w.lo, x.x);
    load8(src + w.hi, x.x + 8);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(first + tid + i * kThreads, v[i]);

  const int pairs = p.rot / 2;
  if (tid < TOK) {
    const int64_t t = t0 + tid;
    int s = t < p.T ? p.slot_map[t] : -1;
    if (s < -1 || (int64_t)s >= (int64_t)p.num_blocks << p.shift) {
      atomicOr(p.err, KDA_DEVERR_BAD_SLOT);
      s = -1;
    }
    slots[tid] = s;
  }
  __syncthreads();
  for (int i = tid; i < TOK * pairs; i += kThreads) {
    const int tok = i / pairs, j = i - tok * pairs;
    const int64_t t = t0 + tok;
    if (t >= p.T) break;
    const int a = p.axis ? p.axis[j] : 0;
    if ((unsigned)a >= (unsigned)p.axes) {
      atomicOr(p.err, KDA_DEVERR_BAD_SLOT);
      slots[tok] = -1;
      continue;
    }
    // whole turns of the frequency itself do not matter
    double turns = p.inv_freq[j] * 0.15915494309189535;
    turns -= floor(turns);
    const uint64_t F = turns < 1.0 ? (uint64_t)(turns * 18446744073709551616.0) : 0;
    const uint64_t x = (uint64_t)(int64_t)p.positions[(int64_t)a * p.T + t] * F;
    const float half_turns = (float)(int32_t)(x >> 32) * 0x1p-31f;
    sincospif(half_turns, &sn[tok][j], &cs[tok][j]);
  }
  __syncthreads();

  for (int base = first + tid; base < last; base += kAhead * kThreads) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int at = base + i * kThreads;
      if (at >= last) break;
      const int tok = at / units, r = at - tok * units, head = r / per_head, u = r - head * per_head;
      const int slot = slots[tok];
      if (slot < 0) continue;
      const bool rotated = head < p.H + p.Hkv;
      const Unit w = unit_of<ADJ>(u, p.rot, rotated);
      float* x = v[i].x;
      if (w.pair >= 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float c = cs[tok][w.pair + j], s = sn[tok][w.pair + j];
          float &a = x[ADJ ? 2 * j : j], &b = x[ADJ ? 2 * j + 1 : 8 + j];
          const float y = fmaf(a, c, -b * s);
          b = fmaf(b, c, a * s);
          a = y;
        }
      }
      const int64_t place = (int64_t)(slot >> p.shift) * p.block_stride + (int64_t)(slot & ((1 << p.shift) - 1)) * p.token_stride;
      __nv_bfloat16* dst = head < p.H ? static_cast<__nv_bfloat16*>(p.q_out) + ((t0 + tok) * p.H + head) * p.d
                           : rotated ? static_cast<__nv_bfloat16*>(p.k_cache) + place + (head - p.H) * p.head_stride
                                     : static_cast<__nv_bfloat16*>(p.v_cache) + place + (head - p.H - p.Hkv) * p.head_stride;
      store8(dst + w.lo, x);
      store8(dst + w.hi, x + 8);
    }
    if (base + kAhead * kThreads < last) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) fetch(base + (kAhead + i) * kThreads, v[i]);
    }
  }
}

template <typename Tin, int TOK, bool ADJ>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
  const int units = a.d / 16 * (a.H + 2 * a.Hkv);
  const int64_t blocks = (a.T + TOK - 1) / TOK;
  const unsigned parts = TOK == 1 ? (unsigned)((units + kThreads - 1) / kThreads) : 1;
  rope_append_kernel<Tin, TOK, ADJ><<<dim3((unsigned)blocks, parts), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// One token a block while that leaves SMs idle.
constexpr int kFewTokens = 1024;
template <typename Tin, bool ADJ>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
  return a.T <= kFewTokens ? launch<Tin, 1, ADJ>(a, st) : launch<Tin, 4, ADJ>(a, st);
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs& a, cudaStream_t st) {
  TraceScope ts("kda_rope_append", st);
  if (a.bf16) return a.adjacent ? launch<__nv_bfloat16, true>(a, st) : launch<__nv_bfloat16, false>(a, st);
  return a.adjacent ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace kda
