// Rotary positions with one or several axes, fused with the write of keys and values to a paged cache.
//
//   angle = pos f,  (a, b) -> (a cos - b sin, b cos + a sin)  for each pair of a head's first rot values
//
// A position times a frequency has more whole turns than fp32 can hold fractions of, so the angle is taken in
// fixed point: F = f / (2 pi) 2^64 modulo 2^64 once for each pair, and pos F modulo 2^64, which wraps at whole turns by
// itself.  Its top 32 bits, as a signed fraction of a turn, are rounded to fp32 and go to sincospi.  The angle is then off by
// 2^-26 of a turn for that rounding, 2^-32 for the bits below and (|f| + 1) |pos| 2^-64 for F's: less than 2^-25 in all
// for frequencies up to 64 and every 32-bit position.
//
// A warp has a token (for few tokens a part of its heads), each lane a unit of 16 values of a head (two pieces of 16
// bytes in bf16): eight pairs, or 16 values to copy, the same ones in every head.  A lane makes the cosines and sines of
// two pairs, gets those of its own eight from other lanes, and goes through the heads with them in registers; loads of
// four heads are under way before it needs them, and no warp waits for another.  A lane's two frequencies are turned
// into fixed point once, as a warp walks over tokens.
//
// Bound by HBM for many tokens: every value read once and written once.  Measured on GB300: 16384 tokens of 32 + 2 x 8
// heads of 128 in bf16, three axes: 65 us, 6.2 TB/s (91 % of the measured copy; by blocks of four tokens with the cosines in
// shared memory: 102 us); one token 4.3 us, 1237 fp32 tokens of 12 + 2 x 4 heads of 64: 5.1 us (latency).
#include "kda_device.cuh"
#include "kda_internal.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// 16 values of a lane, as they come
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const __nv_bfloat16* a, const __nv_bfloat16* b) {
    lo = __ldcs(reinterpret_cast<const uint4*>(a));
    hi = __ldcs(reinterpret_cast<const uint4*>(b));
  }
  __device__ __forceinline__ void wide(float (&x)[16]) const {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Piece<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* a, const float* b) {
    v[0] = __ldcs(reinterpret_cast<const float4*>(a));
    v[1] = __ldcs(reinterpret_cast<const float4*>(a) + 1);
    v[2] = __ldcs(reinterpret_cast<const float4*>(b));
    v[3] = __ldcs(reinterpret_cast<const float4*>(b) + 1);
  }
  __device__ __forceinline__ void wide(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[4 * i] = v[i].x;
      x[4 * i + 1] = v[i].y;
      x[4 * i + 2] = v[i].z;
      x[4 * i + 3] = v[i].w;
    }
  }
};
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
// f / (2 pi) in 64-bit fixed point, without its whole turns: f = m 2^(e - 1075) with a 53-bit m, and m times
// floor(2^64 / (2 pi)), shifted.  In integers, because FP64 arithmetic is slow here (2 us of a token's 8).
__device__ __forceinline__ uint64_t turns_of(double f) {
  constexpr uint64_t kPerRadian = 0x28be60db9391054aull;
  const uint64_t w = (uint64_t)__double_as_longlong(f), m = (w & 0xfffffffffffffull) | 0x10000000000000ull;
  const int shift = 1075 - (int)(w >> 52 & 2047);
  const uint64_t hi = __umul64hi(m, kPerRadian), lo = m * kPerRadian;
  uint64_t turns;
  if (shift >= 128) turns = 0;
  else if (shift >= 64) turns = hi >> (shift - 64);
  else if (shift > 0) turns = hi << (64 - shift) | lo >> shift;
  else turns = shift > -64 ? lo << -shift : 0;
  return (int64_t)w < 0 ? 0 - turns : turns;
}

template <typename Tin, bool ADJ>
__global__ void __launch_bounds__(kThreads)
rope_append_kernel(const RopeArgs p, const int parts) {
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  constexpr int kAhead = sizeof(Tin) == 2 ? 4 : 2;  // heads a lane has under way: 128 bytes
  const int lane = threadIdx.x & 31;
  const int per_head = p.d / 16, at_once = 32 / per_head;  // lanes of a head, heads of a warp
  const int u = lane % per_head, head0 = lane / per_head;
  const int heads = p.H + 2 * p.Hkv, pairs = p.rot / 2;
  // the lane's two pieces of a head, and its first pair
  const bool turned = 16 * u < p.rot;
  const int lo = turned && !ADJ ? 8 * u : 16 * u, hi = turned && !ADJ ? pairs + 8 * u : 16 * u + 8;
  const int from = turned ? 4 * u : 0;  // the lane with the first two of its pairs, 8 u and 8 u + 1

  double freq[2] = {0.0, 0.0};
  int axis[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int j = 2 * lane + i;
    if (j >= pairs) continue;
    freq[i] = p.inv_freq[j];
    if (p.axis) axis[i] = p.axis[j];
  }
  uint64_t F[2];
  bool begun = false;
  // this warp's heads: rounds of at_once
  const int rounds = (heads + at_once - 1) / at_once, each = (rounds + parts - 1) / parts;
  const int64_t warp = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5), warps = (int64_t)gridDim.x * kWarps;
  for (int64_t w = warp; w < p.T * parts; w += warps) {
    const int64_t t = parts == 1 ? w : w / parts;
    const int first = parts == 1 ? 0 : (int)(w - t * parts) * each, end = min(first + each, rounds);
    const int slot = p.slot_map[t];
    const Tin* q = static_cast<const Tin*>(p.q) + t * p.q_stride;
    const Tin* k = static_cast<const Tin*>(p.k) + t * p.k_stride - (int64_t)p.H * p.d;
    const Tin* v = static_cast<const Tin*>(p.v) + t * p.v_stride - (int64_t)(p.H + p.Hkv) * p.d;
    Piece<Tin> got[kAhead];
    auto fetch = [&](int round, Piece<Tin>& x) {
      const int head = round * at_once + head0;
      if (round >= end || head >= heads) return;
      const Tin* src = (head < p.H ? q : head < p.H + p.Hkv ? k : v) + (int64_t)head * p.d;
      x.load(src + lo, src + hi);
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(first + i, got[i]);

    if (!begun) {  // (here, so that the first loads are all under way at once)
      begun = true;
      if (__any_sync(0xffffffffu, (unsigned)axis[0] >= (unsigned)p.axes || (unsigned)axis[1] >= (unsigned)p.axes)) {
        if (lane == 0) atomicOr(p.err, KDA_DEVERR_BAD_SLOT);
        return;
      }
      F[0] = turns_of(freq[0]);
      F[1] = turns_of(freq[1]);
    }
    float c[2], s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t x = (uint64_t)(int64_t)p.positions[(int64_t)axis[i] * p.T + t] * F[i];
      sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &s[i], &c[i]);
    }
    if (slot < 0 || slot >= p.num_blocks << p.shift) {
      if (slot != -1 && lane == 0) atomicOr(p.err, KDA_DEVERR_BAD_SLOT);
      continue;
    }
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, c[i & 1], from + i / 2);
      sn[i] = __shfl_sync(0xffffffffu, s[i & 1], from + i / 2);
      if (!turned) {
        cs[i] = 1.f;
        sn[i] = 0.f;
      }
    }
    __nv_bfloat16* q_out = static_cast<__nv_bfloat16*>(p.q_out) + t * p.H * p.d;
    const int64_t place = (int64_t)(slot >> p.shift) * p.block_stride + (int64_t)(slot & ((1 << p.shift) - 1)) * p.token_stride;
    __nv_bfloat16* k_to = static_cast<__nv_bfloat16*>(p.k_cache) + place;
    __nv_bfloat16* v_to = static_cast<__nv_bfloat16*>(p.v_cache) + place;
    for (int round = first; round < end; round += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int head = (round + i) * at_once + head0;
        if (round + i >= end || head >= heads) break;
        float x[16];
        got[i].wide(x);
        fetch(round + i + kAhead, got[i]);
        const bool rotated = head < p.H + p.Hkv;
        if (rotated && turned) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float &a = x[ADJ ? 2 * j : j], &b = x[ADJ ? 2 * j + 1 : 8 + j];
            const float y = fmaf(a, cs[j], -b * sn[j]);
            b = fmaf(b, cs[j], a * sn[j]);
            a = y;
          }
        }
        __nv_bfloat16* dst = head < p.H ? q_out + head * p.d
                             : rotated ? k_to + (head - p.H) * p.head_stride
                                       : v_to + (head - p.H - p.Hkv) * p.head_stride;
        store8(dst + lo, x);
        store8(dst + hi, x + 8);
      }
    }
  }
}

// Few tokens: the heads of one over four warps (256 tokens: 6.3 us against 8.4; 2048: 16.4 against 12.5).  Many: kBlocks
// blocks an SM walk over them (2 to 8: 68 to 70 us of 16384 tokens).
constexpr int kBlocks = 4, kFewTokens = 512;
template <typename Tin, bool ADJ>
cudaError_t launch(const RopeArgs& a, cudaStream_t st) {
  const int sms = device_sms();
  if (sms <= 0) return cudaErrorInvalidDevice;
  const int parts = a.T <= kFewTokens ? 4 : 1;
  const int64_t blocks = (a.T * parts + kWarps - 1) / kWarps, most = (int64_t)sms * kBlocks;
  return launch_overlapped(rope_append_kernel<Tin, ADJ>, (unsigned)(blocks < most ? blocks : most), kThreads, 0, 1, st, a, parts);
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs& a, cudaStream_t st) {
  TraceScope ts("kda_rope_append", st);
  if (a.bf16) return a.adjacent ? launch<__nv_bfloat16, true>(a, st) : launch<__nv_bfloat16, false>(a, st);
  return a.adjacent ? launch<float, true>(a, st) : launch<float, false>(a, st);
}

}  // namespace kda
