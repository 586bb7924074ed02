// Linear attention with one decay per head over whole sequences, on the tcgen05 tensor cores (bf16 inputs).
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
//
// In chunks of 64 tokens, with S the state before the chunk and G_i the running sum of its log decays:
//   o_i = scale ( e^{G_i} S^T q_i + sum_{j <= i} A_ij v_j ),   A_ij = e^{G_i - G_j} q_i . k_j
//   S'  = e^{G_64} S + U,   U = sum_j w_j k_j v_j^T,           w_j = e^{G_64 - G_j}
// A and U need nothing of the state, so the tensor cores work on them ahead of the serial part, which is
// one fused multiply-add per state element.
//
// A CTA walks over the chunks of one (sequence, head) or of a segment of it.  Everything is laid out with
// the value channel as the tensor core's row (M = 128; with dv = 64 the upper rows are not used):
//   D_A [128 x 64]  = [Q ; K] K^T     rows 0-63 are q_i . k_j (the stack fills the 128 rows an MMA has)
//   D_U [dv x dk]   = V~^T K          V~ = w_j v_j as the exact sum of three bf16 parts, so U has fp32 accuracy;
//                                     V~^T lies in TMEM, which keeps it off the shared memory that bounds the chunk
//   D_2 [dv x 64]   = V^T A^T         A masked, decayed, scaled and rounded to bf16 in shared memory
//   D_1 [dv x 64]   = S^T Q^T         S^T rounded to bf16 in TMEM
// with S^T itself (fp32) in the registers of warps 0-7.  So out is off by the roundings of A and S to
// bf16 (half a step each, of its terms), like its own rounding; the states are not rounded below fp32.
//
// Decays: sums are kept in log2.  A token whose decay is below 2^-150 (g = -inf among them) empties the
// state: sums start again at 0 after it, and pairs with such a token between them are masked, so that no
// infinity meets another and a long sum loses no precision.
//
// Warps: 0 copies and decays, 1, 28 and 29 A, 4-11 state, 12-19 output, 20-27 V~ (two per TMEM lane quadrant each;
// in MODE 1 the output warps make V~ too), 30 the MMAs that do not need the state (D_A, D_U), 31 those that end in
// the output (D_1, D_2).  A lies twice, so that the next chunk's is made while one is multiplied.
//
// Few long sequences would leave most of the device idle, so they are cut into segments: MODE 1 runs
// compute every segment's own contribution U_seg to the state after it (no read-out), a merge kernel
// folds them in order, and MODE 0 runs every segment from its state.
//
// Measured, bf16, H = 32, d = 128: 1 x 8192 tokens 127 us (segments 54, merge 8, last pass 78, which overlap; of 272 MB,
// 2.1 TB/s), 8 sequences of 512 to 8192 tokens 246 us (3.3 TB/s), where the longest's 128 chunks of 2 us follow one another.
// Bound by the instructions and the shared-memory traffic of a chunk, not by HBM: 32 MMAs at one in 120-150 clocks,
// four schedulers at half their issue rate, two state products whose operands change between TMEM, registers
// and shared memory.
#include "kda_internal.h"
#include "kda_tc_common.cuh"
#include "kda_tma.h"

namespace kda {
namespace {

using namespace tcx;

constexpr int kC = 64;                      // tokens of a chunk
constexpr int kThreads = 1024;
constexpr int kCopyWarp = 0, kMmaWarp = 30, kMmaOutWarp = 31, kStateWarp = 4, kStateWarps = 8, kOutWarp = 12, kOutWarps = 8,
              kValueWarp = 20, kValueWarps = 8, kMaskWarps = 3;
__device__ __forceinline__ bool is_mask_warp(int w) { return w == 1 || w == 28 || w == 29; }  // lanes 0-63 of TMEM
// Registers: the state warps hold 64 state values a thread; the other groups of four give them theirs.
constexpr int kStateRegs = 112, kOtherRegs = 48;
static_assert(kStateWarps * 32 * kStateRegs + 24 * 32 * kOtherRegs <= kThreads * 64, "registers of the launch");
constexpr int kStages = 4;
// a stage: [Q | K] of the first 64 channels, [Q | K] of the second, V of the first 64 channels, of the second
constexpr uint32_t kBlk = 8192;             // 64 tokens x 64 channels
constexpr uint32_t kQ = 0, kKey = kBlk, kPair = 2 * kBlk, kV = 4 * kBlk, kStageBytes = 6 * kBlk;
constexpr uint32_t kA = kStages * kStageBytes;           // A [64 i][64 j], twice
constexpr uint32_t kOut = kA + 2 * kBlk, kOutBytes = 1024;  // output rows of each output warp's 32 value channels
constexpr int kRing = 8;                                // decays: read until the state has been updated
constexpr uint32_t kDecay = kOut + kOutWarps * kOutBytes;
struct Decay {
  float G[kC];    // log2 of the decay from the chunk's start, or from the last emptying token, to token i
  float E[kC];    // scale e^{G_i} on the state before the chunk; 0 once it has been emptied
  float W[kC];    // w_j; 0 for tokens past the sequence (before: the log decays)
  int first[kC];  // the first token that reaches token i
  float all, low;  // decay of the state over the whole chunk, in two parts (decay_low)
  int pad[2];
};
constexpr uint32_t kBar = kDecay + kRing * sizeof(Decay);
constexpr uint32_t kSmem = kBar + 256 + 1024;
static_assert(kSmem <= 232448, "shared memory of a CTA");

// TMEM columns
constexpr uint32_t kTmA = 0, kTmS = 64, kTm1 = 128, kTm2 = 192, kTmU = 256, kTmV = 384;  // V~^T: three parts of 32

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kEmpty = -150.f;
constexpr float kNoSegment = -1.f;  // no decay: the segment's kernel has given up (a decay is 0 at least, or NaN)

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

struct Maps {
  CUtensorMap q, k, v;
};
struct Params {
  const float* g;
  int g_per_token;
  const float* h0;
  const int32_t* cu;
  void* out;
  float* hT;
  int B;
  int64_t T, T_tot;
  int H, dv;
  float scale;
  unsigned int* err;
  int nseg;
  int seg_len;       // chunks of a segment
  float* seg_state;  // [B H][nseg][dk dv]: MODE 1 writes U_seg, the merge turns it into the state before the segment
  float2* seg_decay;  // [B H][nseg], in two parts; kNoSegment where a segment, and in the last one's place where any, is missing
};

// Sequence of a CTA, in shared memory, by all threads: the longest first, so that no long one starts
// last; their number is small where lengths differ much, and beyond 64 the order is left as it is.
__device__ __forceinline__ int sequence_by_rank(const int32_t* __restrict__ cu, int B, int r, int* slot) {
  if (cu == nullptr || B > 64) return r;
  if (threadIdx.x < B) {
    const int i = threadIdx.x, n = cu[i + 1] - cu[i];
    int rank = 0;
    for (int j = 0; j < B; ++j) {
      const int m = cu[j + 1] - cu[j];
      rank += m > n || (m == n && j < i);
    }
    if (rank == r) *slot = i;
  }
  __syncthreads();
  return *slot;
}

// The decay 2^x, or that of an emptied state, in two parts: equal chunks and segments decay by equal factors.
__device__ __forceinline__ float2 decay_parts(float x, bool emptied) {
  const float e = emptied ? 0.f : exp2f(x);
  return make_float2(e, decay_low(kLn2 * x, e));
}

// Decays of one chunk (one warp, tokens 2 lane and 2 lane + 1).  Returns log2 of the chunk's decay and
// whether a token emptied the state.
__device__ __forceinline__ float chunk_decay(Decay* d, float g0, float g1, int n, float scale, int lane, bool& emptied) {
  const int i0 = 2 * lane, i1 = i0 + 1;
  const bool e0 = g0 <= kEmpty, e1 = g1 <= kEmpty;
  const float a0 = e0 ? 0.f : g0, a1 = e1 ? 0.f : g1;
  // running sum since the last emptying token, and that token's index
  int last = e1 ? i1 : (e0 ? i0 : -1);
  float sum = e1 ? 0.f : a0 + a1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float s = __shfl_up_sync(0xffffffffu, sum, o);
    const int l = __shfl_up_sync(0xffffffffu, last, o);
    if (lane >= o && last < 0) {
      sum += s;
      last = l;
    }
  }
  float before = __shfl_up_sync(0xffffffffu, sum, 1);
  int lastb = __shfl_up_sync(0xffffffffu, last, 1);
  if (lane == 0) {
    before = 0.f;
    lastb = -1;
  }
  const float G0 = e0 ? 0.f : before + a0, G1 = e1 ? 0.f : G0 + a1;
  const int l0 = e0 ? i0 : lastb, l1 = e1 ? i1 : l0;
  // sum of the decays after a token: from the other end, so that the weights near 1 are the exact ones
  float tail = a0 + a1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float s = __shfl_down_sync(0xffffffffu, tail, o);
    if (lane + o < 32) tail += s;
  }
  const float total = __shfl_sync(0xffffffffu, tail, 0);
  float after = __shfl_down_sync(0xffffffffu, tail, 1);
  if (lane == 31) after = 0.f;
  const int final_last = __shfl_sync(0xffffffffu, l1, 31);
  d->G[i0] = G0;
  d->G[i1] = G1;
  d->E[i0] = l0 < 0 ? scale * exp2f(G0) : 0.f;
  d->E[i1] = l1 < 0 ? scale * exp2f(G1) : 0.f;
  d->W[i0] = i0 < n && i0 >= final_last ? exp2f(a1 + after) : 0.f;
  d->W[i1] = i1 < n && i1 >= final_last ? exp2f(after) : 0.f;
  d->first[i0] = l0 < 0 ? 0 : l0;
  d->first[i1] = l1 < 0 ? 0 : l1;
  emptied = final_last >= 0;
  const float2 e = decay_parts(total, emptied);
  if (lane == 0) {
    d->all = e.x;
    d->low = e.y;
  }
  return total;
}

// V~^T = w_j v_j as three bf16 parts (8 bits each: their sum is exact) into TMEM, token pairs packed: TOK tokens of
// 32 value channels (this warp's TMEM lane quadrant) of every chunk.
template <int TOK, int KB, bool GIVEUP>
__device__ __forceinline__ void make_values(uint8_t* sm, const Decay* decay, uint64_t* full, uint64_t* vt_ready, uint64_t* vt_free,
                                            uint64_t* u_full, volatile int* abort_flag, uint32_t tmem, int set, int nc, int rows,
                                            int dv) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tok0 = set * TOK, hf = tok0 / 32;
  const int ch = (warp & 3) * 32 + lane;  // value channel
  const uint32_t tl = tmem_lane(tmem, warp) + kTmV + tok0 / 2;
  // the channel's place in a row: a 16-byte piece, permuted by the row, and two bytes of it
  const uint32_t base = kV + (uint32_t)(ch >> 6) * kBlk + (uint32_t)tok0 * 128u + (uint32_t)(ch & 7) * 2u;
  const uint32_t piece = (uint32_t)((ch & 63) >> 3) << 4;
  const bool live = (warp & 3) * 32 < dv;
  bool ok = true;
#pragma unroll 1
  for (int c = 0; c < nc; ++c) {
    uint8_t* st = sm + (c % kStages) * kStageBytes;
    ok = warp_wait<GIVEUP>(&full[c % kStages], (uint32_t)((c / kStages) & 1), abort_flag);
    // the products that read this half of the chunk before
    if (ok && c > 0) ok = warp_wait<GIVEUP>(hf == 0 ? vt_free : u_full, (uint32_t)((c - 1) & 1), abort_flag);
    if (!ok) break;
    tc_fence_after();
    const int left = rows - c * kC;
    if (left < tok0 + TOK) {
      // rows past the sequence meet weights of 0, but may hold anything: clear them, a quarter of the channels a warp
      for (int i = lane; i < TOK * 4; i += 32) {
        const int r = tok0 + i / 4, j = (warp & 1) * 4 + i % 4, blk = (warp >> 1) & 1;
        if (r < left) continue;
        if (blk < KB) *reinterpret_cast<uint4*>(st + kKey + blk * kPair + row_chunk(r, j)) = make_uint4(0u, 0u, 0u, 0u);
        if (live) *reinterpret_cast<uint4*>(st + kV + blk * kBlk + row_chunk(r, j)) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (live) {
      const float* W = decay[c % kRing].W + tok0;
#pragma unroll 1
      for (int b = 0; b < TOK / 16; ++b) {
        uint32_t p0[8], p1[8], p2[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint8_t* r0 = st + base + (uint32_t)b * 2048u + (uint32_t)(2 * i) * 128u;
          const uint32_t v0 = *reinterpret_cast<const uint16_t*>(r0 + (piece ^ ((2 * i) & 7) << 4));
          const uint32_t v1 = *reinterpret_cast<const uint16_t*>(r0 + 128 + (piece ^ ((2 * i + 1) & 7) << 4));
          const float2 w = *reinterpret_cast<const float2*>(W + 16 * b + 2 * i);
          const float2 x = mul2(w, make_float2(__uint_as_float(v0 << 16), __uint_as_float(v1 << 16)));
          const uint32_t h0 = __float_as_uint(x.x), h1 = __float_as_uint(x.y);
          const float2 y = sub2(x, make_float2(__uint_as_float(h0 & 0xffff0000u), __uint_as_float(h1 & 0xffff0000u)));
          const uint32_t m0 = __float_as_uint(y.x), m1 = __float_as_uint(y.y);
          const float2 z = sub2(y, make_float2(__uint_as_float(m0 & 0xffff0000u), __uint_as_float(m1 & 0xffff0000u)));
          p0[i] = __byte_perm(h0, h1, 0x7632);
          p1[i] = __byte_perm(m0, m1, 0x7632);
          p2[i] = __byte_perm(__float_as_uint(z.x), __float_as_uint(z.y), 0x7632);
        }
        tmem_st8u(tl + 8 * b, p0);
        tmem_st8u(tl + 32 + 8 * b, p1);
        tmem_st8u(tl + 64 + 8 * b, p2);
      }
      tmem_wait_st();
    }
    tc_fence_before();
    warp_arrive(&vt_ready[hf]);
  }
}

// MODE 0: states and outputs.  MODE 1: a segment's contribution to the state after it, and its decay.
template <int DK, int MODE, typename Tout, int WAITS>
__global__ void __launch_bounds__(kThreads, 1)
linear_chunk_kernel(const __grid_constant__ Maps maps, const Params p) {
  constexpr int KB = DK / 64;   // 64-channel blocks of q and k
  constexpr int KC = DK / 2;    // state columns of a thread
  constexpr bool GIVEUP = WAITS == kWaitsGiveUp;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = aligned_smem(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + kBar);  // [stages] tiles landed and decays written
  uint64_t* empty = full + kStages;                         // [stages] the chunk's last products have been seen done
  uint64_t* a_done = empty + kStages;                       // D_A complete
  uint64_t* a_ready = a_done + 1;                           // [2] A written, D_A read
  uint64_t* vt_ready = a_done + 3;                          // [2] half of V~ written (and the rows past the sequence cleared)
  uint64_t* vt_free = a_done + 5;                           // first half of V~ read by its MMAs (the second: u_full)
  uint64_t* u_full = a_done + 6;                            // D_U complete
  uint64_t* u_empty = a_done + 7;                           // D_U read
  uint64_t* s_ready = a_done + 8;                           // S^T in TMEM
  uint64_t* o_full = a_done + 9;                            // [2] D_1 and D_2 complete
  uint64_t* o_read = a_done + 11;                           // D_1 and D_2 read
  uint64_t* bar_fin = a_done + 13;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(a_done + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* seq_slot = reinterpret_cast<int*>(tmem_slot + 2);
  Decay* decay = reinterpret_cast<Decay*>(sm + kDecay);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H = p.H, dv = p.dv;
  // The merge may be scheduled while the segments run, and the last pass while it runs.  Every CTA of a grid
  // waits for the grid before it, so that none completes before the one it follows.
  if (MODE == 1) griddep_launch_dependents();
  if (p.cu != nullptr && !offsets_ok(p.cu, p.B, p.T_tot)) {
    if (tid == 0) atomicOr(p.err, KDA_DEVERR_BAD_SEQLENS);
    griddep_wait();
    return;
  }
  const int seg = blockIdx.x % p.nseg, chain = blockIdx.x / p.nseg;
  const int h = chain % H, b = sequence_by_rank(p.cu, p.B, chain / H, seq_slot);
  // token coordinates fit 32 bits
  const int t_begin = p.cu ? p.cu[b] : b * (int)p.T;
  const int len = p.cu ? p.cu[b + 1] - t_begin : (int)p.T;
  const int nchunks = (int)(((int64_t)len + kC - 1) / kC);
  const int last_seg = nchunks > 0 ? (nchunks - 1) / p.seg_len : 0;
  if (MODE == 0 ? seg > last_seg : seg >= last_seg) {
    griddep_wait();
    return;
  }
  const int c0 = seg * p.seg_len, nc = (nchunks < c0 + p.seg_len ? nchunks : c0 + p.seg_len) - c0;
  const int t0 = t_begin + c0 * kC;  // the segment's first token
  const int rows = len - c0 * kC;    // tokens from there to the sequence's end

  if (warp == 0) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], kStateWarps + (MODE == 0 ? kOutWarps : 0));
    }
    mbar_init(a_done, 1);
    mbar_init(vt_free, 1);
    mbar_init(u_full, 1);
    mbar_init(u_empty, kStateWarps);
    mbar_init(s_ready, kStateWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&a_ready[i], kMaskWarps);
      mbar_init(&vt_ready[i], (MODE == 0 ? kValueWarps : kValueWarps + kOutWarps) / 2);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(o_read, kOutWarps);
    mbar_init(bar_fin, 2);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (MODE == 0 && warp == 2) {  // rows 0-31 of A see no token past 31: that quarter is cleared once
#pragma unroll
    for (int j = 4; j < 8; ++j) {
      *reinterpret_cast<uint4*>(sm + kA + row_chunk(lane, j)) = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>(sm + kA + kBlk + row_chunk(lane, j)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // the segments' states are read below
  int issued = 0;  // stages whose copies have been started

  if (warp >= kStateWarp && warp < kStateWarp + kStateWarps) {
    // ======================== state
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStateRegs));
    const int half = (warp - kStateWarp) >> 2, row = (warp & 3) * 32 + lane;  // value channel
    const uint32_t tl = tmem_lane(tmem, warp);
    const bool live = row < dv;
    float S[KC];
    {
      const float* init = MODE == 1 ? nullptr
                          : p.nseg > 1 ? p.seg_state + (((int64_t)b * H + h) * p.nseg + seg) * DK * dv
                          : p.h0 ? p.h0 + ((int64_t)b * H + h) * DK * dv : nullptr;
      if (init && live) {
        init += (int64_t)KC * half * dv + row;
#pragma unroll
        for (int i = 0; i < KC; ++i) S[i] = init[(int64_t)i * dv];
      } else {
#pragma unroll
        for (int i = 0; i < KC; ++i) S[i] = 0.f;
      }
    }
    bool ok = true;
    if (MODE == 0 && p.nseg > 1 && p.seg_decay[((int64_t)b * H + h) * p.nseg + last_seg].x == kNoSegment) {
      ok = false;  // the states of this (sequence, head) are not there: every role leaves by the abort flag
      *abort_flag = 1;
    }
#pragma unroll 1
    for (int c = 0; c < nc; ++c) {
      if (!ok) break;
      if constexpr (MODE == 0) {
        // the products that read the S^T before this one
        if (c > 0) ok = warp_wait<GIVEUP>(&o_full[(c - 1) & 1], (uint32_t)(((c - 1) / 2) & 1), abort_flag);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < KC / 32; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) w[j] = pack_bf2(S[32 * i + 2 * j], S[32 * i + 2 * j + 1]);
          tmem_st16u(tl + kTmS + (KC / 2) * half + 16 * i, w);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(s_ready);
      }
      ok = warp_wait<GIVEUP>(u_full, (uint32_t)(c & 1), abort_flag);
      if (!ok) break;
      warp_arrive(&empty[c % kStages]);
      tc_fence_after();
      const float all = decay[c % kRing].all, low = decay[c % kRing].low;
#pragma unroll
      for (int i = 0; i < KC / 32; ++i) {
        float u[32];
        tmem_ld32(tl + kTmU + KC * half + 32 * i, u);
        tmem_landed(u);
        if (i == KC / 32 - 1) {
          tc_fence_before();
          warp_arrive(u_empty);
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 before = make_float2(S[32 * i + j], S[32 * i + j + 1]);
          const float2 s = fma2(make_float2(all, all), before, fma2(make_float2(low, low), before, make_float2(u[j], u[j + 1])));
          S[32 * i + j] = s.x;
          S[32 * i + j + 1] = s.y;
        }
      }
    }
    if (ok && live) {
      float* dst = MODE == 1 ? p.seg_state + (((int64_t)b * H + h) * p.nseg + seg) * DK * dv
                   : p.hT && seg == last_seg ? p.hT + ((int64_t)b * H + h) * DK * dv : nullptr;
      if (dst) {
        dst += (int64_t)KC * half * dv + row;
#pragma unroll
        for (int i = 0; i < KC; ++i) dst[(int64_t)i * dv] = S[i];
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kCopyWarp) {
      // ======================== copies and decays
      const int vb = dv / 64;
      const uint32_t bytes = (uint32_t)((MODE == 0 ? 2 * KB : KB) + vb) * kBlk;
      float total = 0.f, lost = 0.f;  // log2 of the segment's decay, with the sum's rounding error
      bool any = false;
      // The decays of the chunks ahead go to where their weights will be: a load takes longer than a chunk.
      constexpr int kAhead = 4;
      auto fetch_g = [&](int c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = c * kC + 2 * lane + i;
          const float* src = p.g + (r < rows && p.g_per_token ? (int64_t)(t0 + r) * H + h : (int64_t)h);
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(&decay[c % kRing].W[2 * lane + i])), "l"(src),
                       "r"(r < rows ? 4 : 0)
                       : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
#pragma unroll 1
      for (int i = 0; i < kAhead && nc > 0; ++i) fetch_g(i);
      bool ok = true;
#pragma unroll 1
      for (; issued < nc; ++issued) {
        const int c = issued, s = c % kStages;
        if (c >= kStages) ok = warp_wait<GIVEUP>(&empty[s], (uint32_t)((c / kStages - 1) & 1), abort_flag);
        if (!ok) break;
        if (lane == 0) {
          uint8_t* st = sm + s * kStageBytes;
          const int y = t0 + c * kC;
          mbar_arrive_expect_tx(&full[s], bytes);
#pragma unroll
          for (int i = 0; i < KB; ++i) {
            if (MODE == 0) tma_load_2d(st + kQ + i * kPair, &maps.q, h * DK + 64 * i, y, &full[s]);
            tma_load_2d(st + kKey + i * kPair, &maps.k, h * DK + 64 * i, y, &full[s]);
          }
          for (int i = 0; i < vb; ++i) tma_load_2d(st + kV + i * kBlk, &maps.v, h * dv + 64 * i, y, &full[s]);
        }
        __syncwarp();
        const int left = rows - c * kC;
        bool emptied;
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        Decay* d = &decay[c % kRing];
        const float g0 = kLog2e * d->W[2 * lane], g1 = kLog2e * d->W[2 * lane + 1];
        const float x = chunk_decay(d, g0, g1, left < kC ? left : kC, p.scale, lane, emptied) + lost;
        const float sum = total + x;
        lost = x - (sum - total);
        total = sum;
        any |= emptied;
        warp_arrive(&full[s]);
        fetch_g(c + kAhead);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (MODE == 1 && lane == 0) p.seg_decay[((int64_t)b * H + h) * p.nseg + seg] = decay_parts(total + lost, any);
    } else if (warp == kMmaWarp) {
      // ======================== D_A and D_U
      {
        const bool leader = lane == 0;
        constexpr uint32_t id_a = idesc_bf16_f32(128, kC, false, false), id_u = idesc_bf16_f32(128, DK, false, true);
        bool ok = true;
        const int n = WAITS == kFirstCtaStalls && blockIdx.x == 0 ? 0 : nc;
#pragma unroll 1
        for (int c = 0; c < n; ++c) {
          const int s = c % kStages;
          const uint8_t* st = sm + s * kStageBytes;
          if constexpr (MODE == 0) {
            ok = warp_spin<GIVEUP>(&full[s], (uint32_t)((c / kStages) & 1), abort_flag);
            if (ok && c > 0) ok = warp_spin<GIVEUP>(&a_ready[(c - 1) & 1], (uint32_t)(((c - 1) / 2) & 1), abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint64_t dq = smem_desc_sw128(smem_u32(st + kQ), 16, 1024), dk = smem_desc_sw128(smem_u32(st + kKey), 16, 1024);
#pragma unroll 1
            for (int b = 0; b < KB; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_bf16_ss_by(leader, tmem + kTmA, desc_add(dq, b * kPair + i * 32), desc_add(dk, b * kPair + i * 32), id_a, b + i > 0);
            mma_commit_by(leader, a_done);
          }
          if (c > 0) ok = warp_spin<GIVEUP>(u_empty, (uint32_t)((c - 1) & 1), abort_flag);
          const uint64_t d_k = smem_desc_sw128(smem_u32(st + kKey), kPair, 1024);
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {  // by halves of 32 tokens
            ok = ok && warp_spin<GIVEUP>(&vt_ready[hf], (uint32_t)(c & 1), abort_flag);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < 3; ++i)
                mma_bf16_ts_by(leader, tmem + kTmU, tmem + kTmV + 32 * i + 16 * hf + 8 * j, desc_add(d_k, hf * 4096 + j * 2048),
                               id_u, hf + i + j > 0);
            mma_commit_by(leader, hf == 0 ? vt_free : u_full);
          }
          if (!ok) break;
        }
      }
    } else if (warp == kMmaOutWarp) {
      // ======================== D_2 and D_1
      if constexpr (MODE == 0) {
        const bool leader = lane == 0;
        constexpr uint32_t id_1 = idesc_bf16_f32(128, kC, false, false), id_2 = idesc_bf16_f32(128, kC, true, false);
        const uint64_t d_a = smem_desc_sw128(smem_u32(sm + kA), 16, 1024);
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
          const uint8_t* st = sm + (c % kStages) * kStageBytes;
          const uint64_t d_v = smem_desc_sw128(smem_u32(st + kV), kBlk, 1024), d_q = smem_desc_sw128(smem_u32(st + kQ), 16, 1024);
          const uint32_t buf = c & 1;
          ok = warp_spin<GIVEUP>(&a_ready[buf], (uint32_t)((c / 2) & 1), abort_flag);
          if (ok && c > 0) ok = warp_spin<GIVEUP>(o_read, (uint32_t)((c - 1) & 1), abort_flag);
          if (ok && c == nc - 1) {
            // rows past the sequence are cleared with V~; the state tells that the chunk before has passed there
            ok = warp_spin<GIVEUP>(s_ready, (uint32_t)(c & 1), abort_flag) &&
                 warp_spin<GIVEUP>(&vt_ready[0], (uint32_t)(c & 1), abort_flag) &&
                 warp_spin<GIVEUP>(&vt_ready[1], (uint32_t)(c & 1), abort_flag);
          }
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < kC / 16; ++j)
            mma_bf16_ss_by(leader, tmem + kTm2, desc_add(d_v, j * 2048), desc_add(d_a, buf * kBlk + j * 32), id_2, j > 0);
          if (c < nc - 1) ok = warp_spin<GIVEUP>(s_ready, (uint32_t)(c & 1), abort_flag);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_bf16_ts_by(leader, tmem + kTm1, tmem + kTmS + 32 * b + 8 * i, desc_add(d_q, b * kPair + i * 32), id_1, b + i > 0);
          mma_commit_by(leader, &o_full[buf]);
        }
      }
    } else if (warp >= kOutWarp && warp < kOutWarp + kOutWarps) {
      // ======================== output: 32 tokens of 32 value channels, by way of shared memory
      if constexpr (MODE == 1) {
        make_values<16, KB, GIVEUP>(sm, decay, full, vt_ready, vt_free, u_full, abort_flag, tmem, 2 + ((warp - kOutWarp) >> 2), nc, rows,
                                dv);
      } else {
        constexpr int kLanes = 32 * sizeof(Tout) / 16;             // lanes that store a token's 16-byte pieces
        const uint32_t tl = tmem_lane(tmem, warp);
        const bool live = (warp & 3) * 32 < dv;
        uint8_t* stage = sm + kOut + (warp - kOutWarp) * kOutBytes;
        // this lane's 16 bytes of the first token it stores
        const int64_t step = (int64_t)H * dv * sizeof(Tout);
        const int tok0 = 32 * ((warp - kOutWarp) >> 2);
        int r0 = tok0 + lane / kLanes;  // ... and that token's place in the segment
        uint8_t* dst = static_cast<uint8_t*>(p.out) + (int64_t)(t0 + r0) * step + ((int64_t)h * dv + (warp & 3) * 32) * sizeof(Tout) +
                       lane % kLanes * 16;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
          ok = warp_wait<GIVEUP>(&o_full[c & 1], (uint32_t)((c / 2) & 1), abort_flag);
          if (!ok) break;
          warp_arrive(&empty[c % kStages]);
          tc_fence_after();
          const float* E = decay[c % kRing].E + tok0;
          const uint32_t ta = tl + tok0;
          if constexpr (sizeof(Tout) == 2) {
            // read and rounded first, so that the next chunk's products can start, then stored
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x[8], y[8];
              tmem_ld8x2_wait(ta + kTm1 + 8 * i, ta + kTm2 + 8 * i, x, y);
#pragma unroll
              for (int j = 0; j < 8; j += 4) {
                const float4 e = *reinterpret_cast<const float4*>(E + 8 * i + j);
                o[4 * i + j / 2] = pack_bf2(fmaf(e.x, x[j], y[j]), fmaf(e.y, x[j + 1], y[j + 1]));
                o[4 * i + j / 2 + 1] = pack_bf2(fmaf(e.z, x[j + 2], y[j + 2]), fmaf(e.w, x[j + 3], y[j + 3]));
              }
            }
            tc_fence_before();
            warp_arrive(o_read);
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // 16 tokens
              uint16_t* at = reinterpret_cast<uint16_t*>(stage) + lane;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                at[(2 * j) * 32] = (uint16_t)o[8 * g + j];
                at[(2 * j + 1) * 32] = (uint16_t)(o[8 * g + j] >> 16);
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (live && r0 < rows) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(stage + i * 512 + lane * 16);
                dst += (32 / kLanes) * step;
                r0 += 32 / kLanes;
              }
              __syncwarp();
            }
          } else {
#pragma unroll 1
            for (int tk = 0; tk < 32; tk += 8) {
              float x[8], y[8];
              tmem_ld8x2_wait(ta + kTm1 + tk, ta + kTm2 + tk, x, y);
              float* at = reinterpret_cast<float*>(stage) + lane;
#pragma unroll
              for (int j = 0; j < 8; ++j) at[j * 32] = fmaf(E[tk + j], x[j], y[j]);
              if (tk == 24) {
                tc_fence_before();
                warp_arrive(o_read);
              }
              __syncwarp();
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (live && r0 < rows) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(stage + i * 512 + lane * 16);
                dst += (32 / kLanes) * step;
                r0 += 32 / kLanes;
              }
              __syncwarp();
            }
          }
          dst += 32 * step;  // the other half's tokens
          r0 += 32;
        }
      }
    } else if (is_mask_warp(warp)) {
      // ======================== A: masked, decayed, to bf16, 32 columns a warp
      if constexpr (MODE == 0) {
        const int i = (warp & 1) * 32 + lane;  // token, TMEM lane
        const uint32_t tl = tmem_lane(tmem, warp & 1);
        const int col = warp == 1 ? 32 : 0;
        const float scale = p.scale;
        bool ok = true;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
          const Decay* d = &decay[c % kRing];
          ok = warp_wait<GIVEUP>(a_done, (uint32_t)(c & 1), abort_flag);
          // the product that read the A that lies here
          if (ok && c >= 2) ok = warp_wait<GIVEUP>(&o_full[c & 1], (uint32_t)((c / 2 - 1) & 1), abort_flag);
          if (!ok) break;
          tc_fence_after();
          uint8_t* at = sm + kA + (c & 1) * kBlk;
          const float Gi = d->G[i];
          const uint32_t first = (uint32_t)d->first[i], span = (uint32_t)i - first;
#pragma unroll 1
          for (int j0 = col; j0 < col + 32; j0 += 8) {
            float x[8];
            tmem_ld8_wait(tl + kTmA + j0, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float e = ex2(Gi - d->G[j0 + j]);
              x[j] = (uint32_t)(j0 + j) - first <= span ? x[j] * (scale * e) : 0.f;
            }
            *reinterpret_cast<uint4*>(at + row_chunk(i, j0 / 8)) =
                make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7]));
          }
          fence_proxy_async_smem();
          tc_fence_before();
          warp_arrive(&a_ready[c & 1]);
        }
      }
    } else if (warp >= kValueWarp && warp < kValueWarp + kValueWarps) {
      // ======================== V~
      make_values<MODE == 0 ? 32 : 16, KB, GIVEUP>(sm, decay, full, vt_ready, vt_free, u_full, abort_flag, tmem,
                                               (warp - kValueWarp) >> 2, nc, rows, dv);
    }
  }
  tc_fence_before();
  __syncthreads();
  drain_after_abort<kStages>(abort_flag, tid == kCopyWarp * 32, tid == kMmaWarp * 32 || tid == kMmaOutWarp * 32, full, issued,
                             bar_fin, p.err);
  // (by the thread that wrote the decay)
  if (MODE == 1 && tid == kCopyWarp * 32 && *abort_flag) p.seg_decay[((int64_t)b * H + h) * p.nseg + seg].x = kNoSegment;
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Folds the segments of a (sequence, head) in order: seg_state[i] becomes the state before segment i.
// One thread per four state values; fp32 throughout.
constexpr int kMergeThreads = 128;
__global__ void __launch_bounds__(kMergeThreads)
linear_merge_kernel(const float* __restrict__ h0, const int32_t* __restrict__ cu, float* __restrict__ seg_state,
                    float2* __restrict__ seg_decay, int B, int64_t T, int64_t T_tot, int H, int nseg, int seg_len,
                    int elems, int parts) {
  griddep_launch_dependents();
  const bool ok = cu == nullptr || offsets_ok(cu, B, T_tot);
  griddep_wait();
  if (!ok) return;
  const int bh = blockIdx.x / parts, b = bh / H;
  const int at = (blockIdx.x % parts * kMergeThreads + threadIdx.x) * 4;
  const int64_t len = cu ? (int64_t)cu[b + 1] - cu[b] : T;
  const int nchunks = (int)((len + kC - 1) / kC), last = nchunks > 0 ? (nchunks - 1) / seg_len : 0;
  float4 S = h0 ? *reinterpret_cast<const float4*>(h0 + (int64_t)bh * elems + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  float* p = seg_state + (int64_t)bh * nseg * elems + at;
  float2* e = seg_decay + (int64_t)bh * nseg;
  bool missing = false;
  constexpr int kAhead = 4;  // loads under way at a time
  for (int i0 = 0; i0 < last; i0 += kAhead, p += (int64_t)kAhead * elems) {
    float4 u[kAhead];
    float2 d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool in = i0 + i < last;
      u[i] = in ? *reinterpret_cast<const float4*>(p + (int64_t)i * elems) : make_float4(0.f, 0.f, 0.f, 0.f);
      d[i] = in ? e[i0 + i] : make_float2(0.f, 0.f);
      missing |= d[i].x == kNoSegment;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < last) {
        *reinterpret_cast<float4*>(p + (int64_t)i * elems) = S;
        S = f4_fma(d[i].x, S, f4_fma(d[i].y, S, u[i]));
      }
  }
  *reinterpret_cast<float4*>(seg_state + ((int64_t)bh * nseg + last) * elems + at) = S;
  if (blockIdx.x % parts == 0 && threadIdx.x == 0) e[last].x = missing ? kNoSegment : 0.f;
}

// Segments, of n chunks at least so long that all of them, with one short one for each (sequence, head), make at most
// one CTA an SM (a second wave would cost as much as the first).  Measured, a pass over L chunks takes 1.9 L + 6 us and
// the three launches of a cut one 3 n + 19 us, so a cut is taken where 3 n + 12 < 2 L.  Uncut against cut, us:
//   1 x 640, H = 32: 25 / 27;  1 x 1024: 36 / 31;  1 x 2048: 65 / 44;  1 x 4096: 127 / 73;  2 x 4096: 126 / 161;
//   1 x 4096, H = 8: 123 / 32.  With d = 64: 20 / 21, 29 / 24, 52 / 34, 99 / 56, 100 / 126 and 99 / 23.
// Lengths given by offsets are on the device, so half of all tokens stands for the longest of several sequences.
constexpr int kMinSegChunks = 4;
void segments(int B, int64_t T, int64_t T_tot, bool has_cu, int H, int sms, int* nseg, int* seg_len) {
  const int64_t longest = (T + kC - 1) / kC;  // of a sequence, at most
  const int64_t chains = (int64_t)B * H, expected = has_cu && B > 1 ? longest / 2 : longest;
  *nseg = 1;
  *seg_len = longest > 0 ? (int)longest : 1;
  if (chains >= sms) return;
  const int64_t chunks = has_cu ? (T_tot + kC - 1) / kC : B * longest;
  int64_t n = (chunks * H + sms - chains - 1) / (sms - chains);
  if (n < kMinSegChunks) n = kMinSegChunks;
  if (3 * n + 12 >= 2 * expected) return;
  *nseg = (int)((longest + n - 1) / n);
  *seg_len = (int)n;
}

struct DeviceState {
  DeviceOnce once;
  int sms[kMaxDevices] = {};
};
DeviceState g_state;

template <int DK, int WAITS>
cudaError_t allow() {
  cudaError_t e = cudaFuncSetAttribute(linear_chunk_kernel<DK, 0, __nv_bfloat16, WAITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(linear_chunk_kernel<DK, 0, float, WAITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(linear_chunk_kernel<DK, 1, float, WAITS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  return e;
}
cudaError_t device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const cudaError_t e = g_state.once.run(dev, [dev] {
    return cudaDeviceGetAttribute(&g_state.sms[dev], cudaDevAttrMultiProcessorCount, dev);
  });
  if (e == cudaSuccess) *sms = g_state.sms[dev];
  return e;
}
cudaError_t allow_all() {
  static DeviceOnce once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  return once.run(dev, [] {
    cudaError_t e = allow<64, kWaits>();
    if (e == cudaSuccess) e = allow<128, kWaits>();
    if (e == cudaSuccess) e = allow<64, kWaitsGiveUp>();
    if (e == cudaSuccess) e = allow<128, kWaitsGiveUp>();
    if (e == cudaSuccess) e = allow<64, kFirstCtaStalls>();
    if (e == cudaSuccess) e = allow<128, kFirstCtaStalls>();
    return e;
  });
}

// A launch that may start while the kernel before it in the stream drains (`early`); the kernel waits for it itself.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, int threads, uint32_t smem, cudaStream_t st, bool early, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

template <int DK, int WAITS>
cudaError_t launch(const LinearArgs& a, const Maps& maps, const Params& p, cudaStream_t st) {
  const unsigned grid = (unsigned)((int64_t)a.B * a.H * p.nseg);
  if (p.nseg > 1) {
    {
      TraceScope ts("kda_linear_segments", st);
      const cudaError_t e = launch_after(linear_chunk_kernel<DK, 1, float, WAITS>, grid, kThreads, kSmem, st, false, maps, p);
      if (e != cudaSuccess) return e;
    }
    const int elems = DK * a.dv, parts = elems / (4 * kMergeThreads);
    TraceScope ts("kda_linear_merge", st);
    const cudaError_t e = launch_after(linear_merge_kernel, (unsigned)(a.B * a.H * parts), kMergeThreads, 0, st, true, a.h0,
                                       a.cu_seqlens, p.seg_state, p.seg_decay, a.B, a.T, a.T_tot, a.H, p.nseg,
                                       p.seg_len, elems, parts);
    if (e != cudaSuccess) return e;
  }
  TraceScope ts("kda_linear_chunk", st);
  auto* kernel = a.out_bf16 ? linear_chunk_kernel<DK, 0, __nv_bfloat16, WAITS> : linear_chunk_kernel<DK, 0, float, WAITS>;
  if (WAITS == kFirstCtaStalls && p.nseg > 1)  // a segment's contribution has stalled: the last pass does not
    kernel = a.out_bf16 ? linear_chunk_kernel<DK, 0, __nv_bfloat16, kWaits> : linear_chunk_kernel<DK, 0, float, kWaits>;
  return launch_after(kernel, grid, kThreads, kSmem, st, p.nseg > 1, maps, p);
}

}  // namespace

size_t linear_tc_workspace(int B, int64_t T, int H, int dk, int dv) {
  int sms = 0;
  if (device_sms(&sms) != cudaSuccess) return 0;
  size_t most = 0;  // with and without offsets (T is then one sequence's length)
  for (int has_cu = 0; has_cu < 2; ++has_cu) {
    if (!has_cu && B * T > kMaxTokens) continue;  // not a call without offsets
    int nseg, seg_len;
    segments(B, T, has_cu ? T : (int64_t)B * T, has_cu != 0, H, sms, &nseg, &seg_len);
    const size_t n = nseg > 1 ? (size_t)B * H * nseg * ((size_t)dk * dv + 2) * sizeof(float) : 0;
    if (n > most) most = n;
  }
  return align_up(most, 256);
}

cudaError_t linear_tc_launch(const LinearArgs& a, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e == cudaSuccess) e = allow_all();
  if (e != cudaSuccess) return e;
  Params p{};
  p.g = a.g; p.g_per_token = a.g_per_token; p.h0 = a.h0; p.cu = a.cu_seqlens; p.out = a.out; p.hT = a.hT;
  p.B = a.B; p.T = a.T; p.T_tot = a.T_tot; p.H = a.H; p.dv = a.dv; p.scale = a.scale; p.err = a.err;
  segments(a.B, a.T, a.T_tot, a.cu_seqlens != nullptr, a.H, sms, &p.nseg, &p.seg_len);
  p.seg_state = static_cast<float*>(a.workspace);
  p.seg_decay = reinterpret_cast<float2*>(p.seg_state + (size_t)a.B * a.H * p.nseg * a.dk * a.dv);
  Maps maps{};
  if (a.T_tot > 0 &&
      (!tensor_map_2d(&maps.q, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.T_tot, (uint64_t)a.H * a.dk, a.q_stride * 2, kC, 64) ||
       !tensor_map_2d(&maps.k, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.T_tot, (uint64_t)a.H * a.dk, a.k_stride * 2, kC, 64) ||
       !tensor_map_2d(&maps.v, a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.T_tot, (uint64_t)a.H * a.dv, a.v_stride * 2, kC, 64)))
    return cudaErrorInvalidValue;
  auto* run = a.dk == 64 ? launch<64, kWaits> : launch<128, kWaits>;
  if (a.waits == kWaitsGiveUp) run = a.dk == 64 ? launch<64, kWaitsGiveUp> : launch<128, kWaitsGiveUp>;
  if (a.waits == kFirstCtaStalls) run = a.dk == 64 ? launch<64, kFirstCtaStalls> : launch<128, kFirstCtaStalls>;
  return run(a, maps, p, st);
}

}  // namespace kda
