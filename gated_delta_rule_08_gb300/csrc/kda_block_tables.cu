// Block tables, slots and positions of a step from the tokens that each request gains or loses.
//
// With held = ceil(length / block) and after = ceil((length + count) / block), request n takes the blocks
// held .. after - 1 of its row from the free ring, or gives after .. held - 1 back to it.  Where in the ring, and
// where in the packed batch, follows from three running sums over the requests (tokens, blocks taken, blocks given).
//
// One cluster does a step: every CTA forms the sums of all requests in its shared memory, which costs less than
// handing them over, then the new tokens and the blocks given back are spread over all threads, each looking its
// request up by bisection.  A token that starts a new block writes it to the table.  The cluster's barrier lies
// between the last read of lengths and state and their replacement, so a call may update both in place.  No CTA
// reads what another writes: a new token takes its block from the ring if it is a new one, and the ring's places
// read and written are different ones.
//
// Bound by latency (launch, the loads of counts and lengths, the running sums, then ring and table).  Measured on GB300:
// 256 requests of one token 6.3 us, 1000 requests with 39494 tokens in all 10.3 us (a cluster of 8: 12.5).
#include "kda_device.cuh"
#include "kda_internal.h"
#include "tc_ptx.cuh"

namespace kda {
namespace {

constexpr int kThreads = 1024, kFewThreads = 256;  // (a CTA of fewer warps starts sooner)
constexpr int kCluster = 16;
constexpr int kPerCta = 4096;  // tokens that one CTA handles before the others are worth their start

struct Sums {
  int64_t tokens;
  uint32_t taken, given;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.tokens + b.tokens, a.taken + b.taken, a.given + b.given};
}
__device__ __forceinline__ Sums shfl_up(const Sums& a, int o) {
  return {__shfl_up_sync(0xffffffffu, (long long)a.tokens, o), __shfl_up_sync(0xffffffffu, a.taken, o),
          __shfl_up_sync(0xffffffffu, a.given, o)};
}

// the last n in [0, N) with at[n] <= x
__device__ __forceinline__ int find(const int32_t* at, int N, int x) {
  int lo = 0, hi = N - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

__global__ void __launch_bounds__(kThreads)
block_tables_kernel(const BlockTablesArgs p) {
  extern __shared__ int32_t sm[];
  __shared__ Sums warp_sums[32];
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  const int N = p.N, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* first = sm;              // first new token of each request
  int32_t* taken = first + N + 1;   // blocks taken by the requests before
  int32_t* given = taken + N + 1;
  int32_t* length = given + N + 1;
  const int head = p.free_state[0], free = p.free_state[1];
  const int64_t row = (int64_t)p.max_blocks << p.shift, most = row < 0x7fffffff ? row : 0x7fffffff;  // tokens of a request
  const int round = (1 << p.shift) - 1;

  Sums sum{0, 0, 0};  // of the requests before this round's
  bool bad = head < 0 || head >= p.num_blocks || free < 0 || free > p.num_blocks;
  for (int base = 0; base < N; base += (int)blockDim.x) {
    const int n = base + tid;
    Sums own{0, 0, 0};
    if (n < N) {
      const int64_t len = p.lengths[n], count = p.counts[n], now = len + count;
      length[n] = (int)len;
      if (len < 0 || len > most || now < 0 || now > most) {
        bad = true;
      } else {
        const int held = (int)((len + round) >> p.shift), after = (int)((now + round) >> p.shift);
        own = {count > 0 ? count : 0, (uint32_t)(after > held ? after - held : 0), (uint32_t)(held > after ? held - after : 0)};
      }
    }
    Sums scan = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums up = shfl_up(scan, o);
      if (lane >= o) scan = scan + up;
    }
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    if (warp == 0) {  // the warps' sums likewise
      Sums s = lane < (int)blockDim.x / 32 ? warp_sums[lane] : Sums{0, 0, 0};
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Sums up = shfl_up(s, o);
        if (lane >= o) s = s + up;
      }
      warp_sums[lane] = s;
    }
    __syncthreads();
    const Sums before = warp == 0 ? sum : sum + warp_sums[warp - 1];
    sum = sum + warp_sums[31];
    if (base + (int)blockDim.x < N) __syncthreads();
    if (n < N) {  // tokens past 2^31 - 1 have no use: the step does nothing then
      first[n] = (int)(before.tokens + scan.tokens - own.tokens);
      taken[n] = (int)(before.taken + scan.taken - own.taken);
      given[n] = (int)(before.given + scan.given - own.given);
    }
  }
  bad = __syncthreads_or(bad) || sum.tokens > p.T || (int64_t)free + sum.given > p.num_blocks;
  const bool few = !bad && sum.taken > (uint32_t)free;
  const int total = bad || few ? 0 : (int)sum.tokens;
  const int cta = blockIdx.x, ctas = gridDim.x, threads = blockDim.x;
  bool bad_block = false;

  // slots and positions, four tokens a thread
  for (int64_t t0 = ((int64_t)cta * threads + tid) * 4; t0 < p.T; t0 += (int64_t)ctas * threads * 4) {
    int slot[4] = {-1, -1, -1, -1}, pos[4] = {0, 0, 0, 0}, block[4];
    int32_t* entry[4] = {};  // where a new block goes
    int n = t0 < total ? find(first, N, (int)t0) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // (all loads before a store, which they could not pass)
      const int t = (int)t0 + i;
      if (t >= total) break;
      while (n + 1 < N && first[n + 1] <= t) ++n;
      const int x = length[n] + (t - first[n]), b = x >> p.shift, held = (length[n] + round) >> p.shift;
      int32_t* mine = p.block_tables + (int64_t)n * p.max_blocks + b;
      int at = head + taken[n] + (b - held);
      at = at >= p.num_blocks ? at - p.num_blocks : at;
      block[i] = *(b >= held ? p.free_ring + at : mine);
      if (b >= held && (x & round) == 0) entry[i] = mine;
      pos[i] = x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((int)t0 + i >= total) break;
      if (entry[i]) *entry[i] = block[i];
      if ((unsigned)block[i] < (unsigned)p.num_blocks) slot[i] = (block[i] << p.shift) + (pos[i] & round);
      else bad_block = true;
    }
    if (t0 + 3 < p.T) {
      *reinterpret_cast<int4*>(p.slot_map + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int i = 0; t0 + i < p.T; ++i) {
        p.slot_map[t0 + i] = slot[i];
        p.positions[t0 + i] = pos[i];
      }
    }
  }
  // blocks given back, behind those that are free
  if (!bad && !few) {
    for (int r = cta * threads + tid; r < (int)sum.given; r += ctas * threads) {
      const int n = find(given, N, r);
      // (the length after the step: the row keeps its first blocks)
      const int after = (int)(((int64_t)length[n] + p.counts[n] + round) >> p.shift);
      const int block = p.block_tables[(int64_t)n * p.max_blocks + after + (r - given[n])];
      bad_block |= (unsigned)block >= (unsigned)p.num_blocks;
      int64_t at = (int64_t)head + free + r;
      if (at >= p.num_blocks) at -= p.num_blocks;
      p.free_ring[at] = block;
    }
  }
  if (bad_block) atomicOr(p.err, KDA_DEVERR_BAD_SLOT);

  if (ctas > 1) cluster_sync(); else __syncthreads();
  for (int n = cta * threads + tid; n <= N; n += ctas * threads) {
    p.cu_seqlens[n] = total == 0 ? 0 : n < N ? first[n] : total;
    if (n < N) p.new_lengths[n] = bad || few ? length[n] : length[n] + p.counts[n];
  }
  if (cta == 0 && tid == 0) {
    int64_t next = (int64_t)head + sum.taken;
    if (next >= p.num_blocks) next -= p.num_blocks;
    p.new_free_state[0] = bad || few ? head : (int)next;
    p.new_free_state[1] = bad || few ? free : (int)(free + sum.given - sum.taken);
    if (bad) atomicOr(p.err, KDA_DEVERR_BAD_COUNT);
    if (few) atomicOr(p.err, KDA_DEVERR_NO_BLOCKS);
  }
}

constexpr size_t smem_bytes(int N) { return (4 * (size_t)N + 3) * sizeof(int32_t); }

}  // namespace

cudaError_t block_tables_launch(const BlockTablesArgs& a, cudaStream_t st) {
  static DeviceOnce once;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  cudaError_t e = once.run(dev, [] {
    const cudaError_t f = cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)smem_bytes(kMaxTableRequests));
    return f == cudaSuccess ? cudaFuncSetAttribute(block_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) : f;
  });
  if (e != cudaSuccess) return e;
  TraceScope ts("kda_block_tables", st);
  const unsigned ctas = a.T <= kPerCta ? 1 : kCluster;
  const unsigned threads = a.N <= kFewThreads && a.T <= 8 * kFewThreads ? kFewThreads : kThreads;
  return launch_overlapped(block_tables_kernel, ctas, threads, smem_bytes(a.N), ctas, st, a);
}

}  // namespace kda
