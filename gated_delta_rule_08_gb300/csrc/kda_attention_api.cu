// C-ABI entry points of the operators of an attention layer over a paged cache: argument validation and dispatch.
// The public contract is include/kda.h.
#include <cuda_runtime.h>

#include <math.h>

#include "../../include/kda.h"
#include "kda_internal.h"

#define KDA_API extern "C" __attribute__((visibility("default")))

using namespace kda;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// log2 of a supported block size, or -1
int block_shift(int block_size) {
  for (int s = 4; s <= 8; ++s)
    if (block_size == 1 << s) return s;
  return -1;
}

// Distances of blocks, tokens and heads: pieces of 16 bytes, no overlap of what lies next to each other in a block.
bool strides_ok(const int64_t* s, int d) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < d || s[i] >= (int64_t)1 << 36 || s[i] % 8 != 0) return false;
  return true;
}

kda_status ready(unsigned int** err) {
  bool supported = false;
  if (!device_ready(err, &supported)) return KDA_ERR_CUDA;
  return supported ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

bool heads_ok(int H, int Hkv) { return H % Hkv == 0 && H / Hkv <= 128; }

// Rows of a key head and request, in the mean (their numbers are on the device), from which on tiles of 128 rows pay:
// more than one tile of 16, each of which reads the keys again; or more than four where they would leave SMs idle (one
// request of 4000 keys: 48 rows 16.6 us against 31, 64 rows 20.7; 68 rows of the other kernel 24.9).
bool many_rows(const AttentionArgs& a) {
  const int64_t rows = a.T * (a.H / a.Hkv);
  return rows > (int64_t)(a.N * a.Hkv <= 32 ? 64 : 16) * a.N;
}

kda_status attention(AttentionArgs a, int block_size, const int64_t* strides, void* stream) {
  if (a.N < 0 || a.T < 0 || a.H <= 0 || a.Hkv <= 0 || a.num_blocks < 0 || a.max_blocks < 0 || a.window < 0 || a.sinks < 0 ||
      a.max_length < 0 || !(a.scale > 0.f) || isinf(a.scale))
    return KDA_ERR_INVALID_ARG;
  a.shift = block_shift(block_size);
  if (a.shift < 0 || (a.d != 64 && a.d != 128) || !heads_ok(a.H, a.Hkv)) return KDA_ERR_UNSUPPORTED;
  if (a.N > (1 << 20) || a.T > (0x7fffffff - 512) / a.H || (int64_t)a.N * a.H > 0x7fffffff / 64 ||
      (int64_t)a.num_blocks << a.shift > 0x7fffffff || (int64_t)a.N * a.max_blocks > 0x7fffffff)
    return KDA_ERR_UNSUPPORTED;
  if (!strides || !strides_ok(strides, a.d)) return KDA_ERR_INVALID_ARG;
  if (a.q_stride < (int64_t)a.H * a.d || a.q_stride >= (int64_t)1 << 32 || a.q_stride % 8 != 0) return KDA_ERR_INVALID_ARG;
  const bool rows = a.N > 0 && a.T > 0;
  if (rows && (!a.q || !a.k_cache || !a.v_cache || !a.block_tables || !a.lengths || !a.out)) return KDA_ERR_INVALID_ARG;
  if (rows && (a.num_blocks == 0 || a.max_blocks == 0)) return KDA_ERR_INVALID_ARG;
  if (a.out && (a.out == a.q || a.out == a.k_cache || a.out == a.v_cache)) return KDA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.out, 16) ||
      !aligned(a.block_tables, 4) || !aligned(a.lengths, 4) || !aligned(a.cu_seqlens, 4) || !aligned(a.tree_mask, 8))
    return KDA_ERR_INVALID_ARG;
  const kda_status st = ready(&a.err);
  if (st != KDA_OK) return st;
  if (!rows) return KDA_OK;
  const int64_t longest = (int64_t)a.max_blocks << a.shift;
  if (a.max_length == 0 || a.max_length > longest) a.max_length = longest;
  a.block_stride = strides[0]; a.token_stride = strides[1]; a.head_stride = strides[2];
  a.waits = test_wait_timeout();
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return done(many_rows(a) ? attention_tc_launch(a, s) : attention_rows_launch(a, s));
}

}  // namespace

KDA_API kda_status kda_block_tables(const int32_t* counts, const int32_t* lengths, int32_t* block_tables,
                                    int32_t* free_ring, const int32_t* free_state, int32_t* new_lengths,
                                    int32_t* new_free_state, int32_t* slot_map, int32_t* positions, int32_t* cu_seqlens,
                                    int N, int max_blocks, int num_blocks, int block_size, int64_t T, void* stream) {
  if (N < 0 || max_blocks < 0 || num_blocks < 0 || T < 0) return KDA_ERR_INVALID_ARG;
  const int shift = block_shift(block_size);
  if (shift < 0 || N > kMaxTableRequests || T > (1 << 30) || (int64_t)N * max_blocks > 0x7fffffff ||
      (int64_t)num_blocks << shift > 0x7fffffff)
    return KDA_ERR_UNSUPPORTED;
  if (!free_state || !new_free_state || !cu_seqlens) return KDA_ERR_INVALID_ARG;
  if (N > 0 && (!counts || !lengths || !new_lengths)) return KDA_ERR_INVALID_ARG;
  if ((int64_t)N * max_blocks > 0 && !block_tables) return KDA_ERR_INVALID_ARG;
  if ((num_blocks > 0 && !free_ring) || (T > 0 && (!slot_map || !positions))) return KDA_ERR_INVALID_ARG;
  if (counts && (counts == new_lengths || counts == lengths)) return KDA_ERR_INVALID_ARG;
  if (!aligned(counts, 4) || !aligned(lengths, 4) || !aligned(block_tables, 4) || !aligned(free_ring, 4) ||
      !aligned(free_state, 4) || !aligned(new_lengths, 4) || !aligned(new_free_state, 4) || !aligned(slot_map, 16) ||
      !aligned(positions, 16) || !aligned(cu_seqlens, 4))
    return KDA_ERR_INVALID_ARG;
  BlockTablesArgs a{};
  const kda_status st = ready(&a.err);
  if (st != KDA_OK) return st;
  a.counts = counts; a.lengths = lengths; a.block_tables = block_tables; a.free_ring = free_ring; a.free_state = free_state;
  a.new_lengths = new_lengths; a.new_free_state = new_free_state; a.slot_map = slot_map; a.positions = positions;
  a.cu_seqlens = cu_seqlens; a.N = N; a.max_blocks = max_blocks; a.num_blocks = num_blocks; a.shift = shift; a.T = T;
  return done(block_tables_launch(a, static_cast<cudaStream_t>(stream)));
}

KDA_API kda_status kda_rope_append(const void* q, const void* k, const void* v, const double* inv_freq,
                                   const int32_t* axis, const int32_t* positions, const int32_t* slot_map, void* q_out,
                                   void* k_cache, void* v_cache, int64_t T, int H, int Hkv, int d, int rot, int axes,
                                   int interleaved, int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_blocks,
                                   int block_size, const int64_t* cache_strides, kda_dtype dtype, void* stream) {
  if (T < 0 || H <= 0 || Hkv <= 0 || num_blocks < 0 || rot < 0 || axes <= 0) return KDA_ERR_INVALID_ARG;
  const int shift = block_shift(block_size);
  if (shift < 0 || (d != 64 && d != 128) || !heads_ok(H, Hkv) || rot > d || rot % 16 != 0 || axes > 4 ||
      (dtype != KDA_DTYPE_BF16 && dtype != KDA_DTYPE_FP32) || T > 0x7fffffff / H ||
      (int64_t)num_blocks << shift > 0x7fffffff)
    return KDA_ERR_UNSUPPORTED;
  if (!cache_strides || !strides_ok(cache_strides, d)) return KDA_ERR_INVALID_ARG;
  const int piece = dtype == KDA_DTYPE_BF16 ? 8 : 4;
  const int64_t rows[3] = {(int64_t)H * d, (int64_t)Hkv * d, (int64_t)Hkv * d}, strides[3] = {q_stride, k_stride, v_stride};
  for (int i = 0; i < 3; ++i)
    if (strides[i] < rows[i] || strides[i] >= (int64_t)1 << 32 || strides[i] % piece != 0) return KDA_ERR_INVALID_ARG;
  if (T > 0 && (!q || !k || !v || !positions || !slot_map || !q_out || !k_cache || !v_cache || (rot > 0 && !inv_freq)))
    return KDA_ERR_INVALID_ARG;
  if (q_out && (q_out == q || q_out == k || q_out == v || q_out == k_cache || q_out == v_cache)) return KDA_ERR_INVALID_ARG;
  if (k_cache && (k_cache == v_cache || k_cache == q || k_cache == k || k_cache == v)) return KDA_ERR_INVALID_ARG;
  if (v_cache && (v_cache == q || v_cache == k || v_cache == v)) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(inv_freq, 8) || !aligned(axis, 4) || !aligned(positions, 4) || !aligned(slot_map, 4))
    return KDA_ERR_INVALID_ARG;
  RopeArgs a{};
  const kda_status st = ready(&a.err);
  if (st != KDA_OK) return st;
  if (T == 0) return KDA_OK;
  a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride; a.inv_freq = inv_freq;
  a.axis = axis; a.positions = positions; a.slot_map = slot_map; a.q_out = q_out; a.k_cache = k_cache; a.v_cache = v_cache;
  a.block_stride = cache_strides[0]; a.token_stride = cache_strides[1]; a.head_stride = cache_strides[2];
  a.T = T; a.H = H; a.Hkv = Hkv; a.d = d; a.rot = rot; a.axes = axes; a.num_blocks = num_blocks; a.shift = shift;
  a.adjacent = interleaved != 0; a.bf16 = dtype == KDA_DTYPE_BF16;
  return done(rope_append_launch(a, static_cast<cudaStream_t>(stream)));
}

namespace {

AttentionArgs args_of(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      const int32_t* lengths, const int32_t* cu_seqlens, void* out, int N, int64_t T, int H, int Hkv, int d,
                      int64_t q_stride, int num_blocks, int max_blocks, int window, int sinks, int64_t max_length, float scale) {
  AttentionArgs a{};
  a.q = q; a.q_stride = q_stride; a.k_cache = k_cache; a.v_cache = v_cache; a.block_tables = block_tables; a.lengths = lengths;
  a.cu_seqlens = cu_seqlens; a.out = out; a.N = N; a.T = T; a.H = H; a.Hkv = Hkv; a.d = d; a.num_blocks = num_blocks;
  a.max_blocks = max_blocks; a.window = window; a.sinks = sinks; a.max_length = max_length; a.scale = scale;
  return a;
}

}  // namespace

KDA_API kda_status kda_window_attention_fwd(const void* q, const void* k_cache, const void* v_cache,
                                            const int32_t* block_tables, const int32_t* lengths, const int32_t* cu_seqlens,
                                            void* out, int N, int64_t T, int H, int Hkv, int d, int64_t q_stride,
                                            int num_blocks, int block_size, int max_blocks, const int64_t* cache_strides,
                                            int window, int sinks, int64_t max_length, float scale, void* stream) {
  if (N > 0 && T > 0 && !cu_seqlens) return KDA_ERR_INVALID_ARG;
  return attention(args_of(q, k_cache, v_cache, block_tables, lengths, cu_seqlens, out, N, T, H, Hkv, d, q_stride, num_blocks,
                           max_blocks, window, sinks, max_length, scale),
                   block_size, cache_strides, stream);
}

KDA_API kda_status kda_window_attention_decode_step(const void* q, const void* k_cache, const void* v_cache,
                                                    const int32_t* block_tables, const int32_t* lengths, void* out, int N,
                                                    int H, int Hkv, int d, int64_t q_stride, int num_blocks, int block_size,
                                                    int max_blocks, const int64_t* cache_strides, int window, int sinks,
                                                    int64_t max_length, float scale, void* stream) {
  return attention(args_of(q, k_cache, v_cache, block_tables, lengths, nullptr, out, N, N, H, Hkv, d, q_stride, num_blocks,
                           max_blocks, window, sinks, max_length, scale),
                   block_size, cache_strides, stream);
}

KDA_API kda_status kda_tree_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                      const int32_t* lengths, const int32_t* cu_seqlens, const uint64_t* tree_mask,
                                      int mask_words, void* out, int N, int64_t T, int H, int Hkv, int d, int64_t q_stride,
                                      int num_blocks, int block_size, int max_blocks, const int64_t* cache_strides,
                                      int window, int sinks, int64_t max_length, float scale, void* stream) {
  if (mask_words < 1) return KDA_ERR_INVALID_ARG;
  if (mask_words > 16) return KDA_ERR_UNSUPPORTED;
  if (N > 0 && T > 0 && (!cu_seqlens || !tree_mask)) return KDA_ERR_INVALID_ARG;
  AttentionArgs a = args_of(q, k_cache, v_cache, block_tables, lengths, cu_seqlens, out, N, T, H, Hkv, d, q_stride, num_blocks,
                            max_blocks, window, sinks, max_length, scale);
  a.tree_mask = tree_mask;
  a.mask_words = mask_words;
  return attention(a, block_size, cache_strides, stream);
}
