// Internal interfaces between the library's translation units (not exported).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <utility>

#include "pa.h"

namespace pa {

// Counts kernel launches (pa_launch_count).
void note_launch(int n = 1);

// Launch with programmatic stream serialisation (programmatic dependent
// launch): the kernel may start while the previous kernel on the stream is
// finishing; it synchronises with griddepcontrol.wait before touching memory
// that kernel may write.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e == cudaSuccess) note_launch();
  return e;
}

// The same for a grid of thread-block clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem,
                               cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
  if (e == cudaSuccess) note_launch();
  return e;
}

struct DecodeParams {
  const void* q;
  const int32_t* tables;
  const int32_t* lens;
  void* out;
  float* part_o;   // [num_seqs][q_heads][max_splits][head_dim]
  float* part_m;   // [num_seqs][q_heads][max_splits], log2 units
  float* part_l;   // [num_seqs][q_heads][max_splits]
  int* err;
  int maxblk, num_seqs, q_heads, kv_heads, group, num_blocks, block_size, split_tokens, max_splits;
  int tab_entries;  // block-table entries per partition: split_tokens / block_size
  float scale_log2;
  // Shared-prefix mode: attend only tokens [tok_begin, context_len) (the
  // request's own suffix), always write partials, to slots slot_base + c, and
  // check that each table starts with the prefix blocks.
  int tok_begin, slot_base, always_partial;
  const int32_t* prefix_blocks;
  int prefix_nblk;
  int grid_splits;  // partitions the grid covers (normal mode: max_splits)
  // Queries per request (1 = decode; k+1 = speculative verify).  Query i of
  // request r is row r*q_len + i of q / out / the partials and sees tokens
  // [0, context_len - (q_len-1-i)).
  int q_len;
  // Contiguous mode (launch_decode_contig): the cache is [num_slots][contig_len]
  // rows; request r reads slot slot_ids[r] (r if null); slot_tokens (may be
  // null) bounds the rows of each slot that are backed by memory.
  const int32_t* slot_ids;
  const int32_t* slot_tokens;
  int num_slots, contig_len;
  // launch_decode_logits: every column's scaled score (log2 units) of every
  // token of the partition, [num_seqs][kv_heads][cap][group_pad], and the sums
  // of the unrounded probabilities, laid out as part_l
  float* logits;
  float* part_w;
  int group_pad;
};

struct MergeParams {
  const float* part_o;
  const float* part_m;
  const float* part_l;
  const int32_t* lens;
  void* out;
  int num_seqs, q_heads, max_splits, split_tokens, cap;
  // shared-prefix mode: extra_slots partials precede the suffix partitions of
  // [tok_begin, context_len); every row is merged (even a single slot)
  int tok_begin, extra_slots, always;
  int q_len;  // queries per request: row / (q_heads * q_len) is the request
};

struct PrefillParams {
  const void* q;
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* tables;
  void* out;
  int* err;
  int maxblk, num_reqs, total_q, max_q_len, q_heads, kv_heads, group, num_blocks, block_size;
  float scale_log2;
  // Shared-prefix mode (tcgen05 kernel only; causal == 0): one virtual request
  // whose total_q "queries" are the decode queries of a batch, all seeing keys
  // [0, prefix_len) of the prefix table (`tables`, one row); grid.z splits the
  // keys into ranges of key_split; each range writes an unnormalised partial
  // (o, m in log2 units, l) to slot blockIdx.z of the decode workspace.
  int causal;
  int prefix_len, key_split, max_splits;
  // tcgen05 path: CTAs launched (each takes work units b, b + gridDim.x, ...);
  // <= 0 launches one CTA per unit
  int max_ctas;
  // > 0 (one-tile kernel, causal): every request has fixed_q_len queries, rows
  // r*fixed_q_len.. of q and out (q_start unused), and a context shorter than
  // that leaves the first queries without keys (zero rows): the speculative
  // verify
  int fixed_q_len;
  float* part_o;
  float* part_m;
  float* part_l;
};

// Workspace carve-up for decode partials.
struct DecodeWorkspace {
  size_t o_off, m_off, l_off, bytes;
};
DecodeWorkspace decode_workspace_layout(int num_seqs, int q_heads, int head_dim, int max_splits);

// Launchers (return cudaSuccess or the launch error).  `bsub` is the TMA box
// height min(block_size, 16); the tensor maps describe k_cache / v_cache as
// 4-D {64, head_dim/64, kv_heads, num_blocks*block_size} with boxes
// {64, 1, 1, bsub} and the 128-byte swizzle.
cudaError_t launch_decode_partial(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                                  int head_dim, int bsub, pa_dtype dt, cudaStream_t stream);
cudaError_t launch_lse_merge(const MergeParams& p, int head_dim, pa_dtype dt, cudaStream_t stream);
cudaError_t launch_decode_contig(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                                 int head_dim, pa_dtype dt, cudaStream_t stream);
// The decode partition pass (q_len 1, always_partial) that also stores p.logits.
cudaError_t launch_decode_logits(const CUtensorMap& kmap, const CUtensorMap& vmap, const DecodeParams& p,
                                 int head_dim, int bsub, pa_dtype dt, cudaStream_t stream);
cudaError_t launch_chunked_prefill(const CUtensorMap& kmap, const CUtensorMap& vmap, const PrefillParams& p,
                                   int head_dim, int bsub, pa_dtype dt, cudaStream_t stream);
// tcgen05/TMEM kernel for blocks of >= 8 tokens (bsub >= 8): chunked prefill
// (p.causal = 1) and the shared-prefix pass of a decode batch (p.causal = 0,
// partials).  Two 128-row Q tiles per CTA, 128-key K/V tiles, P kept in TMEM.
cudaError_t launch_wait_timeout(int* err, uint64_t limit_ns, cudaStream_t stream);
cudaError_t launch_attn_tc(const CUtensorMap& kmap, const CUtensorMap& vmap, const PrefillParams& p, int head_dim,
                           int bsub, pa_dtype dt, cudaStream_t stream);
// SMs of the current device (cached per device; 0 if the query fails).
int num_sms();
// Grid of a grid-stride copy kernel: enough 256-thread CTAs for `total`
// vectors, at most 16 per SM of the current device.
inline unsigned copy_grid(int64_t total) {
  const int64_t cap = 16 * (int64_t)(num_sms() > 0 ? num_sms() : 1);
  const int64_t want = (total + 255) / 256;
  return (unsigned)(want < cap ? want : cap);
}
// tcgen05 kernel with one 128-row tile per (request, KV head) work unit and
// Q, P in tensor memory (causal with fixed_q_len: the speculative verify).
cudaError_t launch_attn_tile(const CUtensorMap& kmap, const CUtensorMap& vmap, const PrefillParams& p,
                             int head_dim, int bsub, pa_dtype dt, cudaStream_t stream);
cudaError_t launch_reshape_and_cache(const void* k, const void* v, const int32_t* slots, int num_tokens,
                                     void* k_cache, void* v_cache, int64_t num_slots, int row_bytes, int* err,
                                     cudaStream_t stream);
// pointers as the kernel dereferences them (host pools through their mapped
// device addresses); block_bytes = one block of K (or V)
cudaError_t launch_reshape_and_cache_slots(const void* k, const void* v, const int32_t* slot_ids,
                                           const int32_t* positions, int num_tokens, void* k_cache, void* v_cache,
                                           int num_slots, int contig_len, const int32_t* slot_tokens, int row_bytes,
                                           int* err, cudaStream_t stream);
cudaError_t launch_swap_blocks(const void* src_k, const void* src_v, void* dst_k, void* dst_v, const int32_t* pairs,
                               int num_pairs, int num_src, int num_dst, int64_t block_bytes, int* err,
                               cudaStream_t stream);
cudaError_t launch_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int num_pairs,
                               int num_blocks, int64_t block_bytes, int* err, cudaStream_t stream);


// Norm, rotation and cache write of new tokens (pa_norm_rope_and_cache).
struct NormRopeParams {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const void* q_weight;                  // null: no norm
  const void* k_weight;
  const int32_t* positions;  // [num_axes][num_tokens]
  const float* cos_sin;      // [max_position][rot_dim]
  const int32_t* slots;
  void* q_out;
  void* k_cache;
  void* v_cache;
  int* err;
  int64_t num_slots;
  int num_tokens, q_heads, kv_heads, num_axes, max_position, rot_dim, interleaved;
  int sec_end[2];  // pairs before sec_end[0] turn by axis 0, before sec_end[1] by axis 1, the rest by axis 2
  float eps;
};
cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, pa_dtype dt, cudaStream_t stream);

// Attention of drafted trees (pa_verify_tree).
struct TreeParams {
  const void* q;
  const void* v_cache;  // read beside its tensor map for the rare nodes whose V is not finite
  const int32_t* q_start;
  const uint64_t* mask;  // [total_q]
  const int32_t* lens;
  const int32_t* tables;
  void* out;
  int* err;
  int maxblk, num_reqs, total_q, max_q_len, q_heads, kv_heads, group, num_blocks, block_size;
  int split_tokens, max_splits;  // partitions of the context; one: no scratch
  int longest_first;             // 1 (max_splits == 1 only): requests run in order of length (tree_longest_first)
  float scale_log2;
  float* part_o;  // [total_q * q_heads][max_splits][head_dim], as the decode partials
  float* part_m;
  float* part_l;
};
// without the merge: the tcgen05 kernels of attn_tile.cu (128 rows per CTA) and
// attn_tc.cu (256)
cudaError_t launch_tree_pair(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int head_dim,
                             int bsub, pa_dtype dt, cudaStream_t stream);
cudaError_t launch_tree_tile(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int head_dim,
                             int bsub, pa_dtype dt, cudaStream_t stream);
cudaError_t launch_verify_tree(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int head_dim,
                               int bsub, pa_dtype dt, cudaStream_t stream);

struct EvictSelectParams {
  const float* scores;  // [num_rows][kv_heads][score_len]
  const int32_t* score_rows;
  const int32_t* lens;
  int32_t* keep;  // [num_seqs][kv_heads][sink + heavy + recent]
  int32_t* keep_lens;
  int* err;
  int num_rows, kv_heads, score_len, sink, heavy, recent;
  int warp_held, warp_list;  // set by the launcher: keys and listed keys a warp has room for in shared memory
};
cudaError_t launch_evict_select(const EvictSelectParams& p, int num_seqs, cudaStream_t stream);

struct CompactParams {
  void* k_cache;
  void* v_cache;
  const int32_t* tables;
  const int32_t* lens;
  const int32_t* keep;  // [num_seqs][keep_heads][max_keep]
  const int32_t* keep_lens;
  const int32_t* base;  // null: 0
  float* scores;        // null: none
  const int32_t* score_rows;
  int* err;
  int maxblk, cap, keep_heads, max_keep, num_blocks, block_size, kv_heads, num_rows, score_len;
  int row_vecs;  // 16-byte vectors of one head's row
  int columns;   // set by the launcher
};
cudaError_t launch_compact_kv(const CompactParams& p, int num_seqs, cudaStream_t stream);

// pa_decode_accumulate: what the partition pass leaves of the logits, and the
// pass that turns them into weights (after the merge's inputs are complete).
struct AccumulateParams {
  const float* logits;  // [num_seqs][kv_heads][cap][group_pad], log2 units
  const float* part_m;  // as MergeParams
  const float* part_w;  // sums of the unrounded probabilities
  const int32_t* lens;
  const float* scores;
  float* scores_out;
  const int32_t* score_rows;
  int* err;
  int num_seqs, q_heads, kv_heads, group, group_pad, max_splits, split_tokens, cap, num_rows, score_len;
  int chunk, chunks;  // set by the launcher: tokens of a CTA, CTAs of a (request, KV head)
};
cudaError_t launch_merge_accumulate(const MergeParams& mp, const AccumulateParams& ap, int head_dim, pa_dtype dt,
                                    cudaStream_t stream);

}  // namespace pa
