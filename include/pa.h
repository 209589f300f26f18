/*
 * pa.h - C ABI of a paged-KV-cache attention library for NVIDIA GB300 (sm_103a).
 *
 * The KV cache is split into fixed-size physical blocks of `block_size` tokens;
 * a request's logical blocks map to physical blocks through its Block Table,
 * so its KV need not be contiguous ("2.1 PagedAttention", §2-§3).  Attention
 * kernels translate each logical token t into (physical_block_number =
 * table[t / block_size], physical_block_offset = t % block_size) (§5).
 *
 * Conventions for every call below
 * --------------------------------
 * - Cache layout: k_cache and v_cache are separate tensors, each
 *   [num_blocks][block_size][kv_heads][head_dim], row-major, contiguous.
 * - Block tables: int32 [num_seqs][max_blocks_per_seq], row-major; entries
 *   past a request's last logical block are never read (any value).
 * - Element types: PA_FP16 or PA_BF16 for q/k/v/out (inputs and outputs in the
 *   same type); accumulation and softmax are fp32.
 * - head_dim in {64, 128}; block_size in {4, 8, 16, 32};
 *   q_heads % kv_heads == 0 and q_heads / kv_heads <= 16.  Query head h reads
 *   KV head h / (q_heads / kv_heads) (contiguous GQA groups).
 * - Device calls: every pointer is device memory owned by the caller; the
 *   library allocates no device memory and keeps no pointer after returning.
 *   Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL = the
 *   legacy default stream).  All device pointers must be 16-byte aligned.
 * - Ordering: kernels are launched with programmatic dependent launch.  A
 *   kernel of this library may start its set-up while the kernel before it on
 *   the same stream is finishing, and reads only q, block tables, q_start and
 *   context lengths during that set-up; caches, scratch and outputs are read
 *   or written only once the previous kernel has completed.  So those four
 *   inputs must be ready when the call is enqueued (they are if whatever writes
 *   them was enqueued earlier on the stream without allowing early launch of
 *   its successor, as plain kernels and copies do; pa_norm_rope_and_cache, whose
 *   q_out is such an input, pa_evict_select, whose keep_lens may be, and
 *   pa_fork_blocks, whose tables and lengths are, do the same).
 * - Errors: every call returns a pa_status.  Argument errors are caught on the
 *   host before anything is launched.  Data errors that only the device can
 *   see (a block id outside [0, num_blocks), a slot past the pool, a context
 *   length past the table, a wait that timed out) never fault or trap: the
 *   kernel records the first such code in a per-device error word, skips the
 *   offending access, and finishes; read it with pa_get_device_error().
 *   Nothing aborts, nothing throws.
 * - Thread safety: device calls may be made from any host thread.  A pa_alloc
 *   handle is single-threaded.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID = -1,        /* bad argument (shape, pointer, id, range)        */
  PA_ERR_NO_FREE_BLOCKS = -2, /* pool exhausted; allocator state unchanged      */
  PA_ERR_DTYPE = -3,          /* unsupported element type                       */
  PA_ERR_CUDA = -4,           /* a CUDA runtime/driver call failed              */
  PA_ERR_DEVICE_CHECK = -5,   /* pa_get_device_error found a recorded error     */
  PA_ERR_SHARED_BLOCK = -6,   /* append into a shared partial block: cow first  */
  PA_ERR_WORKSPACE = -7,      /* workspace missing or smaller than required     */
  PA_ERR_HOST_MEMORY = -8     /* a host allocation failed; nothing changed      */
} pa_status;

typedef enum { PA_FP16 = 0, PA_BF16 = 1 } pa_dtype;

/* Device error codes recorded by kernels (first one wins). */
enum {
  PA_DEVERR_NONE = 0,
  PA_DEVERR_BLOCK_ID = 1,     /* block-table entry or copy pair outside [0, num_blocks) */
  PA_DEVERR_CONTEXT_LEN = 2,  /* context length < 0 or > max_blocks_per_seq*block_size */
  PA_DEVERR_SLOT = 3,         /* slot_mapping entry >= num_blocks*block_size            */
  PA_DEVERR_TIMEOUT = 4,      /* a bounded wait on a shared-memory barrier expired      */
  PA_DEVERR_QUERY_RANGE = 5,  /* bad q_start / chunk length in chunked prefill          */
  PA_DEVERR_POSITION = 6,     /* rotary position outside [0, max_position)              */
  PA_DEVERR_SCORE_ROW = 7,    /* score row outside the score array, or used twice       */
  PA_DEVERR_KEEP = 8,         /* keep list: bad count, base, or an entry out of range   */
  PA_DEVERR_FORK = 9,         /* fork: parent >= num_seqs, or growth outside [0, max]   */
  PA_DEVERR_NO_BLOCKS = 10    /* fork: fewer free blocks than the new rows need         */
};

typedef struct CUstream_st* pa_stream; /* identical to cudaStream_t */

/* Human-readable name of a pa_status value (static string). */
const char* pa_status_string(int status);

/* Library version, major*10000 + minor*100 + patch. */
int pa_version(void);

/* Number of kernels this library has launched in this process. */
uint64_t pa_launch_count(void);

/* ----------------------------------------------------------------------------
 * pa_reshape_and_cache - scatter new tokens' K/V into their slots.
 *
 * "2.1 PagedAttention" §3: each new token fills the next free slot of its
 * request's current block; the forward pass writes the KV into the blocks the
 * allocator handed out ("Khám phá vLLM … phần 2", prefix caching).  For token
 * i with slot s = slot_mapping[i] >= 0:
 *     k_cache[s / block_size][s % block_size][:][:] = k[i][:][:]   (same for v)
 * A negative slot marks a padding token and is skipped.  The copy is
 * bit-exact.
 *   k, v          [num_tokens][kv_heads][head_dim], contiguous
 *   slot_mapping  int32 [num_tokens]; slots must be distinct
 *   k_cache,v_cache  the pool (see conventions)
 * num_tokens == 0 is a no-op.  A slot >= num_blocks*block_size records
 * PA_DEVERR_SLOT and is skipped.
 * ------------------------------------------------------------------------- */
int pa_reshape_and_cache(const void* k, const void* v, const int32_t* slot_mapping, int num_tokens,
                         void* k_cache, void* v_cache, int num_blocks, int block_size, int kv_heads,
                         int head_dim, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_copy_blocks - the device half of Copy-on-Write.
 *
 * "2.1 PagedAttention" §6: before a request writes a block other requests
 * share, the block is copied to a private block and the request's table
 * entry is repointed (the allocator's pa_alloc_cow does the bookkeeping).
 * For each pair p: block pairs[2p+1] (dst) of k_cache and v_cache becomes a
 * bit-exact copy of block pairs[2p] (src).
 *   pairs  int32 [num_pairs][2] (src, dst), DEVICE memory.  A dst must not
 *          repeat nor be the src of another pair (otherwise the result is
 *          unspecified).  Ids outside [0, num_blocks) record
 *          PA_DEVERR_BLOCK_ID and the pair is skipped.
 * num_pairs == 0 is a no-op.
 * ------------------------------------------------------------------------- */
int pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int num_pairs, int num_blocks,
                   int block_size, int kv_heads, int head_dim, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_swap_blocks - the device half of preemption by swapping.
 *
 * "2.1 PagedAttention" §7: when the GPU pool runs short, a request's blocks
 * are copied to a pool in CPU memory and its GPU blocks are released; later
 * they are copied back into fresh GPU blocks (pa_alloc_swap_out /
 * pa_alloc_swap_in do the bookkeeping and produce the pairs).  For each pair
 * p: block pairs[2p+1] of (dst_k, dst_v) becomes a bit-exact copy of block
 * pairs[2p] of (src_k, src_v).  Both pools have the KV-cache layout
 * [num_*_blocks][block_size][kv_heads][head_dim].
 *   src_*, dst_*  device memory or PAGE-LOCKED host memory (cudaHostAlloc /
 *          cudaHostRegister, mapped); the kernel reads and writes host memory
 *          directly over the CPU-GPU link.  Pageable host memory is rejected
 *          with PA_ERR_INVALID.  All four 16-byte aligned.
 *   pairs  int32 [num_pairs][2] (src, dst), device or page-locked host
 *          memory.  dst ids must not repeat.  A src id outside
 *          [0, num_src_blocks) or a dst id outside [0, num_dst_blocks)
 *          records PA_DEVERR_BLOCK_ID and the pair is skipped.
 * The call is asynchronous on stream; host buffers must stay alive and
 * untouched until it completes.  num_pairs == 0 is a no-op.
 * ------------------------------------------------------------------------- */
int pa_swap_blocks(const void* src_k, const void* src_v, void* dst_k, void* dst_v, const int32_t* pairs,
                   int num_pairs, int num_src_blocks, int num_dst_blocks, int block_size, int kv_heads,
                   int head_dim, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * Paged decode attention (one query token per request).
 *
 * "2.1 PagedAttention" §3 and §5: the kernel reads the request's whole KV
 * history from scattered physical blocks through its Block Table.  For
 * request r and query head h (g = h / (q_heads / kv_heads)):
 *     s_t = scale * <q[r][h], K_r[t][g]>           for t < context_lens[r]
 *     out[r][h] = sum_t softmax(s)_t * V_r[t][g]
 * context_lens[r] counts every token of the request, including the one this
 * step wrote with pa_reshape_and_cache.  A zero context gives a zero row.
 *
 * The context is processed in partitions of `split_tokens` tokens (0 = the
 * library's choice).  pa_decode_split_tokens returns the partition size a
 * call with these arguments uses, or PA_ERR_INVALID if split_tokens is not
 * allowed.  A request with one
 * partition is written straight to `out`; a request with more keeps per
 * partition the unnormalised output o_c, the reference maximum m_c its
 * exponents were taken against (the running maximum, or up to 8 below it in
 * log2 units) and the sum l_c, and pa_lse_merge combines them:
 * M = max_c m_c,  out = sum_c e^(m_c-M) o_c / sum_c e^(m_c-M) l_c.
 *
 *   q             [num_seqs][q_heads][head_dim]
 *   out           [num_seqs][q_heads][head_dim]
 *   block_tables  int32 [num_seqs][max_blocks_per_seq]
 *   context_lens  int32 [num_seqs], each in [0, max_blocks_per_seq*block_size]
 *   split_tokens  0, or a multiple of max(16, block_size) no larger than
 *                 256*block_size
 *   workspace     device scratch of at least pa_decode_workspace_size(...)
 *                 bytes (may be NULL when that size is 0).  Owned by the
 *                 caller; its contents need no initialisation.
 * pa_decode = pa_decode_partial followed by pa_lse_merge on the same stream.
 * ------------------------------------------------------------------------- */
int pa_decode_split_tokens(int max_blocks_per_seq, int block_size, int split_tokens);

size_t pa_decode_workspace_size(int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq,
                                int block_size, int split_tokens);

int pa_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
              int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_heads,
              int kv_heads, int head_dim, int block_size, int num_blocks, float scale,
              int split_tokens, void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype,
              pa_stream stream);

/* First half of pa_decode: per-partition partials (or the final row for
 * requests with a single partition). Same arguments as pa_decode. */
int pa_decode_partial(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads,
                      int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                      void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype,
                      pa_stream stream);

/* Second half of pa_decode: log-sum-exp merge of the partials of every request
 * with more than one partition.  Arguments must match the pa_decode_partial
 * call whose workspace it reads. */
int pa_lse_merge(const void* workspace, size_t workspace_bytes, const int32_t* context_lens,
                 int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq, int block_size,
                 int split_tokens, void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_verify_decode - the attention of the verify step of speculative decoding.
 *
 * "Khám phá vLLM … phần 2", speculative decoding: a proposer drafts k tokens
 * and the large model checks them in ONE forward pass over the context plus
 * the drafts, which yields k+1 distributions.  Its attention is decode with
 * q_len = k+1 queries per request: the drafts' K/V are written first (with
 * pa_reshape_and_cache, into slots the allocator appended), so
 * context_lens[r] = L counts them, and query i (0 <= i < q_len) of request r
 * attends tokens [0, L - (q_len-1-i)) - causal inside the draft.  A query
 * that sees no token gives a zero row.  All q_len*group query rows of a KV
 * head share every K/V tile read, so the pass costs the KV bytes of one
 * decode step.
 *   q, out        [num_seqs][q_len][q_heads][head_dim]
 *   q_len         >= 1, with (q_heads / kv_heads) * q_len <= 32
 *   split_tokens  as pa_decode; 0 = the library's choice, which for q_len > 1
 *                 and contexts up to 8192 tokens is 768 (longer than decode's:
 *                 each partition's partials and merge rows grow with q_len)
 *   workspace     at least pa_verify_workspace_size(...) bytes
 * Everything else as pa_decode (which is the q_len = 1 case).
 * pa_verify_split_tokens returns the partition size such a call uses, or
 * PA_ERR_INVALID.
 * ------------------------------------------------------------------------- */
int pa_verify_split_tokens(int max_blocks_per_seq, int block_size, int q_len, int split_tokens);

size_t pa_verify_workspace_size(int num_seqs, int q_len, int q_heads, int head_dim, int max_blocks_per_seq,
                                int block_size, int split_tokens);

int pa_verify_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                     int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                     void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_verify_decode_tc - the same verify attention on the tensor cores.
 *
 * The computation of pa_verify_decode ("Khám phá vLLM … phần 2",
 * speculative decoding: query i of request r attends tokens
 * [0, context_lens[r] - (q_len-1-i))), read as what it also is: a chunked
 * prefill of a q_len-token chunk at the end of the context.  The
 * (query, group head) rows of one (request, KV head) - at most 128 - are one
 * work unit of a tcgen05 kernel (tensor memory, TMA gathers) that walks the
 * whole context in 128-key tiles; no workspace, no merge.  A unit's gather
 * cost does not depend on its row count, so this form pays when the rows are
 * many (k = 7 drafts x 4 group heads = 32) and the batch gives every SM units.
 *   q, out        [num_seqs][q_len][q_heads][head_dim], as pa_verify_decode
 *   q_len         >= 1, with (q_heads / kv_heads) * q_len <= 128
 *   block_size    8, 16 or 32 (the gather's boxes hold 8-row swizzle atoms)
 *   max_ctas      0: one CTA per unit; > 0: that many CTAs, each taking units
 *                 b, b + max_ctas, ... (one CTA per SM fits)
 * With one CTA per unit, units of at most 32 rows are spread over all four
 * tensor-memory lane quarters (each takes a quarter of every key tile; the
 * four partial results are merged exactly); a capped grid keeps them in one.
 * Results equal pa_verify_decode's within the attention tolerance (the sums
 * are taken in another order); a query that sees no token gives a zero row.
 * Errors as pa_chunked_prefill.
 * ------------------------------------------------------------------------- */
int pa_verify_decode_tc(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                        int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int max_ctas,
                        void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * Contiguous virtual KV, vAttention style ("vAttention 完全拆解") - the
 * competing design, built as a comparison baseline for the paged kernels.
 *
 * Each K and V tensor of each layer is ONE contiguous virtual range
 * [num_slots][max_len][kv_heads][head_dim]; request slot s starts at
 * s*max_len*kv_heads*head_dim*2 bytes, token t of the slot is row
 * s*max_len + t, and no Block Table exists.  Physical pages (CUDA virtual
 * memory: cuMemCreate / cuMemMap / cuMemSetAccess) are mapped into a slot
 * only when pa_vkv_step sees its length reach them:
 *  - pages for n tokens: ceil(roundup(n, 16) * kv_heads*head_dim*2 /
 *    page_bytes) in every one of the 2*num_layers sub-tensors (the attention
 *    kernel reads whole 16-token tiles, so the rounded length is mapped);
 *  - pa_vkv_free_slot keeps the slot's pages mapped; pa_vkv_alloc_slot hands
 *    out the free slot holding the most pages (lowest id on ties), whose
 *    pages the new request reuses;
 *  - a step that needs more than max_pages mapped pages in total unmaps whole
 *    inactive slots (lowest id first, after cudaDeviceSynchronize) and fails
 *    with PA_ERR_NO_FREE_BLOCKS, changing nothing, if even that is not enough.
 * page_bytes = 0 takes the driver's minimum granularity (2 MiB on current
 * GPUs); max_len * kv_heads*head_dim*2 must be a multiple of page_bytes and
 * max_len a multiple of 16.  PA_VKV_DRY_RUN keeps only the bookkeeping (no
 * memory, no GPU needed; page_bytes must then be given).
 * Kernels only ever touch rows below a slot's mapped bound: pa_vkv_decode and
 * pa_vkv_reshape_and_cache check every access against the device copy of the
 * per-slot mapped token counts, which pa_vkv_step updates in stream order.
 * ------------------------------------------------------------------------- */
typedef struct pa_vkv pa_vkv;
#define PA_VKV_DRY_RUN 1

typedef struct {
  int64_t page_bytes;
  int64_t slot_pages;        /* virtual pages per slot per sub-tensor          */
  int64_t pages_mapped;      /* over all sub-tensors                           */
  int64_t pages_pooled;      /* created, currently unmapped                    */
  int64_t pages_created;     /* cuMemCreate calls                              */
  int64_t map_calls;         /* page mappings made (one per page per tensor)   */
  int64_t unmap_calls;
  int64_t bytes_reserved;    /* virtual address space                          */
  int64_t bytes_committed;   /* pages_mapped * page_bytes                      */
  int64_t last_step_map_ns;  /* host time the last pa_vkv_step spent mapping   */
  int64_t total_map_ns;
  int64_t active_slots;
  int64_t step_failures;     /* pa_vkv_step calls refused for want of pages   */
  int64_t bytes_used;        /* K/V bytes of the last step's tokens; tail
                                waste = bytes_committed - bytes_used        */
} pa_vkv_stats;

int pa_vkv_granularity(size_t* out);
int pa_vkv_create(int num_slots, int max_len, int num_layers, int kv_heads, int head_dim, pa_dtype dtype,
                  size_t page_bytes, int64_t max_pages, int flags, pa_vkv** out);
/* Synchronises the device, unmaps and releases every page, frees the range. */
void pa_vkv_destroy(pa_vkv* v);
int pa_vkv_alloc_slot(pa_vkv* v, int* slot_out);
int pa_vkv_free_slot(pa_vkv* v, int slot);
/* lens: HOST int32 [num_slots], the length every slot reaches this iteration
 * (0 for inactive slots).  Maps what is missing, then copies the per-slot
 * mapped token counts to the device on `stream`. */
int pa_vkv_step(pa_vkv* v, const int32_t* lens, pa_stream stream);
/* Base of layer `layer`'s K (is_v = 0) or V tensor; NULL in dry-run mode. */
int pa_vkv_tensor(const pa_vkv* v, int layer, int is_v, void** out);
/* Tokens of each slot backed by mapped pages: into host_out [num_slots] (may
 * be NULL); *device_out (may be NULL) = the device copy the kernels read. */
int pa_vkv_slot_tokens(const pa_vkv* v, int32_t* host_out, const int32_t** device_out);
int pa_vkv_slot_pages(const pa_vkv* v, int slot);
int pa_vkv_get_stats(const pa_vkv* v, pa_vkv_stats* out);

/* Decode over a contiguous [num_slots][max_len][kv_heads][head_dim] cache:
 * request r reads slot slot_ids[r] (device int32 [num_seqs]; NULL: slot r),
 * tokens [0, context_lens[r]).  slot_tokens (device int32 [num_slots], may be
 * NULL = all max_len rows exist) bounds the rows each slot has backed by
 * memory: a context past it records PA_DEVERR_CONTEXT_LEN and its tokens past
 * the bound count as absent; a bad slot id records PA_DEVERR_BLOCK_ID and
 * gives a zero row.  Same math, partitions (pa_decode_split_tokens(max_len/16,
 * 16, split_tokens)) and workspace (pa_decode_workspace_size(num_seqs,
 * q_heads, head_dim, max_len/16, 16, split_tokens)) as pa_decode with 16-token
 * blocks, whose result it equals bit for bit on the same K/V. */
int pa_decode_contiguous(const void* q, const void* k_cache, const void* v_cache, int num_slots, int max_len,
                         const int32_t* slot_ids, const int32_t* slot_tokens, const int32_t* context_lens,
                         int num_seqs, int q_heads, int kv_heads, int head_dim, float scale, int split_tokens,
                         void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream);
/* reshape_and_cache into a contiguous cache: token i to row
 * slot_ids[i]*max_len + positions[i] (slot < 0: padding, skipped); a
 * position outside [0, bound) - bound = slot_tokens[slot] or max_len - records
 * PA_DEVERR_SLOT and is skipped. */
int pa_reshape_and_cache_slots(const void* k, const void* v, const int32_t* slot_ids, const int32_t* positions,
                               int num_tokens, void* k_cache, void* v_cache, int num_slots, int max_len,
                               const int32_t* slot_tokens, int kv_heads, int head_dim, pa_dtype dtype,
                               pa_stream stream);
/* The two calls above on layer `layer` of a manager, with its mapped bounds. */
int pa_vkv_decode(const pa_vkv* v, int layer, const void* q, const int32_t* slot_ids, const int32_t* context_lens,
                  int num_seqs, int q_heads, float scale, int split_tokens, void* workspace, size_t workspace_bytes,
                  void* out, pa_stream stream);
int pa_vkv_reshape_and_cache(const pa_vkv* v, int layer, const void* k, const void* vv, const int32_t* slot_ids,
                             const int32_t* positions, int num_tokens, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_decode_shared_prefix - decode for a batch whose requests all start with
 * the same physical blocks (a shared prompt prefix).
 *
 * "2.1 PagedAttention" §6: with paging, many Block Tables point at the same
 * physical blocks of a common prefix.  Instead of reading those blocks once per
 * request, this call attends the prefix once for every request's queries:
 * rows (request, query head of the group) x prefix keys are dense tiles for the
 * 5th-generation tensor cores, split into key ranges (512 tokens), each
 * producing a log-sum-exp partial; each request's own suffix (tokens
 * prefix_len .. context_lens[r]-1) runs through the paged decode kernel into
 * further partials; the merge combines them.  The result equals pa_decode
 * with the full tables, up to floating-point rounding.
 *   prefix_blocks  int32 [prefix_len / block_size], DEVICE memory: the shared
 *                  physical blocks in logical order.  Every row of
 *                  block_tables must begin with them (checked on the device:
 *                  a mismatch records PA_DEVERR_BLOCK_ID).
 *   prefix_len     host int, > 0, a multiple of block_size, <= every
 *                  context_lens[r] (a shorter context records
 *                  PA_DEVERR_CONTEXT_LEN).  pa_alloc_common_prefix gives the
 *                  number of shared full blocks of a set of sequences.
 *   workspace      at least pa_decode_shared_prefix_workspace_size(...) bytes.
 *   prefix_stream  NULL (or == stream): all three passes run on `stream`.
 *                  Otherwise the prefix pass runs on prefix_stream, with NO
 *                  dependency on `stream`, concurrently with the suffix pass
 *                  (the prefix pass is tensor-core work on a few SMs, the
 *                  suffix pass HBM-bound on the rest); the merge on `stream`
 *                  waits for it.  The caller orders prefix_stream after every
 *                  write of q, prefix_blocks and the prefix's K/V, and after
 *                  every earlier use of the workspace.  In this mode the
 *                  prefix key ranges grow (512 x 2^k tokens) until the prefix
 *                  pass needs at most a quarter of the SMs.
 * Other arguments as pa_decode.  With 4-token blocks this is pa_decode (on
 * `stream`).
 * ------------------------------------------------------------------------- */
size_t pa_decode_shared_prefix_workspace_size(int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq,
                                              int block_size, int prefix_len, int split_tokens);

/* The partition size pa_decode_shared_prefix uses for the suffixes: split_tokens
 * if it is > 0, else about a quarter of the suffix bound
 * (max_blocks_per_seq * block_size - prefix_len), at least 128 tokens and at
 * most pa_decode_split_tokens(max_blocks_per_seq, block_size, 0).  Negative:
 * a pa_status error for invalid arguments. */
int pa_decode_shared_prefix_split_tokens(int max_blocks_per_seq, int block_size, int prefix_len, int split_tokens);

int pa_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache, const int32_t* prefix_blocks,
                            int prefix_len, const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads, int head_dim,
                            int block_size, int num_blocks, float scale, int split_tokens, void* workspace,
                            size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream,
                            pa_stream prefix_stream);

/* ----------------------------------------------------------------------------
 * pa_chunked_prefill - a chunk of prompt tokens per request attends its paged
 * history plus itself, causally.
 *
 * "Khám phá vLLM … phần 2", chunked prefill: a long prompt is prefilled a
 * bounded number of tokens per engine step; the chunk's K/V are written to the
 * cache first (pa_reshape_and_cache) and its queries attend everything before
 * them.  Request r's queries are rows q_start[r] .. q_start[r+1]-1 of q;
 * context_lens[r] includes the chunk, so the chunk starts at absolute
 * position p0 = context_lens[r] - chunk and query i sees keys 0 .. p0 + i.
 *   q, out        [total_q][q_heads][head_dim]
 *   q_start       int32 [num_reqs + 1], non-decreasing, q_start[num_reqs] <= total_q
 *   max_q_len     host-side upper bound of any chunk length (sizes the grid)
 *   max_ctas      with blocks of >= 8 tokens the work is cut into units of
 *                 256 (query, group head) rows of one (request, KV head);
 *                 at most max_ctas CTAs (one per SM) loop over them.  <= 0:
 *                 one CTA per unit.  A caller that runs decode concurrently
 *                 on another stream can leave the remaining SMs to it (decode
 *                 is bound by HBM, not by SM count).  Ignored for 4-token
 *                 blocks.
 * A chunk longer than max_q_len or a context shorter than its chunk records
 * PA_DEVERR_QUERY_RANGE and that request is skipped.
 * ------------------------------------------------------------------------- */
int pa_chunked_prefill(const void* q, const int32_t* q_start, const int32_t* context_lens,
                       const void* k_cache, const void* v_cache, const int32_t* block_tables,
                       int max_blocks_per_seq, int num_reqs, int total_q, int max_q_len, int max_ctas,
                       int q_heads, int kv_heads, int head_dim, int block_size, int num_blocks,
                       float scale, void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_decode_noalloc - pa_decode without a caller-provided workspace.
 *
 * The pages have no counterpart to this call: it only repackages pa_decode
 * for callers that cannot allocate device memory for the decode scratch - a
 * plugin inside a host framework that has already reserved the GPU's memory
 * for its own pool and offers the plugin no allocator, or a latency-critical
 * loop where cudaMalloc/cudaFree (which can synchronise the device) are not
 * acceptable.  The caller still passes all inputs and outputs (same meaning
 * as pa_decode); the split-K partials go to a scratch array held by the
 * library: a file-scope device array of PA_DECODE_NOALLOC_SCRATCH_BYTES
 * (16 MiB) that every GPU loading the library keeps until the process exits.
 * The call allocates nothing.
 *
 * - Size limit: if the scratch this call needs (pa_decode_workspace_size with
 *   the same arguments) exceeds PA_DECODE_NOALLOC_SCRATCH_BYTES it returns
 *   PA_ERR_WORKSPACE and launches nothing; use pa_decode with your own
 *   workspace then.  Requests that fit one partition need no scratch.
 * - Set-up: the first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.  The address is looked up again when the
 *   device's current context changes (after cudaDeviceReset the library's
 *   device code is loaded anew and the array may move); the first call after
 *   such a reset should also come before any capture.
 * - Sharing: all calls share the one array, which keeps the last call's
 *   contents.  Nothing in it has to start at zero (every partial the merge
 *   reads is written earlier in the same call).  Calls that overlap on the
 *   GPU (two streams, or two host threads launching at once) race on the
 *   array and corrupt each other's results: serialise them.
 * ------------------------------------------------------------------------- */
#define PA_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

int pa_decode_noalloc(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_heads,
                      int kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                      int split_tokens, void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_norm_rope_and_cache - what stands between the query/key/value projection
 * and the cache, in one pass: per-head norm, rotary position, and the writes of
 * pa_reshape_and_cache.
 *
 * For token i, every query head x = q[i][h] and key head x = k[i][g]:
 *   norm   (weight not NULL)  x_d <- x_d * rsqrt(mean_d(x_d^2) + eps) * weight_d
 *   rotate the first rot_dim elements: pair p of rot_dim/2 is elements
 *          (p, p + rot_dim/2), or (2p, 2p+1) if interleaved != 0;
 *          (a, b) <- (a cos - b sin, b cos + a sin) with
 *          cos = cos_sin[pos][p], sin = cos_sin[pos][rot_dim/2 + p],
 *          pos = positions[axis(p)][i]
 * computed in fp32 and rounded once.  Queries go to q_out, keys and values
 * (values bit-exactly) to slot slot_mapping[i] of the caches.  A position is
 * any number of the table, not the slot's place in its sequence: the nodes of
 * a drafted tree at one depth share it, and a cache whose tokens were moved
 * (pa_compact_kv) keeps the rotations its keys were written with.
 *   q, k, v       [num_tokens][heads][head_dim], each token's heads
 *                 contiguous, tokens *_stride elements apart (a multiple of 8,
 *                 at least heads*head_dim): rows of one fused projection will do
 *   q_weight, k_weight  [head_dim] in dtype, or NULL: no norm
 *   positions     int32 [num_axes][num_tokens], num_axes 1 to 3 (for images and
 *                 video: time, height, width)
 *   sections      HOST int [num_axes], sum rot_dim/2: pairs [0, s0) turn by axis
 *                 0, the next s1 by axis 1, ...; NULL with one axis
 *   cos_sin       fp32 [max_position][rot_dim]: cosines, then sines
 *   rot_dim       a multiple of 16, 16 <= rot_dim <= head_dim
 *   slot_mapping  int32 [num_tokens] as pa_reshape_and_cache (distinct, < 0: the
 *                 token's K/V are not written; its query still is)
 *   q_out         [num_tokens][q_heads][head_dim]; may be q itself when q's
 *                 rows are contiguous, else it must not overlap the inputs
 * A position outside the table records PA_DEVERR_POSITION (unless the slot is
 * negative: padding) and nothing of that token is written.  A slot past the
 * pool records PA_DEVERR_SLOT and the token's K/V are skipped.  num_tokens == 0
 * is a no-op.
 * ------------------------------------------------------------------------- */
int pa_norm_rope_and_cache(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                           const int32_t* positions, int num_axes, const int32_t* sections, const float* cos_sin,
                           int max_position, int rot_dim, int interleaved, const int32_t* slot_mapping,
                           int num_tokens, int q_heads, void* q_out, void* k_cache, void* v_cache, int num_blocks,
                           int block_size, int kv_heads, int head_dim, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_verify_tree - the verify attention when the draft is a tree.
 *
 * Request r drafted n = q_start[r+1] - q_start[r] tokens (at most 64), node j's
 * K/V in the cache as token context_lens[r] - n + j.  Row i = q_start[r] + j
 * (node j) attends
 *     every token t < context_lens[r] - n, and
 *     node m (token context_lens[r] - n + m) for each bit m < n of tree_mask[i]
 * - for a drafted tree the node itself and its ancestors - and no other; bits
 * from n on are ignored.  A row that sees nothing gives zeros.  A node's K/V
 * never reach a row that does not see it, whatever they hold (stale slots of
 * padding nodes may hold NaN).  Ragged batches are packed: a request may have
 * no rows.  pa_verify_decode is the chain (mask bits 0..j).
 *   q, out        [total_q][q_heads][head_dim]
 *   q_start       int32 [num_reqs + 1], non-decreasing, q_start[num_reqs] <= total_q
 *   tree_mask     uint64 [total_q]; read during set-up, like q and q_start
 *   max_q_len     host-side bound of n, 1..64 (sizes the grid and the scratch)
 *   split_tokens  0 = the library's choice; else a multiple of 128: the context
 *                 is attended in partitions of that size, merged by log-sum-exp.
 *                 The choice goes by the number of requests and heads: a large
 *                 batch runs whole, so give a size (16384, say) where one of its
 *                 contexts is far longer than the rest
 *   workspace     at least pa_verify_tree_workspace_size(...) bytes (may be NULL
 *                 when that is 0)
 *   scale         positive (a normal fp32 number)
 * q_heads / kv_heads up to 16.  Rows of q past q_start[num_reqs] are left as
 * they were in out.  A q_start that decreases or passes total_q, n > max_q_len
 * or a context shorter than n records PA_DEVERR_QUERY_RANGE, a context past the
 * table PA_DEVERR_CONTEXT_LEN; the request is skipped.
 * pa_verify_tree_split_tokens: the partition size of such a call (negative: a
 * pa_status error).
 * ------------------------------------------------------------------------- */
int pa_verify_tree_split_tokens(int num_reqs, int max_q_len, int q_heads, int kv_heads, int max_blocks_per_seq,
                                int block_size, int split_tokens);

size_t pa_verify_tree_workspace_size(int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads,
                                     int head_dim, int max_blocks_per_seq, int block_size, int split_tokens);

int pa_verify_tree(const void* q, const int32_t* q_start, const uint64_t* tree_mask, const int32_t* context_lens,
                   const void* k_cache, const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                   int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads, int head_dim, int block_size,
                   int num_blocks, float scale, int split_tokens, void* workspace, size_t workspace_bytes, void* out,
                   pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_decode_accumulate - pa_decode that also adds up the attention each cached
 * token receives, the score by which pa_evict_select later chooses.
 *
 * out as pa_decode; and for every token t < context_lens[r] and KV head g
 *     scores_out[row][g][t] = scores[row][g][t] + sum over the query heads h of
 *                             group g of softmax(s_h)_t,   row = score_rows[r]
 * in fp32, each entry by one thread in a fixed order (repeatable bit for bit).
 * Entries of other rows and from context_lens[r] on are left as they were; a
 * token appended to a sequence must find zero there (a new sequence's row is
 * zeroed by the caller; pa_compact_kv leaves zeros behind what it keeps).
 * Only this call keeps score: queries of pa_chunked_prefill, pa_verify_decode and
 * pa_verify_tree add nothing, so right after a prompt every score is still what
 * the caller set, and a selection by them would keep the lowest tokens (equal
 * scores).  Decode some steps first, or set the scores of a prompt's tokens.
 * A logit that is NaN or +infinity makes its head's weights, and the scores of
 * all the request's tokens at its KV head, NaN: the softmax is.
 *   scores, scores_out  fp32 [num_rows][kv_heads][score_len]; the same array or
 *                 not overlapping; score_len >= max_blocks_per_seq * block_size
 *                 or at least every context (a longer one records
 *                 PA_DEVERR_CONTEXT_LEN, and its tokens from score_len on get no
 *                 score)
 *   score_rows    int32 [num_seqs], or NULL: row r.  A negative row: the request
 *                 keeps no score.  A row >= num_rows, or one that an earlier
 *                 request of the call has, records PA_DEVERR_SCORE_ROW and the
 *                 request keeps no score either.
 *   workspace     at least pa_decode_accumulate_workspace_size(...) bytes: the
 *                 partials, and the logits of the call: 4 bytes per request, KV
 *                 head, query head of its group (their number rounded up to 1, 2
 *                 or a multiple of 4) and token that the TABLE has room for; the
 *                 second pass has a block of threads for each stretch of it, too.
 *                 So cut the tables to the longest context: 64 requests of <= 4079
 *                 tokens, 32/8 heads, take 45 MB and 96 us then, 1.1 GB and 341 us
 *                 with tables for 131072
 *   split_tokens  as pa_decode; 0 = the library's choice for this call, which
 *                 also depends on num_seqs and kv_heads
 *                 (pa_decode_accumulate_split_tokens tells it)
 * Everything else as pa_decode, whose output it equals bit for bit at the same
 * partition size.
 * ------------------------------------------------------------------------- */
int pa_decode_accumulate_split_tokens(int num_seqs, int q_heads, int kv_heads, int max_blocks_per_seq, int block_size,
                                      int split_tokens);

size_t pa_decode_accumulate_workspace_size(int num_seqs, int q_heads, int kv_heads, int head_dim,
                                           int max_blocks_per_seq, int block_size, int split_tokens);

int pa_decode_accumulate(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                         int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads,
                         int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                         const float* scores, const int32_t* score_rows, int num_rows, int score_len,
                         float* scores_out, void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype,
                         pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_evict_select - which tokens a budget keeps, per request and KV head.
 *
 * With L = context_lens[r] and budget = sink + heavy + recent: all L tokens if
 * L <= budget; else the first `sink`, the last `recent`, and of those between
 * the `heavy` with the largest scores[row][g][t] (equal scores: the lower t
 * first; a NaN counts below every number), in ascending order of t.
 *   keep          int32 [num_seqs][kv_heads][budget]; entries from keep_lens[r]
 *                 on are -1
 *   keep_lens     int32 [num_seqs]: min(L, budget), 0 for a refused request
 *   scores, score_rows, num_rows, score_len as pa_decode_accumulate, but rows
 *                 may repeat; a row outside [0, num_rows) records
 *                 PA_DEVERR_SCORE_ROW, a context outside [0, score_len]
 *                 PA_DEVERR_CONTEXT_LEN, and the request keeps nothing
 * sink, heavy, recent >= 0, budget >= 1.  keep and keep_lens overlap neither one
 * another nor an input (new lengths are another array: PA_ERR_INVALID).
 * ------------------------------------------------------------------------- */
int pa_evict_select(const float* scores, const int32_t* score_rows, int num_rows, int kv_heads, int score_len,
                    const int32_t* context_lens, int num_seqs, int sink, int heavy, int recent, int32_t* keep,
                    int32_t* keep_lens, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_compact_kv - move the kept tokens of each sequence together, in place.
 *
 * For request r, KV head g and i < n = keep_lens[r], with b = base[r]:
 *     token b + i of the sequence becomes token b + keep[r][g][i]
 * (K and V, bit-exactly, and its score), all moves of a head as if at once.
 * After an eviction b = 0 and keep is pa_evict_select's, each head its own
 * list; after a tree's verify b = L - n_drafted and keep is the accepted path,
 * one list for all heads.  Then the sequence has b + n tokens
 * (pa_alloc_compact does the bookkeeping; block_tables are those of before it).
 *   keep          int32 [num_seqs][keep_heads][max_keep], keep_heads 1 (one list
 *                 for all heads) or kv_heads; i <= keep[i] < context_lens[r] - b
 *                 (any ascending list of tokens is)
 *   base          int32 [num_seqs], or NULL: 0
 *   scores        fp32 [num_rows][kv_heads][score_len] or NULL; entries
 *                 [b + n, context_lens[r]) of the row become 0.  score_rows as
 *                 pa_decode_accumulate.
 * The blocks of tokens [b, b + n) must be private to their sequence (copy
 * shared ones first: pa_alloc_cow, pa_copy_blocks).  An entry out of range
 * records PA_DEVERR_KEEP and is skipped (a count outside [0, max_keep], a base
 * outside [0, L] or base + count > L: the request), a bad block id
 * PA_DEVERR_BLOCK_ID, a context outside the table PA_DEVERR_CONTEXT_LEN.
 * ------------------------------------------------------------------------- */
int pa_compact_kv(void* k_cache, void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, const int32_t* keep, int keep_heads, int max_keep,
                  const int32_t* keep_lens, const int32_t* base, int num_seqs, int num_blocks, int block_size,
                  int kv_heads, int head_dim, pa_dtype dtype, float* scores, const int32_t* score_rows, int num_rows,
                  int score_len, pa_stream stream);

/* ============================================================================
 * A paged cache held in 4 bits.
 *
 * An element is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (e2m1), times the
 * scale of its 16 neighbours along the head: a byte with five exponent bits and
 * three of mantissa, bits 14..7 of the same number in fp16.  4.5 bits an
 * element, 0.28 of the 16-bit cache; every element is exact in fp16 and bf16.
 *
 * Layout: k_cache and v_cache are byte arrays [num_blocks][kv_heads][page], a
 * page (one block of one KV head) being block_size * head_dim * 9 / 16 bytes:
 * block_size rows of head_dim / 2 bytes of codes (byte i: element 2i in the low
 * four bits, 2i + 1 in the high; bit 3 of a code is its sign), then block_size
 * rows of head_dim / 16 scales.  Blocks, Block Tables, slots and context lengths
 * are those of the 16-bit cache; a block's bytes are contiguous, so
 * pa_copy_pages moves them.  dtype below is that of k, v, q and out.
 * ========================================================================== */

/* ----------------------------------------------------------------------------
 * pa_quantize_and_cache - pa_reshape_and_cache into a 4-bit cache.
 *
 * For each group of 16 elements x of a token's head
 *     s = the scale nearest to max|x| / 6 (ties to the even byte; at most 10240,
 *         2^-17 apart below 2^-14)
 *     element = the level nearest to x / s (ties to the even code), times s
 * both decided as by exact quotients.  Larger magnitudes than 61440 become
 * that; a group whose scale rounds to 0 becomes zeros; a group with an element
 * that is not finite is held as NaN (scale byte 0xFF).
 *   k, v          [num_tokens][kv_heads][head_dim] with k_stride / v_stride
 *                 elements between tokens (a multiple of 8, at least
 *                 kv_heads * head_dim), so that both may be views of one
 *                 projection's rows
 * Other arguments and errors as pa_reshape_and_cache.
 * ------------------------------------------------------------------------- */
int pa_quantize_and_cache(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slot_mapping,
                          int num_tokens, void* k_cache, void* v_cache, int num_blocks, int block_size, int kv_heads,
                          int head_dim, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_dequantize_kv4 - tokens of a 4-bit cache in 16 bits (exactly).
 *
 *   slots         int32 [num_tokens], repeats allowed; a negative slot gives
 *                 zeros, a slot past the pool zeros and PA_DEVERR_SLOT
 *   k, v          [num_tokens][kv_heads][head_dim]
 * ------------------------------------------------------------------------- */
int pa_dequantize_kv4(const void* k_cache, const void* v_cache, const int32_t* slots, int num_tokens, int num_blocks,
                      int block_size, int kv_heads, int head_dim, void* k, void* v, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_decode_kv4 - pa_decode (q_len 1) and pa_verify_decode (q_len causal queries
 * per request) over a 4-bit cache.
 *
 *   q, out        [num_seqs][q_len][q_heads][head_dim]; query i of request r sees
 *                 tokens [0, context_lens[r] - (q_len-1-i)); one that sees none
 *                 gives a zero row
 *   q_len         >= 1, with (q_heads / kv_heads) * q_len <= 32 and a group of at
 *                 most 16
 *   scale         finite, of either sign, as is scale / ln 2
 *   split_tokens  0, or a multiple of 32 no larger than 1024 * block_size;
 *                 pa_decode_kv4_split_tokens returns the partition size such a
 *                 call uses, or PA_ERR_INVALID
 *   workspace     at least pa_decode_kv4_workspace_size(...) bytes (NULL where
 *                 that is 0)
 * Sums and softmax are fp32; weights are rounded to fp16 for the P.V product
 * (relative error 2^-11), the cache's elements and q are not rounded.  A token
 * that a query does not see leaves it as it is, whatever the token holds (NaN
 * included).  A bad block id records PA_DEVERR_BLOCK_ID and reads as zeros.
 * ------------------------------------------------------------------------- */
int pa_decode_kv4_split_tokens(int num_seqs, int q_len, int q_heads, int kv_heads, int max_blocks_per_seq,
                               int block_size, int split_tokens);

size_t pa_decode_kv4_workspace_size(int num_seqs, int q_len, int q_heads, int kv_heads, int head_dim,
                                    int max_blocks_per_seq, int block_size, int split_tokens);

int pa_decode_kv4(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                  int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                  int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                  void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_chunked_prefill_kv4 - pa_chunked_prefill over a 4-bit cache.
 *
 * The chunk's K and V are written first (pa_quantize_and_cache); query i of
 * request r sees tokens [0, context_lens[r] - chunk + i].
 *   q, out        [total_q][q_heads][head_dim], packed by q_start
 *   q_start       int32 [num_reqs + 1], non-decreasing, q_start[num_reqs] <= total_q
 *   max_q_len     host-side upper bound of any chunk length (sizes the grid); 0
 *                 only in a batch without requests or queries, which is no work
 *   scale         a normal number, of either sign; scale / ln 2 is finite
 *   split_tokens  keys of a partition: 0, or a multiple of 64.  0 takes the
 *                 number of partitions that is the fastest by a count of rounds
 *                 (units of 256 (query, group head) rows of one (request, KV
 *                 head) over the SMs), by the width of block_tables: contexts may
 *                 be cut although there are more units than SMs.
 *                 pa_chunked_prefill_kv4_split_tokens tells it
 *   workspace     at least pa_chunked_prefill_kv4_workspace_size(...) bytes (NULL
 *                 where that is 0)
 * Rounding, and tokens that are not numbers, as pa_decode_kv4; refused requests
 * as pa_chunked_prefill (their rows of out, and rows behind the last chunk, stay
 * as they are).
 * ------------------------------------------------------------------------- */
int pa_chunked_prefill_kv4_split_tokens(int num_reqs, int max_q_len, int q_heads, int kv_heads, int max_blocks_per_seq,
                                        int block_size, int split_tokens);

size_t pa_chunked_prefill_kv4_workspace_size(int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads,
                                             int head_dim, int max_blocks_per_seq, int block_size, int split_tokens);

int pa_chunked_prefill_kv4(const void* q, const int32_t* q_start, const int32_t* context_lens, const void* k_cache,
                           const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq, int num_reqs,
                           int total_q, int max_q_len, int q_heads, int kv_heads, int head_dim, int block_size,
                           int num_blocks, float scale, int split_tokens, void* workspace, size_t workspace_bytes,
                           void* out, pa_dtype dtype, pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_fork_blocks - sequences that go on from others: tables, pages and slots of
 * a batch's next step, worked out on the device.
 *
 * A step of beam search, several samples of one prompt, a batch that sequences
 * leave and join: new row i goes on from row parents[i] of block_tables and
 * grows by grow[i] tokens, without a copy of what it has read so far and
 * without a trip to the host.  With L = context_lens[parents[i]] (0 for a new
 * sequence) and bs = block_size:
 *   - tables_out[i] holds the parent's ceil(L / bs) blocks, shared;
 *   - if it grows and L % bs != 0 it goes on inside its last block, which no one
 *     else may hold then: of the rows that go on inside one block the lowest
 *     keeps it, if every row of the new batch that holds the block is one of
 *     them and the block is not pinned; each other gets a fresh block there and
 *     pairs[i] = (old, fresh), a copy for pa_copy_pages to make before anything
 *     writes; otherwise pairs[i] = (-1, -1);
 *   - fresh blocks follow for the tokens up to L + grow[i]; -1 behind them;
 *   - lens_out[i] = L + grow[i], and slots[i][t] is the slot of token L + t for
 *     t < grow[i], -1 for the others of max_grow.
 * Fresh blocks are those that no row of the new batch shares and that are not
 * pinned, in ascending order, given out row by row (a copy's first).  So the
 * blocks of rows that nothing goes on from are free at once, and num_free
 * [1] says how many are left.  The tables are all that says who holds a block:
 * every sequence of the pool is in the batch, or its blocks are pinned.  Where
 * the blocks do not suffice PA_DEVERR_NO_BLOCKS is recorded and the new batch is
 * empty (tables, pairs and slots -1, lengths 0, num_free the free ones): nothing
 * is lost, since the old tables are as they were.
 *   parents       int32 [num_new]; -1: a new sequence; below: no sequence, an
 *                 empty row that neither holds nor grows
 *   grow          int32 [num_new], each in [0, max_grow]; NULL: max_grow for all
 *   pinned        uint8 [num_blocks], not 0: never handed out nor written; NULL:
 *                 none
 *   max_blocks_out  columns of tables_out
 *   workspace     at least pa_fork_blocks_workspace_size(...) bytes, 16-byte
 *                 aligned; needs no initialisation
 * Up to 65535 rows on either side.  Outputs and workspace overlap neither an
 * input nor one another.  A parent >= num_seqs or a growth out of range records
 * PA_DEVERR_FORK, a parent's length outside its table or a new one past
 * max_blocks_out PA_DEVERR_CONTEXT_LEN, and the row is as one without a
 * sequence.  A bad block id records PA_DEVERR_BLOCK_ID and stays in the table.
 * ------------------------------------------------------------------------- */
size_t pa_fork_blocks_workspace_size(int num_new, int num_blocks);

int pa_fork_blocks(const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                   const int32_t* parents, int num_new, const int32_t* grow, int max_grow, const uint8_t* pinned,
                   int num_blocks, int block_size, int32_t* tables_out, int max_blocks_out, int32_t* lens_out,
                   int32_t* pairs, int32_t* slots, int32_t* num_free, void* workspace, size_t workspace_bytes,
                   pa_stream stream);

/* ----------------------------------------------------------------------------
 * pa_copy_pages - block copies in any number of caches at once.
 *
 * In every cache c, block pairs[2p+1] becomes a bit-exact copy of block
 * pairs[2p]; a pair whose source is negative is none.
 *   caches        HOST array of num_caches device pointers, 16-byte aligned:
 *                 caches of any type whose blocks are block_bytes contiguous
 *                 bytes (a multiple of 16) - K and V of every layer, of 16 bits
 *                 or 4
 *   pairs         int32 [num_pairs][2], device memory, as pa_copy_blocks (pairs
 *                 of pa_fork_blocks as they are)
 * Ids outside [0, num_blocks) record PA_DEVERR_BLOCK_ID, the pair is skipped.
 * ------------------------------------------------------------------------- */
int pa_copy_pages(void* const* caches, int num_caches, const int32_t* pairs, int num_pairs, int num_blocks,
                  int64_t block_bytes, pa_stream stream);

/* Read and clear the calling device's error word.  Synchronises `stream`.
 * *host_code receives the PA_DEVERR_* code (0 = none).  Returns
 * PA_ERR_DEVICE_CHECK if a code was recorded, PA_OK otherwise. */
int pa_get_device_error(int32_t* host_code, pa_stream stream);

/* Self-test of the bounded waits: launches one thread that waits on a
 * shared-memory barrier phase nothing completes, with a limit of wait_ms
 * (1..2000) instead of the kernels' 2 s.  The wait gives up, records
 * PA_DEVERR_TIMEOUT in the error word and the kernel finishes normally, as
 * any kernel of the library does when one of its waits expires; the context
 * stays usable.  Asynchronous on `stream`; PA_ERR_INVALID for wait_ms out of
 * range. */
int pa_selftest_wait_timeout(int wait_ms, pa_stream stream);

/* ============================================================================
 * Host block allocator ("2.1 PagedAttention" §9.1-§9.3, §3, §6).
 *
 * A pool of num_blocks physical blocks with a reference count each and a free
 * queue kept as a doubly linked list (O(1) pop from the head, O(1) removal
 * from the middle).  Sequences own Block Tables that grow a block at a time,
 * only when the last block is full.  Tables may share blocks (refcount =
 * number of tables holding the block); a sequence about to write a shared
 * block copies it first (pa_alloc_cow).  Freeing a sequence releases its
 * blocks in reverse order; blocks whose count reaches zero go to the HEAD of
 * the free queue in that order, so a request's last block is reused first.
 * Freed blocks keep their contents (no clearing).
 *
 * Every call is all-or-nothing: on error the state is unchanged.  Handles are
 * single-threaded.  Sequence ids are any non-negative int.
 * ========================================================================== */
typedef struct pa_alloc pa_alloc;

typedef struct {
  int64_t num_blocks;
  int64_t num_free;
  int64_t num_used;        /* blocks with refcount > 0                        */
  int64_t num_shared;      /* blocks with refcount > 1                        */
  int64_t num_seqs;
  int64_t cow_copies;      /* pa_alloc_cow calls that produced a copy          */
  int64_t alloc_failures;  /* calls that returned PA_ERR_NO_FREE_BLOCKS        */
  int64_t waste_slots;     /* sum over sequences of unused slots in the last block */
} pa_alloc_stats;

/* initial_free_order: NULL for ascending ids, else a permutation of
 * 0..num_blocks-1 giving the initial free-queue order (head first). */
int pa_alloc_create(int num_blocks, int block_size, const int32_t* initial_free_order, pa_alloc** out);
void pa_alloc_destroy(pa_alloc* a);

int pa_alloc_add_seq(pa_alloc* a, int seq_id);

/* Give the next n_tokens tokens of seq_id their slots (slots_out[i] =
 * block*block_size + offset), taking new blocks from the head of the free
 * queue only as the last block fills.  PA_ERR_NO_FREE_BLOCKS if the pool
 * cannot cover them; PA_ERR_SHARED_BLOCK if the partially filled last block is
 * shared (call pa_alloc_cow first).  slots_out may be NULL. */
int pa_alloc_append_slots(pa_alloc* a, int seq_id, int n_tokens, int32_t* slots_out);

/* dst_seq (empty) starts with the first n_tokens tokens of src_seq: its table
 * points at src's first ceil(n_tokens/block_size) blocks, each refcount +1. */
int pa_alloc_share(pa_alloc* a, int dst_seq, int src_seq, int n_tokens);

/* Make seq_id's logical block private.  If its refcount is 1, src_dst_out =
 * {b, b} and nothing changes.  Otherwise a fresh block n is taken from the
 * free queue, the table entry becomes n, b's refcount drops by one, and
 * src_dst_out = {b, n}: the caller must then run pa_copy_blocks on (b, n). */
int pa_alloc_cow(pa_alloc* a, int seq_id, int logical_block, int32_t* src_dst_out);

int pa_alloc_free_seq(pa_alloc* a, int seq_id);

/* seq_id shrinks to its first n_tokens tokens, of which those from first_token
 * on are rewritten by a pa_compact_kv on the stream (first_token == n_tokens:
 * none, a plain truncation, as after rejected drafts).  Blocks behind the last
 * token are released as pa_alloc_free_seq does, so build the tables that
 * pa_compact_kv reads before this call and launch it before anything writes
 * the released blocks.  Blocks with rewritten tokens must be private
 * (PA_ERR_SHARED_BLOCK: pa_alloc_cow first) and leave the prefix cache, as does
 * a private block whose tail is cut off; the sequence registers nothing more
 * where its tokens are no longer known.  PA_ERR_INVALID unless
 * 0 <= first_token <= n_tokens <= its length, or while it is swapped out. */
int pa_alloc_compact(pa_alloc* a, int seq_id, int64_t first_token, int64_t n_tokens);

/* Copy seq_id's Block Table into out[0..cap); *n_out = its length.
 * PA_ERR_INVALID if cap is too small (nothing written). */
int pa_alloc_block_table(const pa_alloc* a, int seq_id, int32_t* out, int cap, int* n_out);

/* Fill a padded batch table: out is [n][max_blocks_per_seq], row i = table of
 * seq_ids[i] padded with -1; lens_out[i] = its token count (may be NULL). */
int pa_alloc_build_tables(const pa_alloc* a, const int* seq_ids, int n, int32_t* out,
                          int max_blocks_per_seq, int32_t* lens_out);

/* Number of leading FULL blocks that all of seq_ids[0..n) hold in common (same
 * physical ids, in order): the shared prefix pa_decode_shared_prefix can use. */
int pa_alloc_common_prefix(const pa_alloc* a, const int* seq_ids, int n, int* n_blocks_out);
int pa_alloc_seq_len(const pa_alloc* a, int seq_id, int64_t* n_tokens_out);
int pa_alloc_num_free(const pa_alloc* a);
/* Refcount of block_id, or PA_ERR_INVALID if it is out of range. */
int pa_alloc_ref(const pa_alloc* a, int block_id);
/* Free-queue snapshot head to tail into out[0..cap); returns the number
 * written, or PA_ERR_INVALID if cap < the queue length. */
int pa_alloc_free_list(const pa_alloc* a, int32_t* out, int cap);
int pa_alloc_get_stats(const pa_alloc* a, pa_alloc_stats* out);

/* ----------------------------------------------------------------------------
 * Automatic prefix caching ("Khám phá vLLM … phần 2", prefix caching;
 * "2.1 PagedAttention" §9.2-§9.3).  Off until pa_alloc_enable_prefix_caching.
 *
 * Only FULL blocks are cached.  Block i of a sequence has the chained hash
 * h_i = pa_block_hash(h_{i-1}, its block_size token ids), with the sequence's
 * salt as h_{-1}; the allocator keeps a map hash -> block.
 *  - pa_alloc_add_seq_cached: a new sequence whose table starts with the
 *    longest run of cached blocks matching its prompt's full blocks, looked up
 *    in order up to the first miss, at most floor((n_tokens-1)/block_size)
 *    blocks (at least one prompt token is left to compute).  Hit blocks get
 *    refcount +1 and, if they were free, leave the free queue.
 *    *n_cached_out = tokens covered (a multiple of block_size).
 *  - pa_alloc_append_tokens: pa_alloc_append_slots for tokens whose ids are
 *    known; each block they fill is registered (hash -> block) unless that
 *    hash is already cached.  After pa_alloc_append_slots (ids unknown) a
 *    sequence registers nothing more.
 *  - Freeing: blocks whose count reaches zero go to the HEAD of the free queue
 *    if they carry no hash (as above) and to the TAIL if they do, in release
 *    order, so cached blocks are evicted oldest-released first and a
 *    request's first block last.
 *  - A cached block loses its hash, and the map its entry, when the free queue
 *    hands it out again (new block, CoW copy), when pa_alloc_compact rewrites
 *    it, and when the one sequence that holds it, in part (shared or cut inside
 *    it), appends to it.
 *  - pa_alloc_share continues the hash chain into dst only when the shared
 *    part ends on a full, hashed block.
 * ------------------------------------------------------------------------- */
typedef struct {
  int64_t lookup_blocks;  /* prompt blocks looked up by pa_alloc_add_seq_cached */
  int64_t hit_blocks;     /* ... of which were found                          */
  int64_t evictions;      /* cached blocks handed out again (hash dropped)     */
  int64_t cached_blocks;  /* entries in the hash map now                       */
} pa_prefix_cache_stats;

/* 64-bit FNV-1a over parent (8 bytes, little-endian) followed by the n token
 * ids (4 bytes each, little-endian, two's complement). */
uint64_t pa_block_hash(uint64_t parent, const int32_t* tokens, int n);
int pa_alloc_enable_prefix_caching(pa_alloc* a);
/* seq_id must be new; tokens may be NULL when n_tokens == 0; n_cached_out may
 * be NULL.  With caching off this is pa_alloc_add_seq and *n_cached_out = 0. */
int pa_alloc_add_seq_cached(pa_alloc* a, int seq_id, const int32_t* tokens, int n_tokens, uint64_t salt,
                            int* n_cached_out);
/* Errors as pa_alloc_append_slots; tokens may be NULL when n_tokens == 0. */
int pa_alloc_append_tokens(pa_alloc* a, int seq_id, const int32_t* tokens, int n_tokens, int32_t* slots_out);
/* *is_cached_out = 1 and *hash_out = its hash if block_id is in the map, else 0. */
int pa_alloc_block_hash(const pa_alloc* a, int block_id, uint64_t* hash_out, int* is_cached_out);
int pa_alloc_get_prefix_cache_stats(const pa_alloc* a, pa_prefix_cache_stats* out);

/* ----------------------------------------------------------------------------
 * Preemption by swapping ("2.1 PagedAttention" §7).  Off until
 * pa_alloc_enable_swap gives the size of the CPU swap pool (its own free
 * queue of ids 0..num_cpu_blocks-1, handed out from the head).
 *  - pa_alloc_swap_out: the sequence's table moves to swap blocks taken from
 *    the swap pool's head, one per GPU block in logical order; its GPU blocks
 *    are released exactly as pa_alloc_free_seq releases them (a block another
 *    sequence shares stays with that sequence; a cached block keeps its
 *    hash).  pairs_out[i] = (gpu block, swap block) for logical block i: run
 *    pa_swap_blocks(gpu pool -> swap pool) on them BEFORE anything writes the
 *    released GPU blocks.
 *  - pa_alloc_swap_in: the sequence gets new GPU blocks from the free queue
 *    (as appends do); pairs_out[i] = (swap block, gpu block); its swap blocks
 *    return to the swap pool's head, its last block first.  Run
 *    pa_swap_blocks(swap pool -> gpu pool) before the sequence is read.
 *  - While swapped out a sequence can only be swapped in, freed (its swap
 *    blocks return to the swap pool's head) or queried; append, share, CoW,
 *    table building and common-prefix calls on it return PA_ERR_INVALID.
 *    Its block table then lists swap-pool ids.
 * cap is the capacity of pairs_out in pairs; *n_out (may be NULL) = the number
 * of pairs needed, also when cap is too small (PA_ERR_INVALID).  A shortage of
 * swap blocks (swap_out) or GPU blocks (swap_in) returns PA_ERR_NO_FREE_BLOCKS
 * and changes nothing.
 * ------------------------------------------------------------------------- */
int pa_alloc_enable_swap(pa_alloc* a, int num_cpu_blocks);

/* ----------------------------------------------------------------------------
 * Checkpoint and resume of the host allocator: its whole state (free queue
 * order, refcounts, every sequence's Block Table, token count and hashing
 * state, the prefix cache, the swap pool and the counters) as a flat list of
 * int64 words.
 *
 * pa_alloc_export writes the words to out[0..cap) and their number to
 * *n_out; with out = NULL and cap = 0 it only reports the number.  Returns
 * PA_ERR_INVALID if cap is smaller than needed (nothing is written then).
 * Equal states give equal words (sequences and cached hashes are written in
 * key order).
 *
 * pa_alloc_import builds a new allocator (owned by the caller, freed with
 * pa_alloc_destroy) from such words.  It validates every count, id and range
 * and the state's consistency (refcounts equal the tables holding each block,
 * the free queue holds exactly the unheld blocks, the cache holds exactly
 * the hashed blocks under their hashes); malformed words give PA_ERR_INVALID
 * and no allocator.  An imported
 * allocator behaves as the exported one for every later call.
 *
 * Layout (version 1): magic 0x504b5641, version, num_blocks, block_size,
 * caching, num_cpu_blocks, cow_copies, alloc_failures, lookup_blocks,
 * hit_blocks, evictions; n_free and the free queue head to tail; ref[],
 * has_hash[] and hash[] of every block; n_cached and (hash, block) pairs;
 * n_cpu_free and the swap pool's free queue; n_seqs and per sequence (by id):
 * id, num_tokens, salt, parent hash, hashable, swapped, n_blocks, blocks,
 * n_pending, pending token ids.
 * ------------------------------------------------------------------------- */
int pa_alloc_export(const pa_alloc* a, int64_t* out, int64_t cap, int64_t* n_out);
int pa_alloc_import(const int64_t* words, int64_t n, pa_alloc** out);
int pa_alloc_num_free_cpu(const pa_alloc* a);
/* 1 if seq_id is swapped out, 0 if resident, PA_ERR_INVALID if unknown. */
int pa_alloc_is_swapped(const pa_alloc* a, int seq_id);
int pa_alloc_swap_out(pa_alloc* a, int seq_id, int32_t* pairs_out, int cap, int* n_out);
int pa_alloc_swap_in(pa_alloc* a, int seq_id, int32_t* pairs_out, int cap, int* n_out);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
