// C ABI of the paged-KV library: argument checks, TMA descriptor cache,
// per-device error word, and the launches (see include/pa.h for the contract).
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <cstring>
#include <mutex>

#include "pa_internal.h"

namespace pa {

namespace {

std::atomic<uint64_t> g_launches{0};

// Per-device error word: kernels record the first data error here.
__device__ int g_device_error;

constexpr int kMaxDevices = 64;
// Automatic partition size: shorter partitions balance the grid better,
// longer ones write fewer partials for the merge.  Measured on GB300: 384 tokens
// is best for contexts up to 8K (batch-64 Llama-8B-style decode), 512 beyond
// (128K-token contexts, where 256 doubles the merge traffic).
constexpr int kAutoSplitShort = 384;
constexpr int kAutoSplitLong = 512;
constexpr int64_t kShortContext = 8192;
// Verify (q_len > 1): each partition writes q_len x the partials of decode and
// the merge has q_len x the rows, so longer partitions pay off.  Measured on
// GB300 (batch 64, contexts 512..4096, k = 3 / 7 drafts, step time in us):
// 256: 108.6 / 143.6, 384: 103.6 / 135.9, 512: 111.4 / 130.7,
// 768: 100.8 / 128.6, 1024: 100.6 / 152.7, 2048: 153.1 / 157.5.
constexpr int kAutoSplitVerify = 768;

std::mutex g_mu;
int* g_err_ptr[kMaxDevices] = {};
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

int current_device() {
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess) return -1;
  return d;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return nullptr;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  return g_encode;
}

// Small cache of KV tensor maps keyed by (pointer, shape, dtype, device).
struct MapKey {
  const void* ptr;
  int64_t rows;
  int kv_heads, head_dim, bsub, dtype, dev;
  bool operator==(const MapKey& o) const {
    return ptr == o.ptr && rows == o.rows && kv_heads == o.kv_heads && head_dim == o.head_dim &&
           bsub == o.bsub && dtype == o.dtype && dev == o.dev;
  }
};
struct MapEntry {
  MapKey key;
  CUtensorMap map;
  uint64_t stamp;
  bool used;
};
constexpr int kMapCache = 32;
MapEntry g_maps[kMapCache];
uint64_t g_stamp = 0;

// 4-D view of a cache tensor: {64, head_dim/64, kv_heads, num_blocks*block_size}
// elements, boxes {64, 1, 1, bsub}, 128-byte swizzle.
bool kv_map(const void* base, int num_blocks, int block_size, int kv_heads, int head_dim, pa_dtype dt,
            CUtensorMap* out) {
  const int bsub = block_size < 16 ? block_size : 16;
  const int64_t rows = (int64_t)num_blocks * block_size;
  MapKey key{base, rows, kv_heads, head_dim, bsub, (int)dt, current_device()};
  {
    std::lock_guard<std::mutex> lk(g_mu);
    for (auto& e : g_maps)
      if (e.used && e.key == key) {
        e.stamp = ++g_stamp;
        *out = e.map;
        return true;
      }
  }
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)(head_dim / 64), (cuuint64_t)kv_heads, (cuuint64_t)rows};
  cuuint64_t strides[3] = {128, (cuuint64_t)head_dim * 2, (cuuint64_t)kv_heads * head_dim * 2};
  cuuint32_t box[4] = {64, 1, 1, (cuuint32_t)bsub};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUtensorMap m;
  CUresult rc = enc(&m, dt == PA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                    const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (rc != CUDA_SUCCESS) return false;
  std::lock_guard<std::mutex> lk(g_mu);
  MapEntry* victim = &g_maps[0];
  for (auto& e : g_maps) {
    if (!e.used) {
      victim = &e;
      break;
    }
    if (e.stamp < victim->stamp) victim = &e;
  }
  victim->key = key;
  victim->map = m;
  victim->stamp = ++g_stamp;
  victim->used = true;
  *out = m;
  return true;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Do two arrays of an and bn elements of 4 bytes share any?
bool overlap4(const void* a, int64_t an, const void* b, int64_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < 4 * (uintptr_t)an : x - y < 4 * (uintptr_t)bn;
}

int check_kv_shape(int num_blocks, int block_size, int kv_heads, int head_dim, pa_dtype dt) {
  if (dt != PA_FP16 && dt != PA_BF16) return PA_ERR_DTYPE;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_INVALID;
  if (block_size != 4 && block_size != 8 && block_size != 16 && block_size != 32) return PA_ERR_INVALID;
  if (kv_heads <= 0 || kv_heads > 1024 || num_blocks <= 0) return PA_ERR_INVALID;
  // row coordinates (one past the pool included) must fit the TMA's int32
  if (((int64_t)num_blocks + 1) * block_size > INT32_MAX) return PA_ERR_INVALID;
  return PA_OK;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

// The address a kernel dereferences for p: device or managed memory as is,
// page-locked host memory through its mapped device address; nullptr for
// pageable host memory (or anything CUDA does not know).
const void* device_view(const void* p) {
  cudaPointerAttributes at{};
  if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  switch (at.type) {
    case cudaMemoryTypeDevice:
    case cudaMemoryTypeManaged:
      return p;
    case cudaMemoryTypeHost:
      return at.devicePointer;
    default:
      return nullptr;
  }
}

struct DecodeSetup {
  int split, max_splits;
  DecodeWorkspace ws;
};

int decode_setup(int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq, int block_size, int split_tokens,
                 DecodeSetup* s) {
  const int split = pa_decode_split_tokens(max_blocks_per_seq, block_size, split_tokens);
  if (split <= 0) return PA_ERR_INVALID;
  const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
  if (cap > INT32_MAX) return PA_ERR_INVALID;
  s->split = split;
  s->max_splits = (int)((cap + split - 1) / split);
  if (s->max_splits < 1) s->max_splits = 1;
  s->ws = s->max_splits > 1 ? decode_workspace_layout(num_seqs, q_heads, head_dim, s->max_splits)
                            : DecodeWorkspace{0, 0, 0, 0};
  return PA_OK;
}

// Shared-prefix decode: the prefix is cut into key ranges of kPrefixKeySplit
// (one partial slot each), the suffix into decode partitions after them.  The
// workspace is laid out for this split; a concurrent prefix pass uses longer
// ranges (fewer slots) in the same layout.
constexpr int kPrefixKeySplit = 512;

int sm_count() {
  static int cached[kMaxDevices] = {};
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return 0;
  if (!cached[d]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d) != cudaSuccess) return 0;
    cached[d] = n;
  }
  return cached[d];
}

// Key range of a prefix pass that runs beside the suffix pass: 512 x 2^k
// tokens, the smallest whose units (pairs of 128-row tiles x KV heads x
// ranges) fit in a quarter of the SMs: the suffix pass is bound by the bytes
// each SM keeps in flight, so the SMs it keeps matter more than how soon the
// prefix pass ends.  Measured on GB300 (256 requests, 2048-token prefix, 32/8
// heads), shared-prefix call: 512-token ranges (128 CTAs) 73.1 us, 1024 (64
// CTAs) 65.5 us, 2048 (32 CTAs) 62.0 us.
int concurrent_key_split(int num_seqs, int group, int kv_heads, int prefix_len) {
  const int64_t row_pairs = ((int64_t)num_seqs * group + 255) / 256;
  const int64_t quarter = sm_count() / 4;
  int ks = kPrefixKeySplit;
  while (ks < prefix_len && row_pairs * kv_heads * ((prefix_len + ks - 1) / ks) > quarter) ks *= 2;
  return ks;
}

// One event per device marks the end of a concurrent prefix pass.
cudaEvent_t prefix_done_event() {
  static cudaEvent_t ev[kMaxDevices] = {};
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!ev[d] && cudaEventCreateWithFlags(&ev[d], cudaEventDisableTiming) != cudaSuccess) return nullptr;
  return ev[d];
}

constexpr int kSuffixSplitMin = 128;  // a multiple of every supported block size

struct SharedPrefixSetup {
  int split, prefix_splits, suffix_splits, max_splits;
  DecodeWorkspace ws;
};

int shared_prefix_setup(int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq, int block_size,
                        int prefix_len, int split_tokens, SharedPrefixSetup* s) {
  if (num_seqs < 0 || q_heads <= 0 || head_dim <= 0) return PA_ERR_INVALID;
  int split = pa_decode_split_tokens(max_blocks_per_seq, block_size, split_tokens);
  if (split <= 0) return PA_ERR_INVALID;
  const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
  if (cap > INT32_MAX || prefix_len <= 0 || prefix_len > cap || prefix_len % block_size != 0) return PA_ERR_INVALID;
  if (split_tokens == 0) {
    // automatic: suffixes are short next to the contexts the decode default
    // is tuned for, so cut them into partitions of about a quarter of their
    // bound (at least kSuffixSplitMin tokens) for more CTAs per KV byte.
    // Measured on GB300 (256 requests, suffixes of 16..512 tokens): 128-token
    // partitions 80.9 us per step, 256: 82.2 us, 384: 84.2 us.
    const int64_t quarter = ((cap - prefix_len) / 4 + block_size - 1) / block_size * block_size;
    const int64_t want = quarter < kSuffixSplitMin ? kSuffixSplitMin : quarter;
    if (want < split) split = (int)want;
  }
  s->split = split;
  s->prefix_splits = (prefix_len + kPrefixKeySplit - 1) / kPrefixKeySplit;
  const int64_t suffix = cap - prefix_len;
  s->suffix_splits = (int)((suffix + split - 1) / split);
  if (s->suffix_splits < 1) s->suffix_splits = 1;
  s->max_splits = s->prefix_splits + s->suffix_splits;
  s->ws = decode_workspace_layout(num_seqs, q_heads, head_dim, s->max_splits);
  return PA_OK;
}

}  // namespace

void note_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

int num_sms() { return sm_count(); }

// Device address of the error word on the current device (set up once).
int* device_error_ptr() {
  const int d = current_device();
  if (d < 0 || d >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_err_ptr[d]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) != cudaSuccess) return nullptr;
    g_err_ptr[d] = static_cast<int*>(p);
  }
  return g_err_ptr[d];
}

}  // namespace pa

using namespace pa;

extern "C" {

const char* pa_status_string(int status) {
  switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_INVALID: return "PA_ERR_INVALID";
    case PA_ERR_NO_FREE_BLOCKS: return "PA_ERR_NO_FREE_BLOCKS";
    case PA_ERR_DTYPE: return "PA_ERR_DTYPE";
    case PA_ERR_CUDA: return "PA_ERR_CUDA";
    case PA_ERR_DEVICE_CHECK: return "PA_ERR_DEVICE_CHECK";
    case PA_ERR_SHARED_BLOCK: return "PA_ERR_SHARED_BLOCK";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
    case PA_ERR_HOST_MEMORY: return "PA_ERR_HOST_MEMORY";
    default: return "PA_UNKNOWN_STATUS";
  }
}

int pa_version(void) { return 100; }

uint64_t pa_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

int pa_reshape_and_cache(const void* k, const void* v, const int32_t* slot_mapping, int num_tokens, void* k_cache,
                         void* v_cache, int num_blocks, int block_size, int kv_heads, int head_dim, pa_dtype dtype,
                         pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  return cuda_status(launch_reshape_and_cache(k, v, slot_mapping, num_tokens, k_cache, v_cache,
                                              (int64_t)num_blocks * block_size, kv_heads * head_dim * 2, err,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

int pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int num_pairs, int num_blocks, int block_size,
                   int kv_heads, int head_dim, pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_pairs < 0) return PA_ERR_INVALID;
  if (num_pairs == 0) return PA_OK;
  if (!k_cache || !v_cache || !pairs || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  return cuda_status(launch_copy_blocks(k_cache, v_cache, pairs, num_pairs, num_blocks,
                                        (int64_t)block_size * kv_heads * head_dim * 2, err,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int pa_swap_blocks(const void* src_k, const void* src_v, void* dst_k, void* dst_v, const int32_t* pairs,
                   int num_pairs, int num_src_blocks, int num_dst_blocks, int block_size, int kv_heads, int head_dim,
                   pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_src_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  st = check_kv_shape(num_dst_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_pairs < 0) return PA_ERR_INVALID;
  if (num_pairs == 0) return PA_OK;
  if (!src_k || !src_v || !dst_k || !dst_v || !pairs) return PA_ERR_INVALID;
  if (!aligned16(src_k) || !aligned16(src_v) || !aligned16(dst_k) || !aligned16(dst_v)) return PA_ERR_INVALID;
  const void* sk = device_view(src_k);
  const void* sv = device_view(src_v);
  void* dk = const_cast<void*>(device_view(dst_k));
  void* dv = const_cast<void*>(device_view(dst_v));
  const int32_t* pr = static_cast<const int32_t*>(device_view(pairs));
  if (!sk || !sv || !dk || !dv || !pr) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  return cuda_status(launch_swap_blocks(sk, sv, dk, dv, pr, num_pairs, num_src_blocks, num_dst_blocks,
                                        (int64_t)block_size * kv_heads * head_dim * 2, err,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int pa_decode_split_tokens(int max_blocks_per_seq, int block_size, int split_tokens) {
  if (max_blocks_per_seq <= 0 || block_size <= 0) return PA_ERR_INVALID;
  const int unit = block_size > 16 ? block_size : 16;
  const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
  int s = split_tokens != 0 ? split_tokens : (cap <= kShortContext ? kAutoSplitShort : kAutoSplitLong);
  if (s <= 0 || s % unit != 0 || s > 256 * block_size) return PA_ERR_INVALID;
  return s;
}

size_t pa_decode_workspace_size(int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq, int block_size,
                                int split_tokens) {
  if (num_seqs < 0 || q_heads <= 0 || head_dim <= 0) return 0;
  DecodeSetup s;
  if (decode_setup(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s) != PA_OK) return 0;
  return s.ws.bytes;
}

namespace {

// The partition pass of decode (q_len = 1) and of the speculative verify
// (q_len = k+1 queries per request, rows r*q_len + i).
int decode_partial_impl(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                        int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                        void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || q_heads <= 0 || q_heads % kv_heads != 0 || q_heads / kv_heads > 16)
    return PA_ERR_INVALID;
  if (q_len < 1 || (q_heads / kv_heads) * q_len > 32) return PA_ERR_INVALID;
  if (max_blocks_per_seq <= 0 || !std::isfinite(scale)) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  DecodeSetup s;
  st = decode_setup(num_seqs * q_len, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s);
  if (st != PA_OK) return st;
  if (s.ws.bytes > 0 && (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  if ((int64_t)s.max_splits * kv_heads > (int64_t)INT32_MAX) return PA_ERR_INVALID;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  DecodeParams p{};
  p.q = q;
  p.tables = block_tables;
  p.lens = context_lens;
  p.out = out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = s.ws.bytes ? reinterpret_cast<float*>(ws + s.ws.o_off) : nullptr;
  p.part_m = s.ws.bytes ? reinterpret_cast<float*>(ws + s.ws.m_off) : nullptr;
  p.part_l = s.ws.bytes ? reinterpret_cast<float*>(ws + s.ws.l_off) : nullptr;
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.split_tokens = s.split;
  p.max_splits = s.max_splits;
  p.grid_splits = s.max_splits;
  p.tab_entries = s.split / block_size;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q_len = q_len;
  const int bsub = block_size < 16 ? block_size : 16;
  return cuda_status(
      launch_decode_partial(km, vm, p, head_dim, bsub, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int lse_merge_impl(const void* workspace, size_t workspace_bytes, const int32_t* context_lens, int num_seqs,
                   int q_len, int q_heads, int head_dim, int max_blocks_per_seq, int block_size, int split_tokens,
                   void* out, pa_dtype dtype, pa_stream stream) {
  if (dtype != PA_FP16 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_INVALID;
  if (num_seqs < 0 || q_heads <= 0 || q_len < 1) return PA_ERR_INVALID;
  // the merge kernels number their (request, query, head) rows in int32
  if ((int64_t)num_seqs * q_len * q_heads > (int64_t)INT32_MAX - 8) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  DecodeSetup s;
  int st = decode_setup(num_seqs * q_len, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s);
  if (st != PA_OK) return st;
  if (s.ws.bytes == 0) return PA_OK;  // a single partition: pa_decode_partial wrote `out`
  if (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)) return PA_ERR_WORKSPACE;
  if (!context_lens || !out || !aligned16(out)) return PA_ERR_INVALID;
  const uint8_t* ws = static_cast<const uint8_t*>(workspace);
  MergeParams p{};
  p.part_o = reinterpret_cast<const float*>(ws + s.ws.o_off);
  p.part_m = reinterpret_cast<const float*>(ws + s.ws.m_off);
  p.part_l = reinterpret_cast<const float*>(ws + s.ws.l_off);
  p.lens = context_lens;
  p.out = out;
  p.num_seqs = num_seqs;
  p.q_heads = q_heads;
  p.max_splits = s.max_splits;
  p.split_tokens = s.split;
  p.cap = max_blocks_per_seq * block_size;
  p.q_len = q_len;
  return cuda_status(launch_lse_merge(p, head_dim, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

int pa_decode_partial(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads,
                      int head_dim, int block_size, int num_blocks, float scale, int split_tokens, void* workspace,
                      size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream) {
  return decode_partial_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, 1,
                             q_heads, kv_heads, head_dim, block_size, num_blocks, scale, split_tokens, workspace,
                             workspace_bytes, out, dtype, stream);
}

int pa_lse_merge(const void* workspace, size_t workspace_bytes, const int32_t* context_lens, int num_seqs,
                 int q_heads, int head_dim, int max_blocks_per_seq, int block_size, int split_tokens, void* out,
                 pa_dtype dtype, pa_stream stream) {
  return lse_merge_impl(workspace, workspace_bytes, context_lens, num_seqs, 1, q_heads, head_dim,
                        max_blocks_per_seq, block_size, split_tokens, out, dtype, stream);
}

int pa_decode_contiguous(const void* q, const void* k_cache, const void* v_cache, int num_slots, int max_len,
                         const int32_t* slot_ids, const int32_t* slot_tokens, const int32_t* context_lens,
                         int num_seqs, int q_heads, int kv_heads, int head_dim, float scale, int split_tokens,
                         void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream) {
  if (num_slots <= 0 || max_len <= 0 || max_len % 16 != 0 || (int64_t)num_slots * max_len > INT32_MAX - 16)
    return PA_ERR_INVALID;
  const int maxblk = max_len / 16;
  int st = check_kv_shape(num_slots * maxblk, 16, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || q_heads <= 0 || q_heads % kv_heads != 0 || q_heads / kv_heads > 16)
    return PA_ERR_INVALID;
  if (!std::isfinite(scale)) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !context_lens || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  DecodeSetup s;
  st = decode_setup(num_seqs, q_heads, head_dim, maxblk, 16, split_tokens, &s);
  if (st != PA_OK) return st;
  if (s.ws.bytes > 0 && (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_slots * maxblk, 16, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_slots * maxblk, 16, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  DecodeParams p{};
  p.q = q;
  p.lens = context_lens;
  p.out = out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = s.ws.bytes ? reinterpret_cast<float*>(ws + s.ws.o_off) : nullptr;
  p.part_m = s.ws.bytes ? reinterpret_cast<float*>(ws + s.ws.m_off) : nullptr;
  p.part_l = s.ws.bytes ? reinterpret_cast<float*>(ws + s.ws.l_off) : nullptr;
  p.err = err;
  p.maxblk = maxblk;
  p.num_seqs = num_seqs;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_slots * maxblk;
  p.block_size = 16;
  p.split_tokens = s.split;
  p.max_splits = s.max_splits;
  p.grid_splits = s.max_splits;
  p.tab_entries = 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q_len = 1;
  p.slot_ids = slot_ids;
  p.slot_tokens = slot_tokens;
  p.num_slots = num_slots;
  p.contig_len = max_len;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  st = cuda_status(launch_decode_contig(km, vm, p, head_dim, dtype, cs));
  if (st != PA_OK) return st;
  return lse_merge_impl(workspace, workspace_bytes, context_lens, num_seqs, 1, q_heads, head_dim, maxblk, 16,
                        split_tokens, out, dtype, stream);
}

int pa_reshape_and_cache_slots(const void* k, const void* v, const int32_t* slot_ids, const int32_t* positions,
                               int num_tokens, void* k_cache, void* v_cache, int num_slots, int max_len,
                               const int32_t* slot_tokens, int kv_heads, int head_dim, pa_dtype dtype,
                               pa_stream stream) {
  if (num_slots <= 0 || max_len <= 0 || max_len % 16 != 0 || (int64_t)num_slots * max_len > INT32_MAX - 16)
    return PA_ERR_INVALID;
  int st = check_kv_shape(num_slots * (max_len / 16), 16, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !slot_ids || !positions || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  return cuda_status(launch_reshape_and_cache_slots(k, v, slot_ids, positions, num_tokens, k_cache, v_cache,
                                                    num_slots, max_len, slot_tokens, kv_heads * head_dim * 2, err,
                                                    reinterpret_cast<cudaStream_t>(stream)));
}

int pa_verify_split_tokens(int max_blocks_per_seq, int block_size, int q_len, int split_tokens) {
  if (q_len < 1) return PA_ERR_INVALID;
  if (split_tokens == 0 && q_len > 1 && max_blocks_per_seq > 0 && block_size > 0 &&
      (int64_t)max_blocks_per_seq * block_size <= kShortContext)
    split_tokens = kAutoSplitVerify;
  return pa_decode_split_tokens(max_blocks_per_seq, block_size, split_tokens);
}

size_t pa_verify_workspace_size(int num_seqs, int q_len, int q_heads, int head_dim, int max_blocks_per_seq,
                                int block_size, int split_tokens) {
  if (num_seqs < 0 || q_len < 1 || q_heads <= 0 || head_dim <= 0) return 0;
  if ((int64_t)num_seqs * q_len > INT32_MAX) return 0;
  split_tokens = pa_verify_split_tokens(max_blocks_per_seq, block_size, q_len, split_tokens);
  if (split_tokens < 0) return 0;
  DecodeSetup s;
  if (decode_setup(num_seqs * q_len, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s) != PA_OK)
    return 0;
  return s.ws.bytes;
}

int pa_verify_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                     int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                     void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream) {
  if (q_len < 1 || (int64_t)num_seqs * q_len > INT32_MAX / 64) return PA_ERR_INVALID;
  split_tokens = pa_verify_split_tokens(max_blocks_per_seq, block_size, q_len, split_tokens);
  if (split_tokens < 0) return split_tokens;
  int st = decode_partial_impl(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, q_len,
                               q_heads, kv_heads, head_dim, block_size, num_blocks, scale, split_tokens, workspace,
                               workspace_bytes, out, dtype, stream);
  if (st != PA_OK) return st;
  return lse_merge_impl(workspace, workspace_bytes, context_lens, num_seqs, q_len, q_heads, head_dim,
                        max_blocks_per_seq, block_size, split_tokens, out, dtype, stream);
}

int pa_decode(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
              int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads,
              int head_dim, int block_size, int num_blocks, float scale, int split_tokens, void* workspace,
              size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream) {
  int st = pa_decode_partial(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, q_heads,
                             kv_heads, head_dim, block_size, num_blocks, scale, split_tokens, workspace,
                             workspace_bytes, out, dtype, stream);
  if (st != PA_OK) return st;
  return pa_lse_merge(workspace, workspace_bytes, context_lens, num_seqs, q_heads, head_dim, max_blocks_per_seq,
                      block_size, split_tokens, out, dtype, stream);
}

int pa_chunked_prefill(const void* q, const int32_t* q_start, const int32_t* context_lens, const void* k_cache,
                       const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq, int num_reqs,
                       int total_q, int max_q_len, int max_ctas, int q_heads, int kv_heads, int head_dim,
                       int block_size, int num_blocks, float scale, void* out, pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_reqs < 0 || num_reqs > 65535 || total_q < 0 || max_q_len < 0 || q_heads <= 0 ||
      q_heads % kv_heads != 0 || kv_heads > 65535 || max_blocks_per_seq <= 0 || !std::isfinite(scale))
    return PA_ERR_INVALID;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PA_ERR_INVALID;
  if (num_reqs == 0 || max_q_len == 0 || total_q == 0) return PA_OK;
  if ((int64_t)max_q_len * (q_heads / kv_heads) > (int64_t)INT32_MAX / 2) return PA_ERR_INVALID;
  if (!q || !q_start || !context_lens || !k_cache || !v_cache || !block_tables || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  PrefillParams p{};
  p.q = q;
  p.q_start = q_start;
  p.lens = context_lens;
  p.tables = block_tables;
  p.out = out;
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.num_reqs = num_reqs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = 1;
  p.max_ctas = max_ctas;
  const int bsub = block_size < 16 ? block_size : 16;
  cudaStream_t st_ = reinterpret_cast<cudaStream_t>(stream);
  // blocks of >= 8 tokens: 5th-generation tensor cores (tcgen05 + TMEM);
  // 4-token blocks: warp-level MMA kernel
  if (bsub >= 8) return cuda_status(launch_attn_tc(km, vm, p, head_dim, bsub, dtype, st_));
  return cuda_status(launch_chunked_prefill(km, vm, p, head_dim, bsub, dtype, st_));
}

int pa_verify_decode_tc(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                        int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                        int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int max_ctas,
                        void* out, pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (block_size < 8 || num_seqs < 0 || num_seqs > 65535 || q_len < 1 || q_heads <= 0 || q_heads % kv_heads != 0 ||
      (q_heads / kv_heads) * q_len > 128 || max_blocks_per_seq <= 0 || !std::isfinite(scale))
    return PA_ERR_INVALID;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  PrefillParams p{};
  p.q = q;
  p.lens = context_lens;
  p.tables = block_tables;
  p.out = out;
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.num_reqs = num_seqs;
  p.total_q = num_seqs * q_len;
  p.max_q_len = q_len;
  p.fixed_q_len = q_len;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.causal = 1;
  p.max_ctas = max_ctas;
  return cuda_status(launch_attn_tile(km, vm, p, head_dim, block_size < 16 ? block_size : 16, dtype,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

size_t pa_decode_shared_prefix_workspace_size(int num_seqs, int q_heads, int head_dim, int max_blocks_per_seq,
                                              int block_size, int prefix_len, int split_tokens) {
  if (block_size < 8)  // 4-token blocks: plain pa_decode is used
    return pa_decode_workspace_size(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, split_tokens);
  SharedPrefixSetup s;
  if (shared_prefix_setup(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, prefix_len, split_tokens,
                          &s) != PA_OK)
    return 0;
  return s.ws.bytes;
}

int pa_decode_shared_prefix_split_tokens(int max_blocks_per_seq, int block_size, int prefix_len, int split_tokens) {
  if (block_size < 8) return pa_decode_split_tokens(max_blocks_per_seq, block_size, split_tokens);
  SharedPrefixSetup s;
  const int st = shared_prefix_setup(1, 1, 64, max_blocks_per_seq, block_size, prefix_len, split_tokens, &s);
  return st != PA_OK ? st : s.split;
}

int pa_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache, const int32_t* prefix_blocks,
                            int prefix_len, const int32_t* block_tables, int max_blocks_per_seq,
                            const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads, int head_dim,
                            int block_size, int num_blocks, float scale, int split_tokens, void* workspace,
                            size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream,
                            pa_stream prefix_stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || q_heads <= 0 || q_heads % kv_heads != 0 || q_heads / kv_heads > 16)
    return PA_ERR_INVALID;
  if (max_blocks_per_seq <= 0 || !std::isfinite(scale)) return PA_ERR_INVALID;
  if (prefix_len <= 0 || prefix_len % block_size != 0 || prefix_len > (int64_t)max_blocks_per_seq * block_size)
    return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (block_size < 8)  // no tensor-core prefix pass for 4-token blocks: same result through pa_decode
    return pa_decode(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, num_seqs, q_heads, kv_heads,
                     head_dim, block_size, num_blocks, scale, split_tokens, workspace, workspace_bytes, out, dtype,
                     stream);
  if (!q || !k_cache || !v_cache || !prefix_blocks || !block_tables || !context_lens || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  SharedPrefixSetup s;
  st = shared_prefix_setup(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, prefix_len, split_tokens, &s);
  if (st != PA_OK) return st;
  if (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)) return PA_ERR_WORKSPACE;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* po = reinterpret_cast<float*>(ws + s.ws.o_off);
  float* pm = reinterpret_cast<float*>(ws + s.ws.m_off);
  float* pl = reinterpret_cast<float*>(ws + s.ws.l_off);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const int bsub = block_size < 16 ? block_size : 16;
  const int G = q_heads / kv_heads;
  const float sl2 = scale * 1.4426950408889634f;
  const bool concurrent = prefix_stream != nullptr && prefix_stream != stream;
  cudaEvent_t done = nullptr;
  if (concurrent && !(done = prefix_done_event())) return PA_ERR_CUDA;
  const int key_split = concurrent ? concurrent_key_split(num_seqs, G, kv_heads, prefix_len) : kPrefixKeySplit;
  const int prefix_splits = (prefix_len + key_split - 1) / key_split;  // <= s.prefix_splits

  // 1. the shared prefix, once for every request's queries (tensor cores)
  PrefillParams pp{};
  pp.q = q;
  pp.tables = prefix_blocks;
  pp.err = err;
  pp.maxblk = prefix_len / block_size;
  pp.num_reqs = 1;
  pp.total_q = num_seqs;
  pp.max_q_len = num_seqs;
  pp.q_heads = q_heads;
  pp.kv_heads = kv_heads;
  pp.group = G;
  pp.num_blocks = num_blocks;
  pp.block_size = block_size;
  pp.scale_log2 = sl2;
  pp.causal = 0;
  pp.prefix_len = prefix_len;
  pp.key_split = key_split;
  pp.max_splits = s.max_splits;
  pp.part_o = po;
  pp.part_m = pm;
  pp.part_l = pl;
  if (concurrent) {
    cudaStream_t ps = reinterpret_cast<cudaStream_t>(prefix_stream);
    st = cuda_status(launch_attn_tc(km, vm, pp, head_dim, bsub, dtype, ps));
    if (st == PA_OK) st = cuda_status(cudaEventRecord(done, ps));
  } else {
    st = cuda_status(launch_attn_tc(km, vm, pp, head_dim, bsub, dtype, cs));
  }
  if (st != PA_OK) return st;

  // 2. each request's own suffix (paged decode, partials after the prefix's)
  DecodeParams dp{};
  dp.q = q;
  dp.tables = block_tables;
  dp.lens = context_lens;
  dp.out = out;
  dp.part_o = po;
  dp.part_m = pm;
  dp.part_l = pl;
  dp.err = err;
  dp.maxblk = max_blocks_per_seq;
  dp.num_seqs = num_seqs;
  dp.q_heads = q_heads;
  dp.kv_heads = kv_heads;
  dp.group = G;
  dp.num_blocks = num_blocks;
  dp.block_size = block_size;
  dp.split_tokens = s.split;
  dp.max_splits = s.max_splits;
  dp.grid_splits = s.suffix_splits;
  dp.tab_entries = s.split / block_size;
  dp.scale_log2 = sl2;
  dp.tok_begin = prefix_len;
  dp.slot_base = prefix_splits;
  dp.always_partial = 1;
  dp.prefix_blocks = prefix_blocks;
  dp.prefix_nblk = prefix_len / block_size;
  dp.q_len = 1;
  st = cuda_status(launch_decode_partial(km, vm, dp, head_dim, bsub, dtype, cs));
  if (st != PA_OK) return st;

  // 3. log-sum-exp merge of prefix and suffix partials
  MergeParams mp{};
  mp.part_o = po;
  mp.part_m = pm;
  mp.part_l = pl;
  mp.lens = context_lens;
  mp.out = out;
  mp.num_seqs = num_seqs;
  mp.q_heads = q_heads;
  mp.max_splits = s.max_splits;
  mp.split_tokens = s.split;
  mp.cap = max_blocks_per_seq * block_size;
  mp.tok_begin = prefix_len;
  mp.extra_slots = prefix_splits;
  mp.always = 1;
  mp.q_len = 1;
  if (concurrent && cudaStreamWaitEvent(cs, done, 0) != cudaSuccess) return PA_ERR_CUDA;
  return cuda_status(launch_lse_merge(mp, head_dim, dtype, cs));
}

int pa_norm_rope_and_cache(const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
                           int64_t v_stride, const void* q_weight, const void* k_weight, float eps,
                           const int32_t* positions, int num_axes, const int32_t* sections, const float* cos_sin,
                           int max_position, int rot_dim, int interleaved, const int32_t* slot_mapping,
                           int num_tokens, int q_heads, void* q_out, void* k_cache, void* v_cache, int num_blocks,
                           int block_size, int kv_heads, int head_dim, pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_tokens < 0 || q_heads <= 0 || q_heads > 16384 || !(eps >= 0.f) || !std::isfinite(eps)) return PA_ERR_INVALID;
  if (rot_dim < 16 || rot_dim % 16 != 0 || rot_dim > head_dim || max_position <= 0) return PA_ERR_INVALID;
  if (num_axes < 1 || num_axes > 3 || (num_axes > 1 && !sections)) return PA_ERR_INVALID;
  const int64_t qrow = (int64_t)q_heads * head_dim, krow = (int64_t)kv_heads * head_dim;
  if (q_stride < qrow || k_stride < krow || v_stride < krow || q_stride % 8 || k_stride % 8 || v_stride % 8)
    return PA_ERR_INVALID;
  NormRopeParams p{};
  p.sec_end[0] = p.sec_end[1] = rot_dim / 2;
  if (sections) {
    int64_t sum = 0;
    for (int a = 0; a < num_axes; ++a) {
      if (sections[a] < 0) return PA_ERR_INVALID;
      sum += sections[a];
      if (a < 2) p.sec_end[a] = (int)(sum < rot_dim / 2 ? sum : rot_dim / 2);
    }
    if (sum != rot_dim / 2) return PA_ERR_INVALID;
  }
  if (num_tokens == 0) return PA_OK;
  if (!q || !k || !v || !positions || !cos_sin || !slot_mapping || !q_out || !k_cache || !v_cache)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cos_sin) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q_weight) || !aligned16(k_weight))
    return PA_ERR_INVALID;
  if (q_out == q && q_stride != qrow) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.slots = slot_mapping;
  p.q_out = q_out;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.err = err;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.num_tokens = num_tokens;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.num_axes = num_axes;
  p.max_position = max_position;
  p.rot_dim = rot_dim;
  p.interleaved = interleaved != 0;
  p.eps = eps;
  return cuda_status(launch_norm_rope(p, head_dim, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

// Workspace of pa_decode_accumulate: the partials of every partition (and the
// sums of their unrounded probabilities), then the logits
// [num_seqs][kv_heads][cap][group_pad].
struct AccumulateSetup {
  int split, max_splits, cap, group_pad;
  DecodeWorkspace ws;
  size_t w_off, logits_off, bytes;
};

int accumulate_setup(int num_seqs, int q_heads, int kv_heads, int head_dim, int max_blocks_per_seq, int block_size,
                     int split_tokens, AccumulateSetup* s) {
  if (num_seqs < 0 || num_seqs > 65535 || kv_heads <= 0 || q_heads <= 0 || q_heads % kv_heads != 0 || head_dim <= 0)
    return PA_ERR_INVALID;
  const int group = q_heads / kv_heads;
  if (group > 16) return PA_ERR_INVALID;
  int split = pa_decode_split_tokens(max_blocks_per_seq, block_size, split_tokens);
  if (split <= 0) return PA_ERR_INVALID;
  if (split_tokens == 0) {
    // A warp takes a partition.  Too few of them leave SMs without their 12
    // warps each: 256, 128 or 64 tokens then.  More than about 54 per SM only
    // add partials, which every CTA of the second pass reads: doubled.
    // Measured on GB300 (us; 4 requests of <= 1500 tokens, 28/4 heads): 384
    // tokens 28.8, 256 20.7, 128 13.1, 64 9.7; 8 of 33..131 thousand, 64/8
    // heads: 256 523, 512 509, 1024 514, 2048 521.
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    const int64_t cap = (int64_t)max_blocks_per_seq * block_size, lists = (int64_t)num_seqs * kv_heads;
    auto units = [&](int sp) { return lists * ((cap + sp - 1) / sp); };
    if (units(split) < 12 * sms)
      for (split = 256; split > 64 && units(split) < 12 * sms;) split /= 2;
    while (units(split) > 54 * sms && split * 2 <= 256 * block_size) split *= 2;
  }
  DecodeSetup d;
  const int st = decode_setup(num_seqs, q_heads, head_dim, max_blocks_per_seq, block_size, split, &d);
  if (st != PA_OK) return st;
  s->group_pad = group <= 2 ? group : (group + 3) / 4 * 4;
  s->split = d.split;
  s->max_splits = d.max_splits;
  s->cap = max_blocks_per_seq * block_size;
  s->ws = decode_workspace_layout(num_seqs, q_heads, head_dim, d.max_splits);
  s->w_off = s->ws.bytes;
  s->logits_off = s->w_off + (((size_t)num_seqs * q_heads * d.max_splits * sizeof(float) + 255) & ~size_t(255));
  s->bytes = s->logits_off + (size_t)num_seqs * kv_heads * s->group_pad * s->cap * sizeof(float);
  return PA_OK;
}

}  // namespace

int pa_decode_accumulate_split_tokens(int num_seqs, int q_heads, int kv_heads, int max_blocks_per_seq, int block_size,
                                      int split_tokens) {
  AccumulateSetup s;
  const int st = accumulate_setup(num_seqs, q_heads, kv_heads, 64, max_blocks_per_seq, block_size, split_tokens, &s);
  return st != PA_OK ? st : s.split;
}

size_t pa_decode_accumulate_workspace_size(int num_seqs, int q_heads, int kv_heads, int head_dim,
                                           int max_blocks_per_seq, int block_size, int split_tokens) {
  AccumulateSetup s;
  if (accumulate_setup(num_seqs, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s) !=
      PA_OK)
    return 0;
  return s.bytes;
}

int pa_decode_accumulate(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                         int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_heads, int kv_heads,
                         int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                         const float* scores, const int32_t* score_rows, int num_rows, int score_len,
                         float* scores_out, void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype,
                         pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || q_heads <= 0 || q_heads % kv_heads != 0 || q_heads / kv_heads > 16)
    return PA_ERR_INVALID;
  if (max_blocks_per_seq <= 0 || !std::isfinite(scale) || num_rows <= 0 || score_len <= 0) return PA_ERR_INVALID;
  if ((int64_t)num_seqs * q_heads > (int64_t)INT32_MAX - 8) return PA_ERR_INVALID;
  if (!score_rows && num_rows < num_seqs) return PA_ERR_INVALID;
  AccumulateSetup s;
  st = accumulate_setup(num_seqs, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s);
  if (st != PA_OK) return st;
  if ((int64_t)s.max_splits * kv_heads > (int64_t)INT32_MAX) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !scores || !scores_out)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned16(scores) ||
      !aligned16(scores_out))
    return PA_ERR_INVALID;
  const int64_t lists = (int64_t)num_rows * kv_heads;
  if (lists > (int64_t(1) << 48) / score_len) return PA_ERR_INVALID;  // no address space holds it
  if (scores != scores_out && overlap4(scores, lists * score_len, scores_out, lists * score_len)) return PA_ERR_INVALID;
  if (!workspace || workspace_bytes < s.bytes || !aligned16(workspace)) return PA_ERR_WORKSPACE;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  DecodeParams p{};
  p.q = q;
  p.tables = block_tables;
  p.lens = context_lens;
  p.out = out;
  p.part_o = reinterpret_cast<float*>(ws + s.ws.o_off);
  p.part_m = reinterpret_cast<float*>(ws + s.ws.m_off);
  p.part_l = reinterpret_cast<float*>(ws + s.ws.l_off);
  p.part_w = reinterpret_cast<float*>(ws + s.w_off);
  p.logits = reinterpret_cast<float*>(ws + s.logits_off);
  p.group_pad = s.group_pad;
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.split_tokens = s.split;
  p.max_splits = s.max_splits;
  p.grid_splits = s.max_splits;
  p.tab_entries = s.split / block_size;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.q_len = 1;
  p.always_partial = 1;
  st = cuda_status(launch_decode_logits(km, vm, p, head_dim, block_size < 16 ? block_size : 16, dtype, cs));
  if (st != PA_OK) return st;
  MergeParams mp{};
  mp.part_o = p.part_o;
  mp.part_m = p.part_m;
  mp.part_l = p.part_l;
  mp.lens = context_lens;
  mp.out = out;
  mp.num_seqs = num_seqs;
  mp.q_heads = q_heads;
  mp.max_splits = s.max_splits;
  mp.split_tokens = s.split;
  mp.cap = s.cap;
  mp.always = 1;
  mp.q_len = 1;
  AccumulateParams ap{};
  ap.logits = p.logits;
  ap.part_m = p.part_m;
  ap.part_w = p.part_w;
  ap.lens = context_lens;
  ap.scores = scores;
  ap.scores_out = scores_out;
  ap.score_rows = score_rows;
  ap.err = err;
  ap.num_seqs = num_seqs;
  ap.q_heads = q_heads;
  ap.kv_heads = kv_heads;
  ap.group = p.group;
  ap.group_pad = s.group_pad;
  ap.max_splits = s.max_splits;
  ap.split_tokens = s.split;
  ap.cap = s.cap;
  ap.num_rows = num_rows;
  ap.score_len = score_len;
  return cuda_status(launch_merge_accumulate(mp, ap, head_dim, dtype, cs));
}

int pa_evict_select(const float* scores, const int32_t* score_rows, int num_rows, int kv_heads, int score_len,
                    const int32_t* context_lens, int num_seqs, int sink, int heavy, int recent, int32_t* keep,
                    int32_t* keep_lens, pa_stream stream) {
  if (num_rows <= 0 || kv_heads <= 0 || kv_heads > 1024 || score_len <= 0 || num_seqs < 0 || num_seqs > 65535)
    return PA_ERR_INVALID;
  if (sink < 0 || heavy < 0 || recent < 0) return PA_ERR_INVALID;
  const int64_t budget = (int64_t)sink + heavy + recent;
  if (budget < 1 || budget > INT32_MAX) return PA_ERR_INVALID;
  if (!score_rows && num_rows < num_seqs) return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!scores || !context_lens || !keep || !keep_lens || !aligned16(scores) || !aligned16(keep)) return PA_ERR_INVALID;
  // every CTA of a row reads the inputs while others write the outputs
  const int64_t nkeep = (int64_t)num_seqs * kv_heads * budget, lists = (int64_t)num_rows * kv_heads;
  if (lists > (int64_t(1) << 48) / score_len) return PA_ERR_INVALID;  // no address space holds it
  const int64_t nscores = lists * score_len;
  const struct { const void* p; int64_t n; } outs[] = {{keep, nkeep}, {keep_lens, num_seqs}};
  for (const auto& o : outs)
    if (overlap4(o.p, o.n, context_lens, num_seqs) || overlap4(o.p, o.n, scores, nscores) ||
        (score_rows && overlap4(o.p, o.n, score_rows, num_seqs)))
      return PA_ERR_INVALID;
  if (overlap4(keep, nkeep, keep_lens, num_seqs)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  EvictSelectParams p{};
  p.scores = scores;
  p.score_rows = score_rows;
  p.lens = context_lens;
  p.keep = keep;
  p.keep_lens = keep_lens;
  p.err = err;
  p.num_rows = num_rows;
  p.kv_heads = kv_heads;
  p.score_len = score_len;
  p.sink = sink;
  p.heavy = heavy;
  p.recent = recent;
  return cuda_status(launch_evict_select(p, num_seqs, reinterpret_cast<cudaStream_t>(stream)));
}

int pa_compact_kv(void* k_cache, void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                  const int32_t* context_lens, const int32_t* keep, int keep_heads, int max_keep,
                  const int32_t* keep_lens, const int32_t* base, int num_seqs, int num_blocks, int block_size,
                  int kv_heads, int head_dim, pa_dtype dtype, float* scores, const int32_t* score_rows, int num_rows,
                  int score_len, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || max_blocks_per_seq <= 0 || max_keep <= 0 ||
      max_keep > INT32_MAX - (1 << 16))
    return PA_ERR_INVALID;
  if (keep_heads != 1 && keep_heads != kv_heads) return PA_ERR_INVALID;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PA_ERR_INVALID;
  if (scores && (num_rows <= 0 || score_len <= 0 || (!score_rows && num_rows < num_seqs) || !aligned16(scores)))
    return PA_ERR_INVALID;
  if (num_seqs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_tables || !context_lens || !keep || !keep_lens) return PA_ERR_INVALID;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  CompactParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.tables = block_tables;
  p.lens = context_lens;
  p.keep = keep;
  p.keep_lens = keep_lens;
  p.base = base;
  p.scores = scores;
  p.score_rows = score_rows;
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.cap = max_blocks_per_seq * block_size;
  p.keep_heads = keep_heads;
  p.max_keep = max_keep;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.kv_heads = kv_heads;
  p.num_rows = num_rows;
  p.score_len = score_len;
  p.row_vecs = head_dim / 8;
  return cuda_status(launch_compact_kv(p, num_seqs, reinterpret_cast<cudaStream_t>(stream)));
}

namespace {

constexpr int kTreeMaxNodes = 64;    // one mask word per node
constexpr int kTreeSplitUnit = 128;  // partitions are whole key tiles
constexpr int kTreeSplitMin = 256;
constexpr int kTreeSplitLong = 4096;  // a short partition; above it, they are cut for balance

struct TreeSetup {
  int split, max_splits;
  DecodeWorkspace ws;
};

int tree_setup(int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads, int head_dim,
               int max_blocks_per_seq, int block_size, int split_tokens, TreeSetup* s) {
  if (num_reqs < 0 || num_reqs > 65535 || total_q < 0 || max_q_len < 1 || max_q_len > kTreeMaxNodes || q_heads <= 0 ||
      kv_heads <= 0 || q_heads % kv_heads != 0 || q_heads / kv_heads > 16 || head_dim <= 0 ||
      max_blocks_per_seq <= 0 || block_size <= 0)
    return PA_ERR_INVALID;
  const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
  if (cap > INT32_MAX - kTreeSplitUnit || (int64_t)total_q * q_heads > INT32_MAX) return PA_ERR_INVALID;
  const int64_t whole = (cap + kTreeSplitUnit - 1) / kTreeSplitUnit * kTreeSplitUnit;
  int64_t split = split_tokens;
  if (split_tokens == 0) {
    // Units (requests x KV heads x tiles of 128 or 256 rows) that give every
    // SM two run whole: a partition's partials (a kilobyte written and read
    // per row) then cost more than the balance brings.  Measured on GB300, 64
    // requests of <= 4096 tokens, 8 KV heads: whole 132 us, 2048-token
    // partitions 153 us (80..128 rows); 162 and 190 us (104..240 rows); whole
    // and in order of length 127 and 143.  The number of units alone decides: a
    // context far longer than the rest of such a batch is still walked whole, by
    // one CTA per KV head (one of 131008 among 63 of 1000..3000, 26..60 nodes:
    // whole 1610 us, 4096-token partitions 365, 16384 271; without it 136), and
    // a caller that has one gives split_tokens.  Fewer units are cut until seven
    // SMs in eight have one, where a partition then is short: starting and ending
    // it takes 6 to 8 us, as much as 800 tokens (us at that and at four per SM:
    // a context of 8000, 32 rows 15 and 23; one of 32000, 64 rows 30 and 62,
    // and 36 with a unit on nearly every SM; 8 of <= 4000, 64 rows 25 and 36).
    // Long ones are cut into about four per SM, which evens out contexts of
    // different lengths (8 of 33..131 thousand, 128 rows: 65536 tokens 649 us,
    // 32768 568, 12288 462, 4096 507), but not below kTreeSplitLong (12 of <=
    // 8000, 64 rows: 4096 tokens 45, 2048 50, 1280 56).  No
    // partition is smaller than its partials are worth, twice the rows (one of
    // 8060, 240 rows: 1024 tokens 25.7 us, 512 24.0, 256 37.8).
    const int64_t rows = (int64_t)max_q_len * (q_heads / kv_heads);
    int64_t units = (int64_t)num_reqs * kv_heads * (rows <= 128 ? 1 : (rows + 255) / 256);
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    split = whole;
    if (units < 2 * sms) {
      units = units > 0 ? units : 1;
      const int64_t most = sms * 7 / 8, parts = units < most ? most / units : 1;
      split = (cap + parts - 1) / parts;
      if (split > kTreeSplitLong) {
        split = cap * units / (4 * sms);
        if (split < kTreeSplitLong) split = kTreeSplitLong;
      }
      split = split > 2 * rows ? split : 2 * rows;
      split = (split + kTreeSplitUnit - 1) / kTreeSplitUnit * kTreeSplitUnit;
      if (split < kTreeSplitMin) split = kTreeSplitMin;
    }
  }
  if (split <= 0 || split % kTreeSplitUnit != 0) return PA_ERR_INVALID;
  if (split > whole) split = whole;
  s->split = (int)split;
  s->max_splits = (int)((cap + split - 1) / split);
  s->ws = s->max_splits > 1 ? decode_workspace_layout(total_q, q_heads, head_dim, s->max_splits)
                            : DecodeWorkspace{0, 0, 0, 0};
  return PA_OK;
}

}  // namespace

int pa_verify_tree_split_tokens(int num_reqs, int max_q_len, int q_heads, int kv_heads, int max_blocks_per_seq,
                                int block_size, int split_tokens) {
  TreeSetup s;
  const int st = tree_setup(num_reqs, 0, max_q_len, q_heads, kv_heads, 64, max_blocks_per_seq, block_size,
                            split_tokens, &s);
  return st != PA_OK ? st : s.split;
}

size_t pa_verify_tree_workspace_size(int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads,
                                     int head_dim, int max_blocks_per_seq, int block_size, int split_tokens) {
  TreeSetup s;
  if (tree_setup(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size,
                 split_tokens, &s) != PA_OK)
    return 0;
  return s.ws.bytes;
}

int pa_verify_tree(const void* q, const int32_t* q_start, const uint64_t* tree_mask, const int32_t* context_lens,
                   const void* k_cache, const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                   int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads, int head_dim, int block_size,
                   int num_blocks, float scale, int split_tokens, void* workspace, size_t workspace_bytes, void* out,
                   pa_dtype dtype, pa_stream stream) {
  int st = check_kv_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  // masked logits are -inf and meet the scale: it must neither vanish nor turn their sign
  if (!std::isnormal(scale) || scale < 0.f) return PA_ERR_INVALID;
  TreeSetup s;
  st = tree_setup(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size,
                  split_tokens, &s);
  if (st != PA_OK) return st;
  if (num_reqs == 0 || total_q == 0) return PA_OK;
  if (!q || !q_start || !tree_mask || !context_lens || !k_cache || !v_cache || !block_tables || !out)
    return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7u))
    return PA_ERR_INVALID;
  if (s.ws.bytes > 0 && (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  CUtensorMap km, vm;
  if (!kv_map(k_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &km) ||
      !kv_map(v_cache, num_blocks, block_size, kv_heads, head_dim, dtype, &vm))
    return PA_ERR_CUDA;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  TreeParams p{};
  p.q = q;
  p.v_cache = v_cache;
  p.q_start = q_start;
  p.mask = tree_mask;
  p.lens = context_lens;
  p.tables = block_tables;
  p.out = out;
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.num_reqs = num_reqs;
  p.total_q = total_q;
  p.max_q_len = max_q_len;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.split_tokens = s.split;
  p.max_splits = s.max_splits;
  // not for the few-row form, whose units are bound by latency and HBM alike:
  // the order costs it more than the shorter end brings (see tree_longest_first)
  p.longest_first =
      s.max_splits == 1 && (int64_t)num_reqs * kv_heads > sm_count() && max_q_len * p.group > 32;
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (s.ws.bytes) {
    p.part_o = reinterpret_cast<float*>(ws + s.ws.o_off);
    p.part_m = reinterpret_cast<float*>(ws + s.ws.m_off);
    p.part_l = reinterpret_cast<float*>(ws + s.ws.l_off);
  }
  return cuda_status(launch_verify_tree(km, vm, p, head_dim, block_size < 16 ? block_size : 16, dtype,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int pa_selftest_wait_timeout(int wait_ms, pa_stream stream) {
  if (wait_ms < 1 || wait_ms > 2000) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  return cuda_status(launch_wait_timeout(err, (uint64_t)wait_ms * 1000000ull, reinterpret_cast<cudaStream_t>(stream)));
}

int pa_get_device_error(int32_t* host_code, pa_stream stream) {
  if (!host_code) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, err, sizeof(int32_t), cudaMemcpyDeviceToHost, s) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaMemsetAsync(err, 0, sizeof(int32_t), s) != cudaSuccess) return PA_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return PA_ERR_CUDA;
  *host_code = v;
  return v ? PA_ERR_DEVICE_CHECK : PA_OK;
}

}  // extern "C"
