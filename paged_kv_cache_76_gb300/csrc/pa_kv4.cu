// C ABI of the 4-bit paged cache and of pages forked on the device: argument
// checks and launches (see include/pa.h for the contract).
#include <cmath>
#include <cstdint>

#include "pa_internal.h"

namespace pa {

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int cuda_status(cudaError_t e) { return e == cudaSuccess ? PA_OK : PA_ERR_CUDA; }

cudaStream_t to_stream(pa_stream s) { return reinterpret_cast<cudaStream_t>(s); }

bool block_size_ok(int bs) { return bs == 4 || bs == 8 || bs == 16 || bs == 32; }

int check_kv4_shape(int num_blocks, int block_size, int kv_heads, int head_dim, pa_dtype dt) {
  if (dt != PA_FP16 && dt != PA_BF16) return PA_ERR_DTYPE;
  if (head_dim != 64 && head_dim != 128) return PA_ERR_INVALID;
  if (!block_size_ok(block_size)) return PA_ERR_INVALID;
  if (kv_heads <= 0 || kv_heads > 1024 || num_blocks <= 0) return PA_ERR_INVALID;
  if ((int64_t)num_blocks * block_size > INT32_MAX) return PA_ERR_INVALID;  // slots are int32
  return PA_OK;
}

int log2_of(int bs) { return bs == 4 ? 2 : bs == 8 ? 3 : bs == 16 ? 4 : 5; }

constexpr int kKv4SplitUnit = 32;  // partitions begin with a block, of any size, and with a tile of 16 tokens

struct Kv4DecodeSetup {
  int split, max_splits;
  bool cluster;
  DecodeWorkspace ws;
};

int kv4_decode_setup(int num_seqs, int q_len, int q_heads, int kv_heads, int head_dim, int max_blocks_per_seq,
                     int block_size, int split_tokens, Kv4DecodeSetup* s) {
  if (num_seqs < 0 || num_seqs > 65535 || q_len < 1 || q_len > 32 || q_heads <= 0 || kv_heads <= 0 || kv_heads > 1024 ||
      q_heads % kv_heads != 0 || head_dim <= 0 || max_blocks_per_seq <= 0 || !block_size_ok(block_size))
    return PA_ERR_INVALID;
  const int group = q_heads / kv_heads;
  if (group > 16 || group * q_len > 32) return PA_ERR_INVALID;
  const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
  if (cap > INT32_MAX - 4096 || (int64_t)num_seqs * q_len * q_heads > INT32_MAX - 8) return PA_ERR_INVALID;
  const int most = 1024 * block_size;
  const int64_t sms = num_sms() > 0 ? num_sms() : 152;
  const int64_t lists = (int64_t)num_seqs * kv_heads * ((group * q_len + 15) / 16);
  int64_t split = split_tokens;
  // Partitions of a list that run at the same time may be a cluster, which joins
  // its parts without a second kernel; more than twelve CTAs find no place in a
  // part of the chip that others already share.
  const int resident = group * q_len <= 8 ? 4 : 3;  // CTAs an SM holds
  auto clusters = [&](int64_t parts, int64_t tokens) {
    return parts > 1 && parts <= kKv4Cluster && tokens / block_size <= kKv4ClusterEntries &&
           lists * parts <= (parts > 12 ? 2 : resident) * sms;
  };
  if (split_tokens == 0) {
    // The number of partitions that is the fastest by this count, in ns, of what
    // was measured on GB300 for 1, 4 and 16 requests of 512..32768 tokens, 28/4 and
    // 32/8 heads, one query and four, with 2..64 partitions (within 2 % of the
    // fastest, on average): a CTA takes longer a token the more share its SM (a
    // cluster's sooner, as they lie together); those after the first round start as
    // others end; starting and ending cost what a count of CTAs does.
    const bool wide = group * q_len > 8;
    const int64_t first = (cap + 4095) / 4096 > (cap + most - 1) / most ? (cap + 4095) / 4096 : (cap + most - 1) / most;
    int64_t best = 0;
    for (int64_t parts = first; parts == first || (parts * 64 <= cap && parts <= first + 256);
         parts += 1 + parts / 12) {
      int64_t tokens = (cap + parts - 1) / parts;
      tokens = (tokens + kKv4SplitUnit - 1) / kKv4SplitUnit * kKv4SplitUnit;
      if (tokens > most) tokens = most;
      const bool joined = clusters(parts, tokens);
      const double x = (double)(lists * parts) / sms;
      double k = joined ? 2.7 * x : std::ceil(x);
      k = k < 1 ? 1 : k > resident ? resident : k;
      const double rounds = x > resident ? 0.7 * x / resident + 0.5 : 1;  // contexts that are not all full
      const double cost = 2200 + 570 * x + (double)tokens * (wide ? 4.7 + 3.7 * k : 3.9 + 2.1 * k) * rounds +
                          (parts == 1 ? 0 : joined ? 720 + 12 * parts : 1230 + 35 * parts);
      if (best == 0 || (int64_t)cost < best) {
        best = (int64_t)cost;
        split = tokens;
      }
    }
  }
  if (split <= 0 || split % kKv4SplitUnit != 0 || split > most) return PA_ERR_INVALID;
  s->split = (int)split;
  s->max_splits = (int)((cap + split - 1) / split);
  if ((int64_t)s->max_splits * kv_heads > INT32_MAX - 8) return PA_ERR_INVALID;
  s->cluster = clusters(s->max_splits, split);
  s->ws = s->max_splits > 1 && !s->cluster ? decode_workspace_layout(num_seqs * q_len, q_heads, head_dim, s->max_splits)
                            : DecodeWorkspace{0, 0, 0, 0};
  return PA_OK;
}

constexpr int kKv4PrefillUnit = 64;  // a key tile of the kernel
constexpr int kKv4PrefillMin = 256;  // keys of a partition chosen here

struct Kv4PrefillSetup {
  int split, max_splits, row_tiles;
  DecodeWorkspace ws;
};

int kv4_prefill_setup(int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads, int head_dim,
                      int max_blocks_per_seq, int block_size, int split_tokens, Kv4PrefillSetup* s) {
  // chunks of no query: only where there are none, or no requests
  if (num_reqs < 0 || num_reqs > 65535 || total_q < 0 || max_q_len < 0 ||
      (max_q_len == 0 && num_reqs > 0 && total_q > 0) || q_heads <= 0 || kv_heads <= 0 || kv_heads > 1024 ||
      q_heads % kv_heads != 0 || q_heads / kv_heads > 16 || head_dim <= 0 || max_blocks_per_seq <= 0 ||
      !block_size_ok(block_size))
    return PA_ERR_INVALID;
  const int64_t cap = (int64_t)max_blocks_per_seq * block_size;
  const int64_t rows = (int64_t)max_q_len * (q_heads / kv_heads);
  if (cap > INT32_MAX - 4096 || (int64_t)total_q * q_heads > INT32_MAX || rows > INT32_MAX - 4096 ||
      (int64_t)max_q_len * q_heads > INT32_MAX)
    return PA_ERR_INVALID;
  s->row_tiles = (int)((rows + 255) / 256);
  const int64_t whole = (cap + kKv4PrefillUnit - 1) / kKv4PrefillUnit * kKv4PrefillUnit;
  int64_t split = split_tokens;
  if (split_tokens == 0) {
    // Partitions that give the shortest time by this count, in quarters of a us:
    // a key tile of a unit takes 3, starting and ending a unit 28, and a merge 20
    // beside its partials' way to memory and back (8 bytes an element).  Units run
    // in rounds of one per SM.  Measured on GB300: a chunk of 2048 over 34816
    // tokens, 64/8 heads (512 units of 544 tiles, 3.4 rounds) whole 1752 us, in
    // two partitions 1639; eight chunks of 257..768 over <= 4847 tokens whole 180
    // (in two 317, before the last steps, when whole took 235); four of 37..131
    // over <= 1632 whole 23, in two 23 to 26, in five 22.
    const int64_t sms = num_sms() > 0 ? num_sms() : 152;
    const int64_t units = (int64_t)num_reqs * kv_heads * s->row_tiles, tiles = whole / kKv4PrefillUnit;
    const int64_t merge_bytes = (int64_t)num_reqs * max_q_len * q_heads * 128 * 8;  // at most
    int64_t best = 0;
    split = whole;  // of no units
    for (int64_t parts = 1; units > 0 && parts <= 64 && (parts == 1 || parts * kKv4PrefillMin <= cap); ++parts) {
      const int64_t rounds = (units * parts + sms - 1) / sms;
      const int64_t cost = rounds * (28 + 3 * ((tiles + parts - 1) / parts)) +
                           (parts > 1 ? 20 + merge_bytes * parts / 1700000 : 0);
      if (best == 0 || cost < best) {
        best = cost;
        split = (tiles + parts - 1) / parts * kKv4PrefillUnit;
      }
    }
  }
  if (split <= 0 || split % kKv4PrefillUnit != 0) return PA_ERR_INVALID;
  if (split > whole) split = whole;
  s->split = (int)split;
  s->max_splits = (int)((cap + split - 1) / split);
  if ((int64_t)num_reqs * kv_heads * s->row_tiles * s->max_splits > INT32_MAX) return PA_ERR_INVALID;
  s->ws = s->max_splits > 1 ? decode_workspace_layout(total_q, q_heads, head_dim, s->max_splits)
                            : DecodeWorkspace{0, 0, 0, 0};
  return PA_OK;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

int pa_quantize_and_cache(const void* k, const void* v, int64_t k_stride, int64_t v_stride, const int32_t* slot_mapping,
                          int num_tokens, void* k_cache, void* v_cache, int num_blocks, int block_size, int kv_heads,
                          int head_dim, pa_dtype dtype, pa_stream stream) {
  const int st = check_kv4_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  const int64_t row = (int64_t)kv_heads * head_dim;
  for (const int64_t s : {k_stride, v_stride})
    if (s < row || s % 8 != 0 || s > INT64_MAX / 4 / num_tokens) return PA_ERR_INVALID;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  Kv4WriteParams p{};
  p.k = k;
  p.v = v;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slot_mapping;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.err = err;
  p.num_tokens = num_tokens;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.kv_heads = kv_heads;
  p.block_shift = log2_of(block_size);
  return cuda_status(launch_quantize_and_cache(p, head_dim, dtype, to_stream(stream)));
}

int pa_dequantize_kv4(const void* k_cache, const void* v_cache, const int32_t* slots, int num_tokens, int num_blocks,
                      int block_size, int kv_heads, int head_dim, void* k, void* v, pa_dtype dtype, pa_stream stream) {
  const int st = check_kv4_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !slots || !k_cache || !v_cache) return PA_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  Kv4ReadParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slots = slots;
  p.k = k;
  p.v = v;
  p.err = err;
  p.num_tokens = num_tokens;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.kv_heads = kv_heads;
  p.block_shift = log2_of(block_size);
  return cuda_status(launch_dequantize_kv4(p, head_dim, dtype, to_stream(stream)));
}

int pa_decode_kv4_split_tokens(int num_seqs, int q_len, int q_heads, int kv_heads, int max_blocks_per_seq,
                               int block_size, int split_tokens) {
  Kv4DecodeSetup s;
  const int st = kv4_decode_setup(num_seqs, q_len, q_heads, kv_heads, 64, max_blocks_per_seq, block_size, split_tokens, &s);
  return st != PA_OK ? st : s.split;
}

size_t pa_decode_kv4_workspace_size(int num_seqs, int q_len, int q_heads, int kv_heads, int head_dim,
                                    int max_blocks_per_seq, int block_size, int split_tokens) {
  Kv4DecodeSetup s;
  if (kv4_decode_setup(num_seqs, q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size, split_tokens,
                       &s) != PA_OK)
    return 0;
  return s.ws.bytes;
}

int pa_decode_kv4(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                  int max_blocks_per_seq, const int32_t* context_lens, int num_seqs, int q_len, int q_heads,
                  int kv_heads, int head_dim, int block_size, int num_blocks, float scale, int split_tokens,
                  void* workspace, size_t workspace_bytes, void* out, pa_dtype dtype, pa_stream stream) {
  int st = check_kv4_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  // in log2 units, as the scores are
  if (!std::isfinite(scale * 1.4426950408889634f)) return PA_ERR_INVALID;
  Kv4DecodeSetup s;
  st = kv4_decode_setup(num_seqs, q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size, split_tokens, &s);
  if (st != PA_OK) return st;
  if (num_seqs == 0) return PA_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  if (s.ws.bytes > 0 && (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  Kv4DecodeParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.tables = block_tables;
  p.lens = context_lens;
  p.out = out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (s.ws.bytes) {
    p.part_o = reinterpret_cast<float*>(ws + s.ws.o_off);
    p.part_m = reinterpret_cast<float*>(ws + s.ws.m_off);
    p.part_l = reinterpret_cast<float*>(ws + s.ws.l_off);
  }
  p.err = err;
  p.maxblk = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.q_len = q_len;
  p.q_heads = q_heads;
  p.kv_heads = kv_heads;
  p.group = q_heads / kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.split_tokens = s.split;
  p.max_splits = s.max_splits;
  p.tab_entries = s.split / block_size;
  p.cluster = s.cluster;
  p.bf16 = dtype == PA_BF16;
  p.scale_log2 = scale * 1.4426950408889634f;
  st = cuda_status(launch_kv4_decode(p, head_dim, to_stream(stream)));
  if (st != PA_OK || s.max_splits == 1 || s.cluster) return st;
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
  mp.cap = max_blocks_per_seq * block_size;
  mp.q_len = q_len;
  return cuda_status(launch_lse_merge(mp, head_dim, dtype, to_stream(stream)));
}

int pa_chunked_prefill_kv4_split_tokens(int num_reqs, int max_q_len, int q_heads, int kv_heads, int max_blocks_per_seq,
                                        int block_size, int split_tokens) {
  Kv4PrefillSetup s;
  const int st = kv4_prefill_setup(num_reqs, 0, max_q_len, q_heads, kv_heads, 64, max_blocks_per_seq, block_size,
                                   split_tokens, &s);
  return st != PA_OK ? st : s.split;
}

size_t pa_chunked_prefill_kv4_workspace_size(int num_reqs, int total_q, int max_q_len, int q_heads, int kv_heads,
                                             int head_dim, int max_blocks_per_seq, int block_size, int split_tokens) {
  Kv4PrefillSetup s;
  if (kv4_prefill_setup(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size,
                        split_tokens, &s) != PA_OK)
    return 0;
  return s.ws.bytes;
}

int pa_chunked_prefill_kv4(const void* q, const int32_t* q_start, const int32_t* context_lens, const void* k_cache,
                           const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq, int num_reqs,
                           int total_q, int max_q_len, int q_heads, int kv_heads, int head_dim, int block_size,
                           int num_blocks, float scale, int split_tokens, void* workspace, size_t workspace_bytes,
                           void* out, pa_dtype dtype, pa_stream stream) {
  int st = check_kv4_shape(num_blocks, block_size, kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  // masked scores are -inf before the scale meets them: it must not vanish
  if (!std::isnormal(scale) || !std::isfinite(scale * 1.4426950408889634f)) return PA_ERR_INVALID;
  Kv4PrefillSetup s;
  st = kv4_prefill_setup(num_reqs, total_q, max_q_len, q_heads, kv_heads, head_dim, max_blocks_per_seq, block_size,
                         split_tokens, &s);
  if (st != PA_OK) return st;
  if (num_reqs == 0 || max_q_len == 0 || total_q == 0) return PA_OK;
  if (!q || !q_start || !context_lens || !k_cache || !v_cache || !block_tables || !out) return PA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out)) return PA_ERR_INVALID;
  if (s.ws.bytes > 0 && (!workspace || workspace_bytes < s.ws.bytes || !aligned16(workspace)))
    return PA_ERR_WORKSPACE;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  Kv4PrefillParams p{};
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.q_start = q_start;
  p.lens = context_lens;
  p.tables = block_tables;
  p.out = out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (s.ws.bytes) {
    p.part_o = reinterpret_cast<float*>(ws + s.ws.o_off);
    p.part_m = reinterpret_cast<float*>(ws + s.ws.m_off);
    p.part_l = reinterpret_cast<float*>(ws + s.ws.l_off);
  }
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
  p.block_shift = log2_of(block_size);
  p.split_tokens = s.split;
  p.max_splits = s.max_splits;
  p.row_tiles = s.row_tiles;
  p.longest_first = s.max_splits == 1 && num_reqs > 1 && (int64_t)num_reqs * kv_heads * s.row_tiles > num_sms();
  p.negative = scale < 0.f;
  p.scale_log2 = std::fabs(scale) * 1.4426950408889634f;
  return cuda_status(launch_kv4_prefill(p, head_dim, dtype, to_stream(stream)));
}

size_t pa_fork_blocks_workspace_size(int num_new, int num_blocks) {
  if (num_new < 0 || num_blocks <= 0) return 0;
  return fork_workspace_layout(num_new, num_blocks).bytes;
}

int pa_fork_blocks(const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                   const int32_t* parents, int num_new, const int32_t* grow, int max_grow, const uint8_t* pinned,
                   int num_blocks, int block_size, int32_t* tables_out, int max_blocks_out, int32_t* lens_out,
                   int32_t* pairs, int32_t* slots, int32_t* num_free, void* workspace, size_t workspace_bytes,
                   pa_stream stream) {
  if (!block_size_ok(block_size) || num_blocks <= 0 || (int64_t)num_blocks * block_size > INT32_MAX)
    return PA_ERR_INVALID;
  if (num_seqs < 0 || num_seqs > 65535 || num_new < 0 || num_new > 65535 || max_blocks_per_seq <= 0 ||
      max_blocks_out <= 0 || max_grow < 0 || (!grow && max_grow > max_blocks_out * (int64_t)block_size))
    return PA_ERR_INVALID;
  const int64_t most = INT32_MAX / 2;  // lengths, and lengths with what they grow by, are int32
  if (max_blocks_per_seq > most / block_size || max_blocks_out > most / block_size || max_grow > most)
    return PA_ERR_INVALID;
  const int64_t n_out = (int64_t)num_new * max_blocks_out, n_slots = (int64_t)num_new * max_grow;
  if (n_slots > (int64_t(1) << 40)) return PA_ERR_INVALID;
  if (!num_free || (num_seqs > 0 && (!block_tables || !context_lens))) return PA_ERR_INVALID;
  if (num_new > 0 && (!parents || !tables_out || !lens_out || !pairs || (!slots && max_grow > 0))) return PA_ERR_INVALID;
  const ForkWorkspace w = fork_workspace_layout(num_new, num_blocks);
  if (!workspace || workspace_bytes < w.bytes || !aligned16(workspace)) return PA_ERR_WORKSPACE;
  // every warp reads the inputs while others write: outputs share no memory with them or one another
  const struct { const void* p; int64_t bytes; } arrays[] = {
      {tables_out, 4 * n_out}, {lens_out, 4 * (int64_t)num_new}, {pairs, 8 * (int64_t)num_new}, {slots, 4 * n_slots},
      {num_free, 4}, {workspace, (int64_t)w.bytes},
      {block_tables, 4 * (int64_t)num_seqs * max_blocks_per_seq}, {context_lens, 4 * (int64_t)num_seqs},
      {parents, 4 * (int64_t)num_new}, {grow, 4 * (int64_t)num_new}, {pinned, num_blocks}};
  constexpr int kOutputs = 6;
  for (int a = 0; a < kOutputs; ++a)
    for (int b = a + 1; b < (int)(sizeof(arrays) / sizeof(arrays[0])); ++b) {
      const uintptr_t x = reinterpret_cast<uintptr_t>(arrays[a].p), y = reinterpret_cast<uintptr_t>(arrays[b].p);
      if (!x || !y || arrays[a].bytes <= 0 || arrays[b].bytes <= 0) continue;
      if (x < y ? y - x < (uintptr_t)arrays[a].bytes : x - y < (uintptr_t)arrays[b].bytes) return PA_ERR_INVALID;
    }
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ForkParams p{};
  p.tables = block_tables;
  p.lens = context_lens;
  p.parents = parents;
  p.grow = grow;
  p.pinned = pinned;
  p.tables_out = tables_out;
  p.lens_out = lens_out;
  p.pairs = pairs;
  p.slots = slots;
  p.num_free = num_free;
  p.state = reinterpret_cast<int32_t*>(ws + w.state);
  p.row_start = reinterpret_cast<int32_t*>(ws + w.row_start);
  p.warp_free = reinterpret_cast<int32_t*>(ws + w.warp_free);
  p.needed = reinterpret_cast<int32_t*>(ws + w.needed);
  p.err = err;
  p.num_old = num_seqs;
  p.maxblk = max_blocks_per_seq;
  p.num_new = num_new;
  p.maxblk_out = max_blocks_out;
  p.max_grow = max_grow;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  p.block_shift = log2_of(block_size);
  return cuda_status(launch_fork_blocks(p, to_stream(stream)));
}

int pa_copy_pages(void* const* caches, int num_caches, const int32_t* pairs, int num_pairs, int num_blocks,
                  int64_t block_bytes, pa_stream stream) {
  if (num_caches < 0 || num_pairs < 0 || num_blocks <= 0 || block_bytes <= 0 || block_bytes % 16 != 0 ||
      block_bytes > INT64_MAX / 2 / num_blocks)
    return PA_ERR_INVALID;
  if (num_caches == 0 || num_pairs == 0) return PA_OK;
  if (!caches || !pairs) return PA_ERR_INVALID;
  for (int i = 0; i < num_caches; ++i)
    if (!caches[i] || !aligned16(caches[i])) return PA_ERR_INVALID;
  int* err = device_error_ptr();
  if (!err) return PA_ERR_CUDA;
  for (int i = 0; i < num_caches; i += kMaxCopyCaches) {
    CopyPagesParams p{};
    p.num_caches = num_caches - i < kMaxCopyCaches ? num_caches - i : kMaxCopyCaches;
    for (int k = 0; k < p.num_caches; ++k) p.caches[k] = caches[i + k];
    p.pairs = pairs;
    p.err = err;
    p.block_vecs = block_bytes / 16;
    p.num_pairs = num_pairs;
    p.num_blocks = num_blocks;
    const int st = cuda_status(launch_copy_pages(p, to_stream(stream)));
    if (st != PA_OK) return st;
  }
  return PA_OK;
}

}  // extern "C"
