// Choosing and moving the tokens a cache keeps, for sm_103a: pa_evict_select
// (per request and KV head, the tokens with the largest accumulated attention)
// and pa_compact_kv (the kept tokens moved together, in place).
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// Order-preserving map of fp32 to uint32 (-0 equals +0, NaN below everything).
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = x == 0.f ? 0u : __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Sum of v over the threads before this one, and over all of them (total);
// scratch: one word per warp and one more.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* scratch, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  uint32_t before = 0, all = 0;
  for (int w = 0; w < nw; ++w) {
    const uint32_t s = scratch[w];
    if (w < warp) before += s;
    all += s;
  }
  __syncthreads();
  total = all;
  return before + x - v;
}

constexpr int kSelThreads = 512;

// One CTA per (KV head, request).  The heavy-th largest key of the candidates
// [sink, L - recent) is found digit by digit (8 bits, from the top: a
// histogram in shared memory, then the digit where the count from above
// passes what is still wanted); a last pass writes the candidates above it,
// and of those equal to it the first ones, in order.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictSelectParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t scan[kSelThreads / 32 + 1];
  __shared__ uint32_t s_digit, s_want;
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.y, g = blockIdx.x;
  const int tid = threadIdx.x;
  const int budget = p.sink + p.heavy + p.recent;
  int32_t* keep = p.keep + ((size_t)r * p.kv_heads + g) * budget;
  const int row = p.score_rows ? __ldg(p.score_rows + r) : r;
  const int L = __ldg(p.lens + r);
  if (row < 0 || row >= p.num_rows || L < 0 || L > p.score_len) {
    if (tid == 0) {
      record_error(p.err, row < 0 || row >= p.num_rows ? PA_DEVERR_SCORE_ROW : PA_DEVERR_CONTEXT_LEN);
      if (g == 0) p.keep_lens[r] = 0;
    }
    for (int i = tid; i < budget; i += kSelThreads) keep[i] = -1;
    return;
  }
  if (tid == 0 && g == 0) p.keep_lens[r] = min(L, budget);
  if (L <= budget) {
    for (int i = tid; i < budget; i += kSelThreads) keep[i] = i < L ? i : -1;
    return;
  }
  for (int i = tid; i < p.sink; i += kSelThreads) keep[i] = i;
  for (int i = tid; i < p.recent; i += kSelThreads) keep[p.sink + p.heavy + i] = L - p.recent + i;
  if (p.heavy == 0) return;
  const float* sc = p.scores + ((size_t)row * p.kv_heads + g) * p.score_len + p.sink;
  const int n = L - p.sink - p.recent;  // > heavy

  uint32_t prefix = 0, want = p.heavy;  // of the keys with this prefix, `want` are still to be chosen
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = score_key(__ldg(sc + i));
      if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    // counts from the top: thread d holds digit 255 - d
    uint32_t total;
    const uint32_t mine = tid < 256 ? hist[255 - tid] : 0u;
    const uint32_t above = block_exclusive(mine, scan, total);
    if (tid < 256 && above < want && above + mine >= want) {
      s_digit = 255 - tid;
      s_want = want - above;
    }
    __syncthreads();
    prefix = (prefix << 8) | s_digit;
    want = s_want;
  }
  // prefix: the heavy-th largest key; `want` of the equal ones are taken
  uint32_t out = 0, ties = 0;  // entries written, equal keys seen
  for (int i0 = 0; i0 < n; i0 += kSelThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < n ? score_key(__ldg(sc + i)) : 0u;
    const bool eq = i < n && k == prefix;
    uint32_t neq;
    const uint32_t my_tie = ties + block_exclusive(eq ? 1u : 0u, scan, neq);
    const bool take = i < n && (k > prefix || (eq && my_tie < want));
    uint32_t taken;
    const uint32_t at = out + block_exclusive(take ? 1u : 0u, scan, taken);
    if (take) keep[p.sink + at] = p.sink + i;
    out += taken;
    ties += neq;
  }
}

// ----------------------------------------------------------------------------
// In-place compaction: destination i, source keep[i] >= i.  A CTA takes one
// 64-byte column of one head's K or V rows (or the head's scores) and walks
// the entries in order, CHUNK at a time: all loads of a chunk, a barrier, its
// stores.  A store to place i can only overwrite a source read by an entry
// <= i (sources are never before their destinations), which is in this chunk
// or an earlier one, so no entry reads what another has written.
constexpr int kMoveThreads = 256;
constexpr int kMoveLanes = 4;                            // 16-byte vectors of a column
constexpr int kMoveRows = kMoveThreads / kMoveLanes;     // rows per step
constexpr int kMoveUnroll = 4;                           // steps per chunk

struct MoveRange {
  int base, n, L;
};

// The request's range, checked; false: nothing is moved.
__device__ __forceinline__ bool move_range(const CompactParams& p, int r, MoveRange& m, bool report) {
  m.L = __ldg(p.lens + r);
  m.n = __ldg(p.keep_lens + r);
  m.base = p.base ? __ldg(p.base + r) : 0;
  if (m.L < 0 || m.L > p.cap) {
    if (report) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
    return false;
  }
  if (m.base < 0 || m.base > m.L || m.n < 0 || m.n > p.max_keep || m.n > m.L - m.base) {
    if (report) record_error(p.err, PA_DEVERR_KEEP);
    return false;
  }
  return true;
}

__global__ void __launch_bounds__(kMoveThreads) compact_kv_kernel(const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.z, g = blockIdx.y, part = blockIdx.x;
  const int tid = threadIdx.x;
  MoveRange m;
  if (!move_range(p, r, m, tid == 0 && g == 0 && part == 0)) return;
  const int32_t* keep = p.keep + ((size_t)r * p.keep_heads + (p.keep_heads == 1 ? 0 : g)) * p.max_keep;
  const int room = m.L - m.base;

  if (part == 2 * p.columns) {  // the scores of this head
    const int row = p.score_rows ? __ldg(p.score_rows + r) : r;
    if (row < 0) return;
    bool twice = false;
    if (p.score_rows)
      for (int i = tid; i < r; i += kMoveThreads) twice |= __ldg(p.score_rows + i) == row;
    twice = __syncthreads_or(twice);
    if (row >= p.num_rows || twice) {
      if (tid == 0) record_error(p.err, PA_DEVERR_SCORE_ROW);
      return;
    }
    if (m.L > p.score_len) {
      if (tid == 0) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
      return;
    }
    float* sc = p.scores + ((size_t)row * p.kv_heads + g) * p.score_len + m.base;
    for (int i0 = 0; i0 < m.n; i0 += kMoveThreads) {
      const int i = i0 + tid;
      const int src = i < m.n ? __ldg(keep + i) : -1;
      const bool ok = src >= i && src < room;
      const float x = ok ? sc[src] : 0.f;
      __syncthreads();
      if (ok) sc[i] = x;
    }
    __syncthreads();  // every source has been read
    for (int i = m.n + tid; i < room; i += kMoveThreads) sc[i] = 0.f;
    return;
  }

  const int is_v = part >= p.columns;
  const int col = (is_v ? part - p.columns : part) * kMoveLanes + tid % kMoveLanes;  // 16-byte vector of the head's row
  uint4* cache = reinterpret_cast<uint4*>(is_v ? p.v_cache : p.k_cache);
  const int32_t* table = p.tables + (size_t)r * p.maxblk;
  const size_t token_vecs = (size_t)p.kv_heads * p.row_vecs;
  // address of token t's vector, or null (bad block id)
  auto at = [&](int t) -> uint4* {
    const int b = __ldg(table + t / p.block_size);
    if (b < 0 || b >= p.num_blocks) {
      record_error(p.err, PA_DEVERR_BLOCK_ID);
      return nullptr;
    }
    return cache + ((size_t)b * p.block_size + t % p.block_size) * token_vecs + (size_t)g * p.row_vecs + col;
  };
  for (int i0 = 0; i0 < m.n; i0 += kMoveRows * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    uint4* dst[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = i0 + u * kMoveRows + tid / kMoveLanes;
      dst[u] = nullptr;
      if (i < m.n) {
        const int src = __ldg(keep + i);
        if (src < i || src >= room) {
          record_error(p.err, PA_DEVERR_KEEP);
        } else if (src != i) {
          const uint4* s = at(m.base + src);
          dst[u] = at(m.base + i);
          if (s && dst[u]) x[u] = *s;
          else dst[u] = nullptr;
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (dst[u]) *dst[u] = x[u];
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectParams& p, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0) return cudaSuccess;
  return launch_pdl(evict_select_kernel, dim3(p.kv_heads, num_seqs), dim3(kSelThreads), 0, stream, p);
}

cudaError_t launch_compact_kv(const CompactParams& p0, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0) return cudaSuccess;
  CompactParams p = p0;
  p.columns = p.row_vecs / kMoveLanes;
  return launch_pdl(compact_kv_kernel, dim3(2 * p.columns + (p.scores ? 1 : 0), p.kv_heads, num_seqs),
                    dim3(kMoveThreads), 0, stream, p);
}

}  // namespace pa
