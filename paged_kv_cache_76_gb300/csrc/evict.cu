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

// A cluster of CTAs takes one (KV head, request): each holds its part of the
// row's keys in shared memory, read once.  The heavy-th largest key of the
// candidates [sink, L - recent) is found digit by digit (11, 11 and 10 bits
// from the top): a histogram per CTA, summed over the cluster through
// distributed shared memory, then the digit at which the count from above
// passes what is still wanted.  Then every warp counts its run of keys above
// and equal to it, the counts before a warp give its place in the list, and it
// writes the indices in order by ballots; of the equal keys the first ones.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelMaxHeld = 40960;  // keys of a CTA in shared memory; the rest are read again

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictSelectParams p) {
  extern __shared__ uint4 smem_raw[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem_raw);  // [3][kSelBins]
  uint32_t* keys = hist + 3 * kSelBins;                    // [held]
  __shared__ uint32_t scan[kSelWarps + 1];
  __shared__ uint32_t s_digit, s_want;
  __shared__ __align__(16) uint32_t s_count[4];            // this CTA's keys above and equal to the threshold
  __shared__ uint32_t w_above[kSelWarps], w_equal[kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 3 * kSelBins; i += kSelThreads) hist[i] = 0;
  griddep_wait();
  griddep_launch_dependents();
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int r = blockIdx.y, g = blockIdx.x / C;
  const int budget = p.sink + p.heavy + p.recent;
  int32_t* keep = p.keep + ((size_t)r * p.kv_heads + g) * budget;
  const int row = p.score_rows ? __ldg(p.score_rows + r) : r;
  const int L = __ldg(p.lens + r);
  const int t0 = rank * kSelThreads + tid, tn = C * kSelThreads;  // this thread among the cluster's
  if (row < 0 || row >= p.num_rows || L < 0 || L > p.score_len) {
    if (t0 == 0) {
      record_error(p.err, row < 0 || row >= p.num_rows ? PA_DEVERR_SCORE_ROW : PA_DEVERR_CONTEXT_LEN);
      if (g == 0) p.keep_lens[r] = 0;
    }
    for (int64_t i = t0; i < budget; i += tn) keep[i] = -1;
    return;
  }
  if (t0 == 0 && g == 0) p.keep_lens[r] = min(L, budget);
  if (L <= budget) {
    for (int64_t i = t0; i < budget; i += tn) keep[i] = i < L ? (int)i : -1;
    return;
  }
  for (int64_t i = t0; i < p.sink; i += tn) keep[i] = (int)i;
  for (int64_t i = t0; i < p.recent; i += tn) keep[p.sink + p.heavy + i] = (int)(L - p.recent + i);
  if (p.heavy == 0) return;
  const float* sc = p.scores + ((size_t)row * p.kv_heads + g) * p.score_len + p.sink;
  const int n = L - p.sink - p.recent;  // > heavy
  // this CTA's run of candidates, and each warp's run of it (whole warps wide)
  const int run = ((n - 1) / (C * kSelThreads) + 1) * kSelThreads;
  const int c0 = (int)min((int64_t)rank * run, (int64_t)n), m = min(run, n - c0);
  sc += c0;
  auto key = [&](int i) { return i < p.held ? keys[i] : score_key(__ldg(sc + i)); };
  __syncthreads();  // hist is zero

  // first digit while the keys come in
  constexpr int U = 8;
  for (int i0 = tid; i0 < m; i0 += U * kSelThreads) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kSelThreads < m) x[u] = __ldg(sc + i0 + u * kSelThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kSelThreads;
      if (i < m) {
        const uint32_t k = score_key(x[u]);
        if (i < p.held) keys[i] = k;
        atomicAdd(&hist[k >> 21], 1u);
      }
    }
  }
  uint32_t prefix = 0, want = p.heavy;  // of the keys with this prefix, `want` are still to be chosen
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
    uint32_t* h = hist + d * kSelBins;
    if (d > 0) {
      for (int i = tid; i < m; i += kSelThreads) {
        const uint32_t k = key(i);
        if ((k >> (shift + bits)) == prefix) atomicAdd(&h[(k >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    // the cluster's counts of this thread's four digits, from the top
    uint4 b = make_uint4(0, 0, 0, 0);
    const int d0 = kSelBins - 4 * (tid + 1);
    if (C == 1) {
      __syncthreads();
      b = *reinterpret_cast<const uint4*>(h + d0);
    } else {
      cluster_sync();
      for (int q = 0; q < C; ++q) {
        const uint4 v = cluster_ld4(smem_u32(h + d0), q);
        b.x += v.x, b.y += v.y, b.z += v.z, b.w += v.w;
      }
    }
    uint32_t total;
    uint32_t above = block_exclusive(b.x + b.y + b.z + b.w, scan, total);
    const uint32_t bin[4] = {b.w, b.z, b.y, b.x};  // digits d0 + 3 .. d0
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (above < want && above + bin[e] >= want) {
        s_digit = d0 + 3 - e;
        s_want = want - above;
      }
      above += bin[e];
    }
    __syncthreads();
    prefix = (prefix << bits) | s_digit;
    want = s_want;
  }
  // prefix: the heavy-th largest key; `want` of the equal ones are taken
  const int wrun = ((m + kSelThreads - 1) / kSelThreads) * 32;
  const int w0 = min(warp * wrun, m), w1 = min(w0 + wrun, m);
  uint32_t gt = 0, eq = 0;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const uint32_t k = i0 + lane < w1 ? key(i0 + lane) : 0u;
    gt += __popc(__ballot_sync(kAll, i0 + lane < w1 && k > prefix));
    eq += __popc(__ballot_sync(kAll, i0 + lane < w1 && k == prefix));
  }
  if (lane == 0) {
    w_above[warp] = gt;
    w_equal[warp] = eq;
  }
  __syncthreads();
  uint32_t above = 0, equal = 0;  // keys before this warp's run
  if (C > 1) {
    if (tid == 0) {
      uint32_t a = 0, e = 0;
      for (int w = 0; w < kSelWarps; ++w) a += w_above[w], e += w_equal[w];
      s_count[0] = a;
      s_count[1] = e;
    }
    cluster_sync();
    for (int q = 0; q < rank; ++q) {
      const uint4 v = cluster_ld4(smem_u32(s_count), q);
      above += v.x;
      equal += v.y;
    }
    cluster_sync();  // no CTA leaves while another reads its counts
  }
  for (int w = 0; w < warp; ++w) {
    above += w_above[w];
    equal += w_equal[w];
  }
  uint32_t out = above + min(equal, want);
  const uint32_t before = (1u << lane) - 1;
  int32_t* to = keep + p.sink;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const bool in = i0 + lane < w1;
    const uint32_t k = in ? key(i0 + lane) : 0u;
    const uint32_t beq = __ballot_sync(kAll, in && k == prefix);
    const bool take = in && (k > prefix || (k == prefix && equal + __popc(beq & before) < want));
    const uint32_t bt = __ballot_sync(kAll, take);
    if (take) to[out + __popc(bt & before)] = p.sink + c0 + i0 + lane;
    out += __popc(bt);
    equal += __popc(beq);
  }
}

// ----------------------------------------------------------------------------
// In-place compaction: destination i, source keep[i] >= i.  A cluster of CTAs
// takes one 64-byte column of one head's K or V rows (or the head's scores)
// and walks the entries in order, kMoveChunk per CTA and step: all loads of a
// step, a barrier, its stores.  A store to place i can only overwrite a source
// read by an entry <= i (sources are never before their destinations), which
// is in this step or an earlier one, so no entry reads what another has
// written; for the same reason the next step's loads may be under way.
//
// Bound by HBM (2 * 64 bytes per entry and column), and before that by the
// chain of loads to an address: the entry, its block id, its row.  So the walk
// is a pipeline: while step c is stored, the rows of c+1, the block ids of c+2
// and the entries of c+3 are loaded.
constexpr int kMoveThreads = 256;
constexpr int kMoveLanes = 4;                          // 16-byte vectors of a column
constexpr int kMoveRows = kMoveThreads / kMoveLanes;   // rows side by side
constexpr int kMoveUnroll = 4;
constexpr int kMoveChunk = kMoveRows * kMoveUnroll;    // entries of a CTA and step

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
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int r = blockIdx.z, g = blockIdx.y, part = blockIdx.x / C;
  const int tid = threadIdx.x;
  MoveRange m;
  if (!move_range(p, r, m, tid == 0 && g == 0 && blockIdx.x == 0)) return;
  const int32_t* keep = p.keep + ((size_t)r * p.keep_heads + (p.keep_heads == 1 ? 0 : g)) * p.max_keep;
  const int room = m.L - m.base;
  // all loads of the step before its stores, in every CTA of the cluster
  auto meet = [&] {
    if (C == 1) __syncthreads();
    else cluster_sync();
  };

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
    constexpr int U = 8;
    const int step = C * U * kMoveThreads;
    for (int64_t i0 = 0; i0 < m.n; i0 += step) {
      float x[U];
      bool ok[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + (rank * U + u) * kMoveThreads + tid;
        const int src = i < m.n ? __ldg(keep + i) : -1;
        ok[u] = src >= i && src < room && i < m.n;
        if (ok[u]) x[u] = sc[src];
      }
      meet();
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (ok[u]) sc[i0 + (rank * U + u) * kMoveThreads + tid] = x[u];
    }
    meet();  // every source has been read
    for (int64_t i = (int64_t)m.n + rank * kMoveThreads + tid; i < room; i += C * kMoveThreads) sc[i] = 0.f;
    return;
  }

  const int is_v = part >= p.columns;
  const int col = (is_v ? part - p.columns : part) * kMoveLanes + tid % kMoveLanes;  // 16-byte vector of the head's row
  uint4* cache = reinterpret_cast<uint4*>(is_v ? p.v_cache : p.k_cache) + (size_t)g * p.row_vecs + col;
  const int32_t* table = p.tables + (size_t)r * p.maxblk;
  const size_t token_vecs = (size_t)p.kv_heads * p.row_vecs;
  const int shift = __ffs(p.block_size) - 1;  // a power of two
  // cache row of token t, or -1 (bad block id)
  auto slot_of = [&](int t) -> int {
    const int b = __ldg(table + (t >> shift));
    if (b < 0 || b >= p.num_blocks) {
      record_error(p.err, PA_DEVERR_BLOCK_ID);
      return -1;
    }
    return (b << shift) + (t & (p.block_size - 1));
  };
  const int steps = (m.n + C * kMoveChunk - 1) / (C * kMoveChunk);
  // entry u of this thread in step c
  auto entry = [&](int c, int u) { return (c * C + rank) * kMoveChunk + u * kMoveRows + tid / kMoveLanes; };
  // the source token of each entry, -1: none (past the end, in place already, or out of range)
  auto load_keep = [&](int c, int (&src)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = entry(c, u);
      src[u] = c < steps && i < m.n ? __ldg(keep + i) : -1;
    }
  };
  auto load_slots = [&](int c, const int (&src)[kMoveUnroll], int (&from)[kMoveUnroll], int (&to)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = entry(c, u);
      from[u] = to[u] = -1;
      if (c < steps && i < m.n && src[u] != i) {
        if (src[u] < i || src[u] >= room) {
          record_error(p.err, PA_DEVERR_KEEP);
        } else {
          from[u] = slot_of(m.base + src[u]);
          to[u] = slot_of(m.base + i);
          if (to[u] < 0) from[u] = -1;
        }
      }
    }
  };
  auto load_rows = [&](const int (&from)[kMoveUnroll], uint4 (&x)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (from[u] >= 0) x[u] = cache[(size_t)from[u] * token_vecs];
  };
  int src2[kMoveUnroll], src3[kMoveUnroll];            // entries of steps c+2, c+3
  int from0[kMoveUnroll], to0[kMoveUnroll];            // step c
  int from1[kMoveUnroll], to1[kMoveUnroll];            // step c+1
  uint4 x0[kMoveUnroll], x1[kMoveUnroll];
  load_keep(0, src2);
  load_keep(1, src3);
  load_slots(0, src2, from0, to0);
  load_rows(from0, x0);
  load_slots(1, src3, from1, to1);
  load_keep(2, src2);
  for (int c = 0; c < steps; ++c) {
    load_rows(from1, x1);
    load_keep(c + 3, src3);
    int from2[kMoveUnroll], to2[kMoveUnroll];
    load_slots(c + 2, src2, from2, to2);
    meet();  // every load of step c has been made
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      if (from0[u] >= 0) cache[(size_t)to0[u] * token_vecs] = x0[u];
      x0[u] = x1[u];
      from0[u] = from1[u], to0[u] = to1[u];
      from1[u] = from2[u], to1[u] = to2[u];
      src2[u] = src3[u];
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectParams& p0, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0) return cudaSuccess;
  EvictSelectParams p = p0;
  // CTAs per row: enough that each holds 8192 keys or fewer, as long as that
  // leaves no more than about four CTAs per SM in all (16: opt-in, for the few
  // long rows that would leave SMs idle)
  const int64_t rows = (int64_t)p.kv_heads * num_seqs, sms = num_sms() > 0 ? num_sms() : 152;
  int cluster = 1;
  while (cluster < 16 && (int64_t)cluster * 8192 < p.score_len && rows * cluster * 2 <= 4 * sms) cluster *= 2;
  while (cluster < 8 && (int64_t)cluster * kSelMaxHeld < p.score_len) cluster *= 2;
  const int64_t run = ((int64_t)p.score_len / ((int64_t)cluster * kSelThreads) + 1) * kSelThreads;
  p.held = (int)(run < kSelMaxHeld ? run : kSelMaxHeld);
  const size_t smem = (size_t)(3 * kSelBins + p.held) * 4;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (3 * kSelBins + kSelMaxHeld) * 4);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  return launch_pdl_cluster(evict_select_kernel, cluster, dim3((unsigned)(p.kv_heads * cluster), num_seqs),
                            dim3(kSelThreads), smem, stream, p);
}

cudaError_t launch_compact_kv(const CompactParams& p0, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0) return cudaSuccess;
  CompactParams p = p0;
  p.columns = p.row_vecs / kMoveLanes;
  const int parts = 2 * p.columns + (p.scores ? 1 : 0);
  // few sequences of long lists: clusters share a column, as long as that
  // leaves no more than four CTAs per SM and each has a step to take
  const int64_t ctas = (int64_t)parts * p.kv_heads * num_seqs, sms = num_sms() > 0 ? num_sms() : 152;
  int cluster = 1;
  while (cluster < 8 && ctas * cluster * 2 <= 4 * sms && (int64_t)cluster * kMoveChunk < p.max_keep) cluster *= 2;
  return launch_pdl_cluster(compact_kv_kernel, cluster, dim3((unsigned)(parts * cluster), p.kv_heads, num_seqs),
                            dim3(kMoveThreads), 0, stream, p);
}

}  // namespace pa
