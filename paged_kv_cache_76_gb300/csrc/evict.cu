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

// A cluster of CTAs takes one (KV head, request): each holds its part of the
// row's keys in shared memory, read once.  The heavy-th largest key of the
// candidates [sink, L - recent) is found digit by digit (11, 11 and 10 bits
// from the top): a histogram per CTA, then the digit at which the count from
// above passes what is still wanted.  The 2048 digits are 16 slices.  In a
// cluster each slice has an owner to which the others add their non-empty
// digits (few: scores share a handful of exponents, and later digits only
// count keys of the chosen prefix), and every CTA adds its 16 slice sums to
// every other's, so one cluster barrier per digit does: each CTA then finds the
// slice in its own sums and reads that slice's 128 digits from the owner.
// Then every warp counts its run of keys above and equal to the result, the
// counts before a warp give its place in the list, and it writes the indices
// in order by ballots; of the equal keys the first ones.
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;
constexpr int kSelSlices = 16;                       // one per warp
constexpr int kSelSlice = kSelBins / kSelSlices;     // four digits per lane
static_assert(kSelSlices == kSelWarps && kSelSlice == 128, "a warp sums a slice");
constexpr int kSelMaxHeld = 40960;  // keys of a CTA in shared memory; the rest are read again

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictSelectParams p) {
  extern __shared__ uint4 smem_raw[];
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem_raw);  // [kSelBins] this CTA's digits
  uint32_t* sums = hist + kSelBins;                        // [3][kSelBins] the cluster's, of the slices it owns
  uint32_t* keys = sums + 3 * kSelBins;                    // [held]
  __shared__ uint32_t slices[3][kSelSlices];               // the cluster's slice sums
  __shared__ __align__(16) uint32_t s_count[4];            // this CTA's keys above and equal to the threshold
  __shared__ uint32_t w_above[kSelWarps], w_equal[kSelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kSelBins; i += kSelThreads) smem_raw[i] = make_uint4(0, 0, 0, 0);  // hist and sums
  if (tid < 3 * kSelSlices) (&slices[0][0])[tid] = 0;
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
  if (C == 1) __syncthreads();  // the counts are zero, in every CTA
  else cluster_sync();

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
    if (d > 0) {
      for (int i = tid; i < m; i += kSelThreads) {
        const uint32_t k = key(i);
        if ((k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1)], 1u);
      }
    }
    __syncthreads();
    // slice `warp` of this CTA's digits, four of them in each lane
    uint32_t* mine = hist + warp * kSelSlice + 4 * lane;
    const uint4 v = *reinterpret_cast<const uint4*>(mine);
    *reinterpret_cast<uint4*>(mine) = make_uint4(0, 0, 0, 0);  // for the next digit
    const uint32_t sum = __reduce_add_sync(kAll, v.x + v.y + v.z + v.w);
    uint32_t* total = sums + d * kSelBins;  // [kSelBins]
    if (C == 1) {
      *reinterpret_cast<uint4*>(total + warp * kSelSlice + 4 * lane) = v;
      if (lane == 0) slices[d][warp] = sum;
      __syncthreads();
    } else {
      const uint32_t at = smem_u32(total + warp * kSelSlice + 4 * lane), owner = warp % C;
      if (v.x) cluster_add(at, owner, v.x);
      if (v.y) cluster_add(at + 4, owner, v.y);
      if (v.z) cluster_add(at + 8, owner, v.z);
      if (v.w) cluster_add(at + 12, owner, v.w);
      if (lane < C && sum) cluster_add(smem_u32(&slices[d][warp]), lane, sum);
      cluster_sync();
    }
    // every warp: lane l holds slice 15 - l, so that a scan counts from the top
    const uint32_t sl = lane < kSelSlices ? slices[d][kSelSlices - 1 - lane] : 0u;
    uint32_t upto = sl;
#pragma unroll
    for (int o = 1; o < kSelSlices; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += y;
    }
    const int hit = __ffs(__ballot_sync(kAll, upto >= want)) - 1;  // one of the 16: they hold all
    want -= __shfl_sync(kAll, upto - sl, hit);
    const int slice = kSelSlices - 1 - hit;
    // its digits, lane l: the four below 128 - 4 l
    const uint32_t q0 = smem_u32(total + slice * kSelSlice + kSelSlice - 4 * (lane + 1));
    const uint4 q = C == 1 ? *reinterpret_cast<const uint4*>(total + slice * kSelSlice + kSelSlice - 4 * (lane + 1))
                           : cluster_ld4(q0, slice % C);
    const uint32_t four = q.x + q.y + q.z + q.w;
    upto = four;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += y;
    }
    const int at = __ffs(__ballot_sync(kAll, upto >= want)) - 1;
    uint32_t above = upto - four, digit = slice * kSelSlice + kSelSlice - 1 - 4 * lane;  // lane `at`'s are wanted
    if (above + q.w < want) {
      above += q.w;
      --digit;
      if (above + q.z < want) {
        above += q.z;
        --digit;
        if (above + q.y < want) {
          above += q.y;
          --digit;
        }
      }
    }
    want -= __shfl_sync(kAll, above, at);
    prefix = (prefix << bits) | __shfl_sync(kAll, digit, at);
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
    if (lane < rank) {  // C <= 16: a lane per CTA before this one
      const uint4 v = cluster_ld4(smem_u32(s_count), lane);
      above = v.x;
      equal = v.y;
    }
    above = __reduce_add_sync(kAll, above);
    equal = __reduce_add_sync(kAll, equal);
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
// is a pipeline: while step c is stored, the rows of c+1 and c+2 are on their
// way into shared memory (cp.async: no registers, four CTAs on an SM), and the
// block ids of c+3 and the entries of c+4 into registers.
constexpr int kMoveThreads = 256;
constexpr int kMoveLanes = 4;                          // 16-byte vectors of a column
constexpr int kMoveRows = kMoveThreads / kMoveLanes;   // rows side by side
constexpr int kMoveUnroll = 4;
constexpr int kMoveChunk = kMoveRows * kMoveUnroll;    // entries of a CTA and step
constexpr int kMoveStages = 3;
constexpr int kMoveSmall = 64;                         // longest list of the one-step kernel

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

__global__ void __launch_bounds__(kMoveThreads, 4) compact_kv_kernel(const CompactParams p) {
  __shared__ uint4 ring[kMoveStages][kMoveUnroll][kMoveThreads];
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
  const int steps = (m.n + C * kMoveChunk - 1) / (C * kMoveChunk);
  // entry u of this thread in step c
  auto entry = [&](int c, int u) { return (c * C + rank) * kMoveChunk + u * kMoveRows + tid / kMoveLanes; };
  // Every load is made a step before its value is used.
  // the source token of each entry of step c (past the end: its own place)
  auto load_keep = [&](int c, int (&src)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = entry(c, u);
      src[u] = c < steps && i < m.n ? __ldg(keep + i) : i;
    }
  };
  // block ids of the entries to move and of their places; `src` becomes -1
  // where there is nothing to move or the entry is refused
  auto load_ids = [&](int c, int (&src)[kMoveUnroll], int (&from)[kMoveUnroll]) {
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = entry(c, u), t = src[u];
      const bool in = t >= i && t < room;
      bad |= t != i && !in;
      src[u] = t != i && in ? m.base + t : -1;
      from[u] = src[u] >= 0 ? __ldg(table + (src[u] >> shift)) : 0;
    }
    if (bad) record_error(p.err, PA_DEVERR_KEEP);
  };
  auto load_to = [&](int c, int (&to)[kMoveUnroll]) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = entry(c, u);
      to[u] = c < steps && i < m.n ? __ldg(table + ((m.base + i) >> shift)) : 0;
    }
  };
  uint32_t moves = 0;  // four bits per step in the ring: the entries to store
  auto load_rows = [&](int c, const int (&src)[kMoveUnroll], const int (&from)[kMoveUnroll]) {
    moves <<= 4;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const bool in = from[u] >= 0 && from[u] < p.num_blocks;
      bad |= !in;
      if (src[u] >= 0 && in) {
        const size_t row = (size_t)from[u] * p.block_size + (src[u] & (p.block_size - 1));
        cp_async16(smem_u32(&ring[c % kMoveStages][u][tid]), cache + row * token_vecs, 16u);
        moves |= 1u << u;
      }
    }
    if (bad) record_error(p.err, PA_DEVERR_BLOCK_ID);
    cp_async_commit();
  };
  int src[kMoveUnroll], from[kMoveUnroll], next[kMoveUnroll], to[kMoveUnroll];
  load_keep(0, src);
  load_keep(1, next);
  load_ids(0, src, from);
  load_to(0, to);
  load_rows(0, src, from);
  load_ids(1, next, from);
  load_keep(2, src);
  load_rows(1, next, from);
  load_ids(2, src, from);
  load_keep(3, next);
  for (int c = 0; c < steps; ++c) {
    load_rows(c + 2, src, from);  // into the stage of step c - 1, whose rows this thread has stored
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) src[u] = next[u];
    load_ids(c + 3, src, from);
    load_keep(c + 4, next);
    cp_async_wait<2>();  // step c's rows are here
    meet();              // ... in every CTA
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const bool in = to[u] >= 0 && to[u] < p.num_blocks;
      if ((moves >> (8 + u)) & 1) {
        bad |= !in;
        const size_t row = (size_t)to[u] * p.block_size + ((m.base + entry(c, u)) & (p.block_size - 1));
        if (in) cache[row * token_vecs] = ring[c % kMoveStages][u][tid];
      }
    }
    if (bad) record_error(p.err, PA_DEVERR_BLOCK_ID);
    load_to(c + 1, to);
  }
  cp_async_wait_all();
}

// Lists of at most kMoveSmall entries (a tree's accepted path): a CTA takes a
// head's K and V rows whole, all loads, a barrier, all stores.  Bound by the
// launch and one chain of loads.
template <int VECS>
__global__ void __launch_bounds__(kMoveThreads) compact_small_kernel(const CompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.y, g = blockIdx.x, tid = threadIdx.x;
  MoveRange m;
  if (!move_range(p, r, m, tid == 0 && g == 0)) return;
  constexpr int ROWS = kMoveThreads / VECS;            // rows side by side
  constexpr int U = kMoveSmall / ROWS;
  const int32_t* keep = p.keep + ((size_t)r * p.keep_heads + (p.keep_heads == 1 ? 0 : g)) * p.max_keep;
  const int room = m.L - m.base;
  const int32_t* table = p.tables + (size_t)r * p.maxblk;
  const int shift = __ffs(p.block_size) - 1;
  const size_t token_vecs = (size_t)p.kv_heads * VECS;
  const size_t at = (size_t)g * VECS + tid % VECS;
  uint4* kc = reinterpret_cast<uint4*>(p.k_cache) + at;
  uint4* vc = reinterpret_cast<uint4*>(p.v_cache) + at;
  auto slot_of = [&](int t) -> int {
    const int b = __ldg(table + (t >> shift));
    if (b < 0 || b >= p.num_blocks) {
      record_error(p.err, PA_DEVERR_BLOCK_ID);
      return -1;
    }
    return (b << shift) + (t & (p.block_size - 1));
  };
  uint4 xk[U], xv[U];
  int to[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = u * ROWS + tid / VECS;
    to[u] = -1;
    if (i < m.n) {
      const int src = __ldg(keep + i);
      if (src < i || src >= room) {
        record_error(p.err, PA_DEVERR_KEEP);
      } else if (src != i) {
        const int from = slot_of(m.base + src);
        to[u] = slot_of(m.base + i);
        if (from < 0) to[u] = -1;
        if (to[u] >= 0) {
          xk[u] = kc[(size_t)from * token_vecs];
          xv[u] = vc[(size_t)from * token_vecs];
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (to[u] >= 0) {
      kc[(size_t)to[u] * token_vecs] = xk[u];
      vc[(size_t)to[u] * token_vecs] = xv[u];
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
  const size_t smem = (size_t)(4 * kSelBins + p.held) * 4;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (4 * kSelBins + kSelMaxHeld) * 4);
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
  if (p.max_keep <= kMoveSmall && !p.scores)
    return p.row_vecs == 16 ? launch_pdl(compact_small_kernel<16>, dim3(p.kv_heads, num_seqs), dim3(kMoveThreads), 0,
                                         stream, p)
                            : launch_pdl(compact_small_kernel<8>, dim3(p.kv_heads, num_seqs), dim3(kMoveThreads), 0,
                                         stream, p);
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
