// Choosing and moving the tokens a cache keeps, for sm_103a: pa_evict_select
// (per request and KV head, the tokens with the largest accumulated attention)
// and pa_compact_kv (the kept tokens moved together, in place).
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// Loads here are plain ones, not through the read-only path: scores, lists and
// lengths may come from the kernel before, which may still run when a CTA of
// these starts (they wait for it first).

// Order-preserving map of fp32 to uint32 (-0 equals +0, NaN below everything).
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 + 0 is +0
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return x == x ? k : 0u;
}

// A cluster of CTAs takes one (KV head, request), a CTA a run of its candidates
// [sink, L - recent), a warp a run of that.  The heavy-th largest key is found
// digit by digit (11, 11 and 10 bits from the top): a histogram per CTA, then
// the digit at which the count from above passes what is still wanted.  The
// 2048 digits are 16 slices.  In a cluster each slice has an owner to which the
// others add their non-empty digits (few: scores share a handful of exponents,
// and later digits only count keys of the chosen prefix), and every CTA adds
// its 16 slice sums to every other's, so one cluster barrier per digit does:
// a warp finds the slice in its CTA's sums and reads that slice's 128 digits
// from the owner.
//
// The keys are gone over three times: for the first digit; to list the keys of
// the chosen first digit, each warp its own (a few in a hundred: the other
// digits, and the counts of keys above and equal to the result, come from the
// list; a warp whose list does not hold them goes over its keys); and to write
// the indices in order, by ballots, each warp from the counts before it - of
// the equal keys the first ones.
// Bound by the instructions and atomics per key and the latency of the steps
// between (memory is 4 bytes per candidate): keys stay in shared memory as far
// as that leaves every CTA resident at once, and the rest are read again from
// L2.  Measured on GB300: 512 rows of 2300 keys 8.7 us, 64 of 85000 20 us, 8 of
// 131000 13 us; 64 of 32768 to 131009, where the longest row's CTAs decide (every
// row's cluster is the same), 34 us.  A range for the threshold from a sample of the row, to save
// most atomics, was slower: the sample's own steps cost more.
constexpr int kSelBins = 2048;
constexpr int kSelSlices = 16;
constexpr int kSelSlice = kSelBins / kSelSlices;     // 128 digits, four per lane
constexpr int kSelBatch = 8;                         // keys of a lane loaded together

// Shared memory in words before the lists and keys, for a cluster of C.
__host__ __device__ constexpr int select_words(int C) { return kSelBins + (C == 1 ? kSelBins : 3 * kSelBins / C); }

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) evict_select_kernel(const EvictSelectParams p) {
  constexpr int NW = THREADS / 32;
  extern __shared__ uint4 smem_raw[];
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int lc = 31 - __clz(C);  // C is a power of two
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem_raw);  // [kSelBins] this CTA's digits
  uint32_t* sums = hist + kSelBins;                        // the cluster's, of the slices it owns, per digit
  const int sums_stride = C == 1 ? 0 : kSelBins >> lc;
  uint32_t* lists = hist + select_words(C);                // [NW][p.warp_list] listed keys
  uint32_t* keys = lists + NW * p.warp_list;               // [NW][p.warp_held]
  __shared__ uint32_t slices[3][kSelSlices];               // the cluster's slice sums
  __shared__ __align__(16) uint32_t s_count[4];            // this CTA's keys above and equal to the result
  __shared__ uint32_t w_above[NW], w_equal[NW];
  __shared__ uint32_t s_want, s_prefix, s_before[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int zero = (kSelBins + (C == 1 ? 0 : 3 * sums_stride)) / 4;
  for (int i = tid; i < zero; i += THREADS) smem_raw[i] = make_uint4(0, 0, 0, 0);
  if (tid < 3 * kSelSlices) (&slices[0][0])[tid] = 0;
  // No early launch of the next kernel: keep_lens may be the context lengths
  // that one reads in its set-up.
  griddep_wait();
  const int r = blockIdx.y, g = blockIdx.x >> lc;
  const int budget = p.sink + p.heavy + p.recent;
  int32_t* keep = p.keep + ((size_t)r * p.kv_heads + g) * budget;
  const int row = p.score_rows ? p.score_rows[r] : r;
  const int L = p.lens[r];
  const int t0 = rank * THREADS + tid, tn = C * THREADS;  // this thread among the cluster's
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
  const int run = (((n - 1) / THREADS >> lc) + 1) * THREADS;
  const int c0 = (int)min((int64_t)rank * run, (int64_t)n), m = min(run, n - c0);
  sc += c0;
  const int wrun = ((m + THREADS - 1) / THREADS) * 32;
  const int w0 = min(warp * wrun, m), w1 = min(w0 + wrun, m);
  // the first keys of the run stay in shared memory, in multiples of a batch:
  // every warp reads its share of the others again
  uint32_t* held = keys + warp * p.warp_held - w0;
  const int h1 = w0 + p.warp_held;
  // f(k, place, in) for each key of the warp's run, 32 at a time, in order; the
  // run's whole batches in shared memory take the short way (in: true)
  auto each_key = [&](auto&& f) {
    int i0 = w0;
    const int fast = min(w1, h1) - 32 * kSelBatch;
    for (; i0 <= fast; i0 += 32 * kSelBatch) {
      uint32_t k[kSelBatch];
#pragma unroll
      for (int u = 0; u < kSelBatch; ++u) k[u] = held[i0 + 32 * u + lane];
#pragma unroll
      for (int u = 0; u < kSelBatch; ++u) f(k[u], i0 + 32 * u + lane, true);
    }
    for (; i0 < w1; i0 += 32 * kSelBatch) {
      uint32_t k[kSelBatch];
#pragma unroll
      for (int u = 0; u < kSelBatch; ++u) {
        const int i = i0 + 32 * u + lane;
        k[u] = i >= w1 ? 0u : i < h1 ? held[i] : score_key(sc[i]);
      }
#pragma unroll
      for (int u = 0; u < kSelBatch; ++u)
        if (i0 + 32 * u < w1) f(k[u], i0 + 32 * u + lane, i0 + 32 * u + lane < w1);
    }
  };
  if (C == 1) __syncthreads();  // the counts are zero, in every CTA
  else cluster_sync();

  // first digit while the keys come in
  for (int i0 = w0; i0 < w1; i0 += 32 * kSelBatch) {
    float x[kSelBatch];
    if (i0 + 32 * kSelBatch <= min(w1, h1)) {
#pragma unroll
      for (int u = 0; u < kSelBatch; ++u) x[u] = sc[i0 + 32 * u + lane];
#pragma unroll
      for (int u = 0; u < kSelBatch; ++u) {
        const uint32_t k = score_key(x[u]);
        held[i0 + 32 * u + lane] = k;
        atomicAdd(&hist[k >> 21], 1u);
      }
      continue;
    }
#pragma unroll
    for (int u = 0; u < kSelBatch; ++u)
      if (i0 + 32 * u + lane < w1) x[u] = sc[i0 + 32 * u + lane];
#pragma unroll
    for (int u = 0; u < kSelBatch; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i0 + 32 * u >= w1) break;
      if (i < w1) {
        const uint32_t k = score_key(x[u]);
        if (i < h1) held[i] = k;
        atomicAdd(&hist[k >> 21], 1u);
      }
    }
  }
  uint32_t prefix = 0, want = p.heavy;  // of the keys with this prefix, `want` are still to be chosen
  uint32_t gt = 0;                      // this lane's keys above the first digit
  uint32_t* list = lists + warp * p.warp_list;
  int listed = p.warp_list + 1;         // this warp's keys of the first digit; more than fit: not listed
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
    if (d == 1) {
      listed = 0;
      each_key([&](uint32_t k, int, bool in) {
        gt += (k >> 21) > prefix;  // a key behind the end is 0: not above anything
        const bool same = in && (k >> 21) == prefix;
        if (same) atomicAdd(&hist[(k >> 10) & 2047u], 1u);
        const uint32_t eq = __ballot_sync(kAll, same);
        const int at = listed + __popc(eq & ((1u << lane) - 1));
        if (same && at < p.warp_list) list[at] = k;
        listed += __popc(eq);
      });
      __syncwarp();
    } else if (d == 2) {
      if (listed <= p.warp_list) {
        for (int j = lane; j < listed; j += 32)
          if ((list[j] >> 10) == prefix) atomicAdd(&hist[list[j] & 1023u], 1u);
      } else {
        each_key([&](uint32_t k, int, bool in) {
          if (in && (k >> 10) == prefix) atomicAdd(&hist[k & 1023u], 1u);
        });
      }
    }
    __syncthreads();
    // a warp's slices of this CTA's digits, four of them in each lane
    for (int sl = warp; sl < kSelSlices; sl += NW) {
      uint4* mine = reinterpret_cast<uint4*>(hist + sl * kSelSlice) + lane;
      const uint4 v = *mine;
      *mine = make_uint4(0, 0, 0, 0);  // for the next digit
      const uint32_t sum = __reduce_add_sync(kAll, v.x + v.y + v.z + v.w);
      uint32_t* total = sums + d * sums_stride + (sl >> lc) * kSelSlice + 4 * lane;
      if (C == 1) {
        *reinterpret_cast<uint4*>(total) = v;
        if (lane == 0) slices[d][sl] = sum;
      } else {
        const uint32_t at = smem_u32(total), owner = sl & (C - 1);
        if (v.x) cluster_add(at, owner, v.x);
        if (v.y) cluster_add(at + 4, owner, v.y);
        if (v.z) cluster_add(at + 8, owner, v.z);
        if (v.w) cluster_add(at + 12, owner, v.w);
        if (lane < C && sum) cluster_add(smem_u32(&slices[d][sl]), lane, sum);
      }
    }
    if (C == 1) __syncthreads();
    else cluster_sync();
    // one warp (all of them would meet at the slice's owner), counting from the
    // top: lane l has slices 15 .. 15 - l
    if (warp == 0) {
      uint32_t upto = 0, sl = 0;  // the keys of the first lane + 1 slices, of the last of them
#pragma unroll
      for (int j = 0; j < kSelSlices; ++j) {
        const uint32_t x = slices[d][kSelSlices - 1 - j];
        if (j <= lane) upto += x;
        if (j == lane) sl = x;
      }
      const int hit = __ffs(__ballot_sync(kAll, upto >= want)) - 1;  // one of the 16: they hold all
      want -= __shfl_sync(kAll, upto - sl, hit);
      const int slice = kSelSlices - 1 - hit;
      // its digits, lane l: the four below 128 - 4 l
      const uint32_t* from = sums + d * sums_stride + (slice >> lc) * kSelSlice + kSelSlice - 4 * (lane + 1);
      const uint4 q = C == 1 ? *reinterpret_cast<const uint4*>(from) : cluster_ld4(smem_u32(from), slice & (C - 1));
      const uint32_t four = q.x + q.y + q.z + q.w;
      upto = four;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += y;
      }
      const int at = __ffs(__ballot_sync(kAll, upto >= want)) - 1;
      // which of its four digits, lane `at`'s is wanted (selects: a divergent
      // branch before a shuffle costs a thousand clocks here)
      const uint32_t a0 = upto - four, a1 = a0 + q.w, a2 = a1 + q.z, a3 = a2 + q.y;
      const int e = (a1 < want) + (a2 < want) + (a3 < want);
      const uint32_t above = e == 0 ? a0 : e == 1 ? a1 : e == 2 ? a2 : a3;
      const uint32_t keys_of = e == 0 ? q.w : e == 1 ? q.z : e == 2 ? q.y : q.x;
      const uint32_t next = (prefix << bits) | (uint32_t)(slice * kSelSlice + kSelSlice - 1 - 4 * lane - e);
      // all keys of the digit are taken: the last key below them does for T, none equal to it taken
      const bool all = want - above == keys_of;
      if (lane == at) {
        s_want = all ? 0u : want - above;
        s_prefix = all ? (next << shift) - 1 : next;
      }
    }
    __syncthreads();
    want = s_want;
    prefix = s_prefix;
    if (want == 0) break;
  }
  // prefix: T, the heavy-th largest key, and `want` of the keys equal to it are
  // taken (none, where it was enough to know the keys above)
  uint32_t eq = 0;
  if (listed <= p.warp_list) {
    gt = __reduce_add_sync(kAll, gt);
    for (int j0 = 0; j0 < listed; j0 += 32) {
      const uint32_t k = list[min(j0 + lane, p.warp_list - 1)];
      gt += __popc(__ballot_sync(kAll, j0 + lane < listed && k > prefix));
      eq += __popc(__ballot_sync(kAll, j0 + lane < listed && k == prefix));
    }
  } else {
    gt = 0;
    each_key([&](uint32_t k, int, bool in) {
      gt += __popc(__ballot_sync(kAll, in && k > prefix));
      eq += __popc(__ballot_sync(kAll, in && k == prefix));
    });
  }
  if (lane == 0) {
    w_above[warp] = gt;
    w_equal[warp] = eq;
  }
  __syncthreads();
  // keys before this warp's run: lane w holds warp w's, then lane q CTA q's
  const uint32_t wa = lane < NW ? w_above[lane] : 0u, we = lane < NW ? w_equal[lane] : 0u;
  uint32_t above = __reduce_add_sync(kAll, lane < warp ? wa : 0u);
  uint32_t equal = __reduce_add_sync(kAll, lane < warp ? we : 0u);
  if (C > 1) {
    const uint32_t a = __reduce_add_sync(kAll, wa), e = __reduce_add_sync(kAll, we);
    if (tid == 0) {
      s_count[0] = a;
      s_count[1] = e;
    }
    cluster_sync();
    if (warp == 0) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (lane < rank) v = cluster_ld4(smem_u32(s_count), lane);
      v.x = __reduce_add_sync(kAll, v.x);
      v.y = __reduce_add_sync(kAll, v.y);
      if (lane == 0) s_before[0] = v.x, s_before[1] = v.y;
    }
    cluster_sync();  // no CTA leaves while another reads its counts
    above += s_before[0];
    equal += s_before[1];
  }
  const uint32_t out = above + min(equal, want);
  const uint32_t before = (1u << lane) - 1;
  int32_t* to = keep + p.sink;
  to += out;
  each_key([&](uint32_t k, int i, bool in) {
    uint32_t bt = __ballot_sync(kAll, in && k > prefix);
    const uint32_t beq = __ballot_sync(kAll, in && k == prefix);
    if (beq) {  // the first ones of the equal keys
      bt |= __ballot_sync(kAll, ((beq >> lane) & 1) && equal + __popc(beq & before) < want);
      equal += __popc(beq);
    }
    if ((bt >> lane) & 1) to[__popc(bt & before)] = p.sink + c0 + i;
    to += __popc(bt);
  });
}

template <int THREADS>
cudaError_t launch_select_t(EvictSelectParams& p, int cluster, int num_seqs, cudaStream_t stream) {
  auto kern = evict_select_kernel<THREADS>;
  constexpr int kMost = 224 * 1024;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  // keys held: as many as leave room for every CTA at once
  const int64_t sms = num_sms() > 0 ? num_sms() : 152;
  int64_t per_sm = ((int64_t)p.kv_heads * num_seqs * cluster + sms - 1) / sms;
  if (per_sm > 2048 / THREADS) per_sm = 2048 / THREADS;
  const int64_t run = ((int64_t)p.score_len / ((int64_t)cluster * THREADS) + 1) * THREADS;  // at most, of a CTA
  // lists: a quarter of a warp's run and a little, 32 KB in all at most
  constexpr int NW = THREADS / 32;
  const int64_t quarter = run / (4 * NW) + 32;
  p.warp_list = (int)(quarter < 8192 / NW ? quarter : 8192 / NW);
  const int64_t room = (kMost / per_sm - 4096) / 4 - select_words(cluster) - NW * p.warp_list;
  const int64_t batches = (run / NW + 32 * kSelBatch - 1) / (32 * kSelBatch);  // of a warp
  const int64_t fit = room < 0 ? 0 : room / (NW * 32 * kSelBatch);
  p.warp_held = (int)(batches < fit ? batches : fit) * 32 * kSelBatch;
  const size_t smem = (size_t)(select_words(cluster) + NW * (p.warp_list + p.warp_held)) * 4;
  return launch_pdl_cluster(kern, cluster, dim3((unsigned)(p.kv_heads * cluster), num_seqs), dim3(THREADS), smem,
                            stream, p);
}

// ----------------------------------------------------------------------------
// In-place compaction: destination i, source keep[i] >= i.  A cluster of CTAs
// takes one column (64 or 128 bytes) of one head's K or V rows and walks the
// entries in order, a step at a time: all loads of a step, a barrier, its
// stores.  A store to place i can only overwrite a source read by an entry
// <= i (sources are never before their destinations), which is in this step or
// an earlier one, so no entry reads what another has written; for the same
// reason the next steps' loads may be under way.
//
// Bound by HBM (twice the column per entry), and before that by the chain of
// loads to an address: the entry, its block id, its row.  So the walk is a
// pipeline: while step c is stored, the rows of c+1 and c+2 are on their way
// into shared memory (cp.async: no registers), and the block ids of c+3 and the
// entries of c+4 into registers; every load is made a step before its value is
// used.  Measured on GB300, 8 heads of 128: 8 lists of 8192 per head (537 MB)
// 93 us, 0.85 of the copy rate; one 18 us.
constexpr int kMoveThreads = 256;                      // of the one-step kernel
constexpr int kMoveUnroll = 4;
constexpr int kMoveStages = 3;
constexpr int kMoveSmall = 64;                         // longest list of the one-step kernel

struct MoveRange {
  int base, n, L;
};

// The request's range, checked; false: nothing is moved.  PAST_L1: see compact_scores_kernel.
template <bool PAST_L1 = false>
__device__ __forceinline__ bool move_range(const CompactParams& p, int r, MoveRange& m, bool report) {
  m.L = PAST_L1 ? __ldcg(p.lens + r) : p.lens[r];
  m.n = PAST_L1 ? __ldcg(p.keep_lens + r) : p.keep_lens[r];
  m.base = !p.base ? 0 : PAST_L1 ? __ldcg(p.base + r) : p.base[r];
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

template <int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) compact_kv_kernel(const CompactParams p) {
  constexpr int kMoveThreads = THREADS, kMoveLanes = LANES;
  constexpr int kMoveRows = kMoveThreads / kMoveLanes;   // rows side by side
  constexpr int kMoveChunk = kMoveRows * kMoveUnroll;    // entries of a CTA and step
  extern __shared__ uint4 smem_raw[];
  uint4 (*ring)[kMoveUnroll][kMoveThreads] = reinterpret_cast<uint4 (*)[kMoveUnroll][kMoveThreads]>(smem_raw);
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
      src[u] = c < steps && i < m.n ? keep[i] : i;
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

// The scores of a (KV head, request), moved by the same rule, and zeros behind
// them.  A launch of its own: inside the kernel above the columns that also
// moved scores were the last to end (8 lists of 8192 per head over contexts of
// 80000: 124 us; apart, 93 and 7).  A cluster shares a long row: one SM's stores
// alone take 14 us for the zeros of a context of 131000.
constexpr int kScoreThreads = 256;

__device__ __forceinline__ void move_scores(const CompactParams& p) {
  const int C = (int)cluster_size(), rank = (int)cluster_rank();
  const int r = blockIdx.y, g = blockIdx.x / C, tid = threadIdx.x;
  auto meet = [&] {
    if (C == 1) __syncthreads();
    else cluster_sync();
  };
  MoveRange m;
  if (!move_range<true>(p, r, m, false)) return;  // reported by the rows' kernel
  const int row = p.score_rows ? __ldcg(p.score_rows + r) : r;
  if (row < 0) return;
  bool twice = false;  // an earlier request has this row: its alone are moved
  if (p.score_rows)
    for (int i = tid; i < r; i += kScoreThreads) twice |= __ldcg(p.score_rows + i) == row;
  const bool bad = __syncthreads_or(twice) || row >= p.num_rows;
  if (bad || m.L > p.score_len) {
    if (tid == 0) record_error(p.err, bad ? PA_DEVERR_SCORE_ROW : PA_DEVERR_CONTEXT_LEN);
    return;
  }
  const int32_t* keep = p.keep + ((size_t)r * p.keep_heads + (p.keep_heads == 1 ? 0 : g)) * p.max_keep;
  const int room = m.L - m.base;
  float* sc = p.scores + ((size_t)row * p.kv_heads + g) * p.score_len + m.base;
  constexpr int U = 8;
  for (int64_t c = 0; c < m.n; c += C * U * kScoreThreads) {
    const int64_t i0 = c + rank * U * kScoreThreads + tid;
    int src[U];
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + u * kScoreThreads;
      src[u] = i < m.n ? __ldcg(keep + i) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (src[u] < i0 + u * kScoreThreads || src[u] >= room) src[u] = -1;
      if (src[u] >= 0) x[u] = __ldcg(sc + src[u]);
    }
    meet();  // all loads of the step before its stores
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (src[u] >= 0) sc[i0 + u * kScoreThreads] = x[u];
  }
  meet();  // every score has been read
  // zeros on [n, room): single ones up to a 16-byte boundary, then vectors
  const int t0 = rank * kScoreThreads + tid;
  const int n4 = min(m.n + (int)((16 - (reinterpret_cast<uintptr_t>(sc + m.n) & 15)) / 4) % 4, room);
  if (t0 < n4 - m.n) sc[m.n + t0] = 0.f;
  const int vecs = (room - n4) / 4;
  for (int64_t i = t0; i < vecs; i += C * kScoreThreads)
    reinterpret_cast<float4*>(sc + n4)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (t0 < room - n4 - 4 * vecs) sc[n4 + 4 * vecs + t0] = 0.f;
}

// Runs beside the rows' kernel, with which it shares nothing that either
// writes: it starts when every CTA of that kernel has started (and so has
// waited for all that came before), and waits for its end before its own, so
// that what follows finds both done (8 lists of 8192: 101 us for both, 109 one
// after the other; one list 20 and 25).  Its loads go past L1, whose lines may be
// older than that.
__global__ void __launch_bounds__(kScoreThreads) compact_scores_kernel(const CompactParams p) {
  move_scores(p);
  griddep_wait();
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
      const int src = keep[i];
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
  // One CTA per SM: clusters of up to 8 share a row while there are SMs for
  // them and a thousand keys for each CTA.  A second CTA on an SM only halves
  // both (an earlier form, 64 rows of 85000 keys: clusters of 2, 4, 8 of 1024
  // threads 30, 42, 80 us; of 512 threads 41, 34, 56).  More rows than SMs: small
  // CTAs, the steps between the keys cost what short rows do (512 rows of 2300:
  // 256 threads 8.7 us, 512 12.7, 1024 22.5).
  const int64_t rows = (int64_t)p.kv_heads * num_seqs, sms = num_sms() > 0 ? num_sms() : 152;
  int cluster = 1;
  while (cluster < 8 && rows * cluster * 2 <= sms && (int64_t)cluster * 1024 < p.score_len) cluster *= 2;
  const int64_t per_cta = (p.score_len + cluster - 1) / cluster;
  if (rows * cluster > sms && per_cta <= 8192) return launch_select_t<256>(p, cluster, num_seqs, stream);
  return per_cta <= 2048 ? launch_select_t<512>(p, cluster, num_seqs, stream)
                         : launch_select_t<1024>(p, cluster, num_seqs, stream);
}

template <int LANES, int THREADS>
cudaError_t launch_move_t(CompactParams& p, int num_seqs, cudaStream_t stream) {
  auto kern = compact_kv_kernel<LANES, THREADS>;
  constexpr int SMEM = kMoveStages * kMoveUnroll * THREADS * 16;
  constexpr int CHUNK = THREADS / LANES * kMoveUnroll;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  p.columns = p.row_vecs / LANES;
  // few sequences of long lists: clusters share a column, as long as that
  // leaves no more than 1024 threads per SM and each CTA has a step to take
  const int64_t threads = 2 * (int64_t)p.columns * p.kv_heads * num_seqs * THREADS;
  const int64_t sms = num_sms() > 0 ? num_sms() : 152;
  int cluster = 1;
  while (cluster < 8 && threads * cluster * 2 <= 1024 * sms && (int64_t)cluster * CHUNK < p.max_keep) cluster *= 2;
  return launch_pdl_cluster(kern, cluster, dim3((unsigned)(2 * p.columns * cluster), p.kv_heads, num_seqs),
                            dim3(THREADS), SMEM, stream, p);
}

cudaError_t launch_compact_kv(const CompactParams& p0, int num_seqs, cudaStream_t stream) {
  if (num_seqs == 0) return cudaSuccess;
  CompactParams p = p0;
  cudaError_t e;
  // 128-byte columns, whole lines, when they fill the GPU: 512 threads while
  // every CTA fits at once (8 lists of 8192 per head: 93 us; 256 threads 112,
  // 64-byte columns 102), 256 when they do not (64 lists of 1024: 86; 512
  // threads 99, 64-byte columns 92).  Fewer: 64-byte columns, twice the CTAs
  // (one list: 18; 128-byte columns 21 to 28).
  const int64_t ctas = (int64_t)p.row_vecs / 4 * p.kv_heads * num_seqs, sms = num_sms() > 0 ? num_sms() : 152;
  const dim3 lists(p.kv_heads, num_seqs);
  if (p.max_keep <= kMoveSmall)
    e = p.row_vecs == 16 ? launch_pdl(compact_small_kernel<16>, lists, dim3(kMoveThreads), 0, stream, p)
                         : launch_pdl(compact_small_kernel<8>, lists, dim3(kMoveThreads), 0, stream, p);
  else if (ctas <= sms)
    e = launch_move_t<4, 256>(p, num_seqs, stream);
  else if (ctas <= 2 * sms)
    e = launch_move_t<8, 512>(p, num_seqs, stream);
  else
    e = launch_move_t<8, 256>(p, num_seqs, stream);
  if (e != cudaSuccess || !p.scores) return e;
  const int64_t rows = (int64_t)p.kv_heads * num_seqs;
  int cluster = 1;
  while (cluster < 8 && rows * cluster * 2 <= 4 * sms && (int64_t)cluster * 8 * kScoreThreads < p.score_len) cluster *= 2;
  return launch_pdl_cluster(compact_scores_kernel, cluster, dim3((unsigned)(p.kv_heads * cluster), num_seqs),
                            dim3(kScoreThreads), 0, stream, p);
}

}  // namespace pa
