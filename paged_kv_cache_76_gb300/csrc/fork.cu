// Pages of the cache shared, copied, taken and given back on the device:
// pa_fork_blocks (Block Tables of sequences that go on from others) and
// pa_copy_pages (the copies it asks for, in any number of caches).
//
// fork_blocks keeps no counts from call to call.  What a page is, follows from
// the tables that go on: state[b] of block b is
//   kFree  no new row holds it (kPinned: and it is pinned);
//   i >= 0 only rows that go on writing inside it hold it, i the first of them:
//          row i keeps it, the others get copies;
//   kHeld  some row holds it and does not write inside it: writers get copies.
// A holder that does not write stores kHeld, a writer takes the minimum with its
// row, so the order of either does not change what comes out, and nothing but
// one word per writing row is atomic.  Then free pages (kFree and not pinned) go
// to the rows in order of their number, so equal calls give equal tables.
//
//   clear   state = kFree
//   mark    a warp per (old row, 512 columns): if a new row goes on from it, its
//           blocks; the pages that new rows write in
//   count   free pages of each warp's span of blocks; pages that each row needs,
//           summed up
//   write   tables, lengths, pairs and slots; a row finds its free pages by the
//           counts before each span and a vote in the span (a list of them all,
//           made before, was one more barrier: 16.4 us for the last two below)
//
// The steps are dependent and small: a table of 64 sequences of 4096 tokens is
// 64 KB, so what they cost is the barriers between them.  Small batches are one
// CTA's, with the scratch in its shared memory; above that it is one cooperative
// launch of a CTA per SM.
#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kFree = 0x7F7F7F7F;
constexpr int kHeld = -1;
constexpr int kPinned = -2;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kCtaThreads = 512;   // of the one CTA of small batches
constexpr int kGridThreads = 256;  // of a CTA per SM
constexpr int kMaxWarps = 16;
constexpr int kMaxSpans = 2048;  // of blocks, a warp's each
constexpr int kColumns = 512;    // of a row that a warp takes at a time

__device__ __forceinline__ int warps_per_cta() { return (int)blockDim.x >> 5; }

// Scratch that other CTAs write (or, of one CTA, shared memory): never from L1.
__device__ __forceinline__ int ld_scratch(const int32_t* p) { return *reinterpret_cast<const volatile int32_t*>(p); }

// A new row.  One without a sequence has parent kNone and nothing else, but for
// the error code of a refused one (as a negative growth).
constexpr int kNone = -2;
struct Row {
  int parent, len, grow;
  int tail;  // page it goes on inside, or -1
};

__device__ __forceinline__ int pages_of(const ForkParams& p, int tokens) {  // tokens below 2^31 - 32
  return (tokens + p.block_size - 1) >> p.block_shift;
}
__device__ __forceinline__ int have_of(const ForkParams& p, const Row& w) { return pages_of(p, w.len); }
__device__ __forceinline__ int want_of(const ForkParams& p, const Row& w) { return pages_of(p, w.len + max(w.grow, 0)); }

__device__ __forceinline__ Row load_row(const ForkParams& p, int i) {
  Row w{kNone, 0, 0, -1};
  const int parent = __ldcg(p.parents + i);
  if (parent < -1) return w;
  const int grow = p.grow ? __ldcg(p.grow + i) : p.max_grow;
  if (parent >= p.num_old || grow < 0 || grow > p.max_grow) {
    w.grow = -PA_DEVERR_FORK;
    return w;
  }
  const int len = parent < 0 ? 0 : __ldcg(p.lens + parent);
  if (len < 0 || len > p.maxblk * p.block_size || ((int64_t)len + grow) > (int64_t)p.maxblk_out * p.block_size) {
    w.grow = -PA_DEVERR_CONTEXT_LEN;
    return w;
  }
  w.parent = parent;
  w.len = len;
  w.grow = grow;
  if (parent >= 0 && grow > 0 && (len & (p.block_size - 1))) {
    const int b = __ldcg(p.tables + (size_t)parent * p.maxblk + (len >> p.block_shift));
    if (b >= 0 && b < p.num_blocks) w.tail = b;
  }
  return w;
}

// Every step asks for new rows, and to find out what one is takes three loads,
// one behind the other: a CTA does that once, for as many as it has room for.
constexpr int kHeldRows = 1024;
__device__ void hold_rows(const ForkParams& p, Row* held) {
  for (int i = threadIdx.x; i < min(p.num_new, kHeldRows); i += (int)blockDim.x) held[i] = load_row(p, i);
  __syncthreads();
}
__device__ __forceinline__ Row row_of(const ForkParams& p, const Row* held, int i) {
  return i < kHeldRows ? held[i] : load_row(p, i);
}

// Does row i, which goes on inside page w.tail, need a copy of it?
__device__ __forceinline__ bool needs_copy(const ForkParams& p, const Row& w, int i) {
  return w.tail >= 0 && (ld_scratch(p.state + w.tail) != i || (p.pinned && __ldg(p.pinned + w.tail)));
}

// after step_count
__device__ __forceinline__ bool is_free(const ForkParams& p, int b) { return ld_scratch(p.state + b) == kFree; }

__device__ void step_clear(const ForkParams& p, int rank, int ranks) {
  for (int b = rank * (int)blockDim.x + threadIdx.x; b < p.num_blocks; b += ranks * (int)blockDim.x) p.state[b] = kFree;
}

// Every item looks at all parents, so its cost grows with old rows times new ones:
// nothing up to a few hundred rows (512 rows of 256 blocks 14.9 us in all), most of
// the call from a few thousand on.  Measured on GB300, as many new rows as old: 1024
// of 256 blocks 23 us, 2048 of 128 50, 4096 of 64 143, 8192 of 64 447, 16384 of 64
// 1.7 ms, 65535 of 16 24 ms.  Past kHeldRows a parent's row is loaded anew, too.
__device__ void step_mark(const ForkParams& p, const Row* held, int rank, int ranks) {
  const int lane = threadIdx.x & 31;
  const int chunks = (p.maxblk + kColumns - 1) / kColumns;
  const int64_t items = (int64_t)p.num_old * chunks;
  for (int64_t it = (int64_t)rank * warps_per_cta() + (threadIdx.x >> 5); it < items;
       it += (int64_t)ranks * warps_per_cta()) {
    const int old = (int)(it / chunks), c0 = (int)(it - (int64_t)old * chunks) * kColumns;
    // the new rows that go on from this one: any at all, any that leaves its tail as it is
    bool some = false, rests = false;
    int have = 0;
    for (int i = lane; i < p.num_new; i += 32) {
      if ((i < kHeldRows ? held[i].parent : __ldcg(p.parents + i)) != old) continue;
      const Row w = row_of(p, held, i);
      if (w.parent < 0) continue;
      some = true;
      have = have_of(p, w);
      if (w.tail >= 0) {
        if (c0 == 0) atomicMin(p.state + w.tail, i);
      } else {
        rests = true;
      }
    }
    if (!__any_sync(kAll, some)) continue;
    rests = __any_sync(kAll, rests);
    have = __reduce_max_sync(kAll, have);
    const int end = min(have - (rests ? 0 : 1), c0 + kColumns);
    const int32_t* row = p.tables + (size_t)old * p.maxblk;
    bool bad = false;
    for (int j = c0 + lane; j < end; j += 8 * 32) {
      int b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = j + 32 * k < end ? __ldcg(row + j + 32 * k) : -1;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (j + 32 * k >= end) continue;
        if (b[k] >= 0 && b[k] < p.num_blocks) p.state[b[k]] = kHeld;
        else bad = true;
      }
    }
    if (bad) record_error(p.err, PA_DEVERR_BLOCK_ID);
  }
}

// Warp w of all takes blocks [w * span, (w + 1) * span).
__device__ __forceinline__ int span_of(const ForkParams& p, int ranks) {
  const int warps = ranks * warps_per_cta();
  return ((p.num_blocks + warps - 1) / warps + 31) & ~31;
}

__device__ void step_count(const ForkParams& p, int rank, int ranks) {
  const int warp = rank * warps_per_cta() + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int span = span_of(p, ranks);
  const int64_t b0 = (int64_t)warp * span;
  const int b1 = (int)min((int64_t)p.num_blocks, b0 + span);
  int n = 0;
#pragma unroll 4
  for (int64_t b = b0 + lane; b < b1; b += 32) {
    const bool pinned = p.pinned && __ldg(p.pinned + b), free = ld_scratch(p.state + b) == kFree;
    if (free && pinned) p.state[b] = kPinned;
    n += free && !pinned;
  }
  n = __reduce_add_sync(kAll, n);
  if (lane == 0) p.warp_free[warp] = n;
}

// One CTA: how many free pages the rows before each row need, and all of them.  A
// warp's rows together may need more than 32 bits hold: past kMany, more than a
// pool has blocks (2^29), their sum stays there, and the batch is refused.
constexpr int kMany = (1 << 30) - 1;
__device__ void step_rows(const ForkParams& p, const Row* held) {
  __shared__ int sums[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t before = 0;
  for (int base = 0; base < p.num_new; base += (int)blockDim.x) {
    const int i = base + threadIdx.x;
    int need = 0;
    if (i < p.num_new) {
      const Row w = row_of(p, held, i);
      if (w.grow < 0) record_error(p.err, -w.grow);
      need = want_of(p, w) - have_of(p, w) + needs_copy(p, w, i);
    }
    int x = need;  // inclusive in the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, x, o);
      if (lane >= o) x = min(x + y, kMany);
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t at = before + x - need;
    for (int w = 0; w < warps_per_cta(); ++w) {
      if (w < warp) at += sums[w];
      before += sums[w];
    }
    // more pages than there are blocks cannot be had: any such offset will do
    if (i < p.num_new) p.row_start[i] = (int)min(at, (int64_t)INT32_MAX);
    __syncthreads();
  }
  if (threadIdx.x == 0) *p.needed = (int)min(before, (int64_t)INT32_MAX);
}

// Free pages before each warp's span (before[warps]: of all), worked out by every
// CTA for itself.
__device__ void sum_up(const ForkParams& p, int rank, int ranks, int* before) {
  __shared__ int sums[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = ranks * warps_per_cta(), per = (warps + (int)blockDim.x - 1) / (int)blockDim.x;
  const int w0 = min((int)threadIdx.x * per, warps), w1 = min(w0 + per, warps);
  int n = 0;
  for (int w = w0; w < w1; ++w) {
    const int f = ld_scratch(p.warp_free + w);
    before[w] = f;
    n += f;
  }
  int x = n;  // inclusive in the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int at = x - n, total = 0;
  for (int w = 0; w < warps_per_cta(); ++w) {
    if (w < warp) at += sums[w];
    total += sums[w];
  }
  for (int w = w0; w < w1; ++w) {
    const int f = before[w];
    before[w] = at;
    at += f;
  }
  if (threadIdx.x == 0) before[warps] = total;
  __syncthreads();
}

// The warp writes free pages k, k + 1, ... to dst[0 .. n), the first of them to
// `near` too: there are that many.
constexpr int kNear = 32;
__device__ void put_free(const ForkParams& p, int ranks, const int* before, int k, int n, int32_t* dst, int* near) {
  const int lane = threadIdx.x & 31, span = span_of(p, ranks);
  const int warps = ranks * warps_per_cta();
  int lo = 0, hi = warps;  // before[lo] <= k < before[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (before[mid] <= k) lo = mid;
    else hi = mid;
  }
  for (int done = 0; done < n && lo < warps; ++lo) {
    int at = before[lo];
    if (before[lo + 1] == at) continue;
    const int64_t b0 = (int64_t)lo * span;
    const int b1 = (int)min((int64_t)p.num_blocks, b0 + span);
    for (int64_t b = b0; b < b1 && done < n; b += 32) {
      const bool f = b + lane < b1 && is_free(p, (int)b + lane);
      const unsigned v = __ballot_sync(kAll, f);
      const int j = at + __popc(v & ((1u << lane) - 1u)) - k;
      if (f && j >= 0 && j < n) {
        dst[j] = (int)b + lane;
        if (j < kNear) near[j] = (int)b + lane;
      }
      at += __popc(v);
      done = at - k;
    }
  }
}

__device__ void step_write(const ForkParams& p, const Row* held, int rank, int ranks) {
  __shared__ int before[kMaxSpans + 1], nears[kMaxWarps][kNear];
  int* near = nears[threadIdx.x >> 5];
  sum_up(p, rank, ranks, before);
  const int lane = threadIdx.x & 31;
  const int chunks = (p.maxblk_out + kColumns - 1) / kColumns;
  const int64_t items = (int64_t)p.num_new * chunks;
  const int total = before[ranks * warps_per_cta()], needed = ld_scratch(p.needed);
  const bool refused = needed > total;
  if (rank == 0 && threadIdx.x == 0) {
    if (refused) record_error(p.err, PA_DEVERR_NO_BLOCKS);
    *p.num_free = refused ? total : total - needed;
  }
  for (int64_t it = (int64_t)rank * warps_per_cta() + (threadIdx.x >> 5); it < items;
       it += (int64_t)ranks * warps_per_cta()) {
    const int i = (int)(it / chunks), c0 = (int)(it - (int64_t)i * chunks) * kColumns;
    const int end = min(p.maxblk_out, c0 + kColumns);
    int32_t* dst = p.tables_out + (size_t)i * p.maxblk_out;
    const Row w = refused ? Row{kNone, 0, 0, -1} : row_of(p, held, i);
    const int want = want_of(p, w), grow = max(w.grow, 0);
    const bool copy = needs_copy(p, w, i);
    const int shared = have_of(p, w) - copy;  // the parent's blocks, and fresh ones from here on
    const int f0 = max(c0, shared), f1 = min(end, want);
    const int32_t* src = p.tables + (size_t)max(w.parent, 0) * p.maxblk;
    int b[8];
    auto load = [&](int j) {
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = j + 32 * k < min(end, shared) ? __ldcg(src + j + 32 * k) : -1;
    };
    auto store = [&](int j) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = j + 32 * k;
        if (c < end && (c < shared || c >= want)) dst[c] = b[k];
      }
    };
    load(c0 + lane);  // on their way while free pages are looked for
    if (f0 < f1) put_free(p, ranks, before, ld_scratch(p.row_start + i) + f0 - shared, f1 - f0, dst + f0, near);
    store(c0 + lane);
    for (int j = c0 + lane + 8 * 32; j < end; j += 8 * 32) {
      load(j);
      store(j);
    }
    __syncwarp();
    auto page = [&](int c) {  // of a new token's column, as it has just been written
      return c < shared ? w.tail : c - f0 < kNear ? near[c - f0] : ld_scratch(dst + c);
    };
    if (lane == 0) {
      if (c0 == 0) p.lens_out[i] = w.len + grow;
      if (copy ? shared >= c0 && shared < end : c0 == 0) {
        p.pairs[2 * i] = copy ? w.tail : -1;
        p.pairs[2 * i + 1] = copy ? page(shared) : -1;
      }
    }
    // slots of the new tokens in these columns; those of no token with the first
    int32_t* slots = p.slots + (size_t)i * p.max_grow;
    const int64_t bs = p.block_size;
    const int t0 = (int)min((int64_t)grow, max(c0 * bs - w.len, (int64_t)0));
    const int t1 = (int)min((int64_t)grow, max(end * bs - w.len, (int64_t)0));
    for (int t = t0 + lane; t < t1; t += 32) {
      const int pos = w.len + t, b = page(pos >> p.block_shift);
      slots[t] = b >= 0 && b < p.num_blocks ? b * p.block_size + (pos & (p.block_size - 1)) : -1;
    }
    if (c0 == 0)
      for (int t = grow + lane; t < p.max_grow; t += 32) slots[t] = -1;
    __syncwarp();  // near is another row's next
  }
}

// The steps, `sync` a barrier of all ranks' threads that makes their writes seen.
template <typename Sync>
__device__ __forceinline__ void fork_steps(const ForkParams& p, int rank, int ranks, Sync sync) {
  __shared__ Row held[kHeldRows];
  step_clear(p, rank, ranks);
  hold_rows(p, held);
  sync();
  step_mark(p, held, rank, ranks);
  sync();
  if (rank == ranks - 1) step_rows(p, held);
  step_count(p, rank, ranks);
  sync();
  step_write(p, held, rank, ranks);
}

// One CTA, its scratch in shared memory: a step is a barrier, not a trip to L2.
__global__ void __launch_bounds__(kCtaThreads) fork_cta_kernel(const ForkParams p0) {
  extern __shared__ __align__(16) int32_t scratch[];
  griddep_wait();  // and no early start of the next kernel, which may read the tables before it waits
  ForkParams p = p0;
  p.state = scratch;
  p.row_start = p.state + p.num_blocks;
  p.warp_free = p.row_start + p.num_new;
  p.needed = p.warp_free + kMaxWarps;
  fork_steps(p, 0, 1, [] { __syncthreads(); });
}

__global__ void __launch_bounds__(kGridThreads) fork_grid_kernel(const ForkParams p) {
  fork_steps(p, blockIdx.x, gridDim.x, [] { cooperative_groups::this_grid().sync(); });
}

// ----------------------------------------------------------------------------
// copy_pages: blockIdx.z the cache, y strides over pairs, x over a block's 16-byte
// vectors.  All layers' copies of a step are one launch.  Measured on GB300: 512
// pairs, about half of them copies, of 32 KB in four caches 7.0 us (L2 and HBM, 63
// MB read and written); 16 pairs 1.7.
// ----------------------------------------------------------------------------
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ CopyPagesParams p) {
  constexpr int U = 4;  // vectors in flight per thread
  griddep_wait();
  griddep_launch_dependents();
  uint4* cache = static_cast<uint4*>(p.caches[blockIdx.z]);
  for (int pi = blockIdx.y; pi < p.num_pairs; pi += gridDim.y) {
    const int src = __ldg(p.pairs + 2 * pi), dst = __ldg(p.pairs + 2 * pi + 1);
    if (src < 0) continue;  // no copy
    if (src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) record_error(p.err, PA_DEVERR_BLOCK_ID);
      continue;
    }
    const uint4* s = cache + (int64_t)src * p.block_vecs;
    uint4* d = cache + (int64_t)dst * p.block_vecs;
    for (int64_t i0 = (int64_t)blockIdx.x * blockDim.x * U + threadIdx.x; i0 < p.block_vecs;
         i0 += (int64_t)gridDim.x * blockDim.x * U) {
      uint4 a[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * (int)blockDim.x < p.block_vecs) a[u] = s[i0 + u * (int)blockDim.x];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + u * (int)blockDim.x < p.block_vecs) d[i0 + u * (int)blockDim.x] = a[u];
    }
  }
}

constexpr int kCtaBlocks = 16384;
int cta_scratch(int num_blocks, int num_new) { return (num_blocks + num_new + kMaxWarps + 1) * 4; }

int fork_ranks() {
  const int sms = num_sms(), most = kMaxSpans / (kGridThreads / 32);
  return sms > most ? most : sms > 0 ? sms : 1;
}

}  // namespace

// state, row_start, warp_free, needed
ForkWorkspace fork_workspace_layout(int num_new, int num_blocks) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  ForkWorkspace w{};
  w.state = 0;
  w.row_start = al((size_t)num_blocks * 4);
  w.warp_free = w.row_start + al((size_t)num_new * 4);
  w.needed = w.warp_free + al((size_t)fork_ranks() * (kGridThreads / 32) * 4);
  w.bytes = w.needed + 256;
  return w;
}

cudaError_t launch_fork_blocks(const ForkParams& p, cudaStream_t stream) {
  // Entries that the steps go over, up to which one CTA is the faster: it needs no
  // barrier of the whole grid, about two microseconds each.  Measured on GB300 with
  // the list (us, one CTA and a CTA per SM): 16 rows of <= 95 blocks 5.7 and 12; 512
  // of <= 256 70 and 15.8; 64 of <= 8190 (more blocks than it has room for) 16.1.
  // Without it 6.4, 14.9 and 14.5 by the form that is taken.
  constexpr int64_t kCtaWork = 48 << 10;
  const int64_t work = (int64_t)p.num_old * p.maxblk + (int64_t)p.num_new * p.maxblk_out + p.num_blocks;
  if (p.num_blocks <= kCtaBlocks && p.num_new <= kHeldRows && work <= kCtaWork) {
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && !attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(fork_cta_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 cta_scratch(kCtaBlocks, kHeldRows));
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
    return launch_pdl(fork_cta_kernel, dim3(1), dim3(kCtaThreads), cta_scratch(p.num_blocks, p.num_new), stream, p);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(fork_ranks());
  cfg.blockDim = dim3(kGridThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fork_grid_kernel, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_copy_pages(const CopyPagesParams& p, cudaStream_t stream) {
  int64_t bx = (p.block_vecs + 1023) / 1024;
  if (bx > 8) bx = 8;
  const int by = p.num_pairs < 65535 ? p.num_pairs : 65535;
  return launch_pdl(copy_pages_kernel, dim3((unsigned)bx, by, p.num_caches), dim3(256), 0, stream, p);
}

}  // namespace pa
