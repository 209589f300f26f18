// What the two attention kernels of pa_verify_tree share: the geometry of a
// work unit, and the care that a drafted node's values reach only the rows
// that see the node.
#pragma once

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

// A request's part of the batch.  Row i*G + g is query i (node i), head g of
// the group; keys [0, hist) are seen by every row, key hist + j by the rows
// whose mask has bit j.
struct TreeReq {
  int qs, n, ctx, hist;
};

// The fields that the tcgen05 kernels read as they do a prefill's.
inline PrefillParams tree_prefill_params(const TreeParams& tp) {
  PrefillParams p{};
  p.q = tp.q;
  p.q_start = tp.q_start;
  p.lens = tp.lens;
  p.tables = tp.tables;
  p.out = tp.out;
  p.err = tp.err;
  p.maxblk = tp.maxblk;
  p.num_reqs = tp.num_reqs;
  p.total_q = tp.total_q;
  p.max_q_len = tp.max_q_len;
  p.q_heads = tp.q_heads;
  p.kv_heads = tp.kv_heads;
  p.group = tp.group;
  p.num_blocks = tp.num_blocks;
  p.block_size = tp.block_size;
  p.scale_log2 = tp.scale_log2;
  return p;
}

// The request from immutable inputs; 0, or the error code of a request that is
// skipped.
__device__ __forceinline__ int tree_request(const TreeParams& p, int r, TreeReq& q) {
  q.qs = __ldg(p.q_start + r);
  const int qe = __ldg(p.q_start + r + 1);
  q.n = qe - q.qs;
  q.ctx = __ldg(p.lens + r);
  q.hist = q.ctx - q.n;
  if (q.qs < 0 || qe < q.qs || qe > p.total_q || q.n > p.max_q_len || q.hist < 0) return PA_DEVERR_QUERY_RANGE;
  if (q.ctx > p.maxblk * p.block_size) return PA_DEVERR_CONTEXT_LEN;
  return 0;
}

// Where units outnumber the SMs (one CTA each), the last ones decide when the
// kernel ends, so the requests run longest first: the request of index r in
// that order, ties by number, among the kTreeWindow requests around it.  Every
// thread of the CTA calls it; scratch: kTreeWindow + 1 words of shared memory.
// Measured on GB300, 64 requests of 509..4079 tokens, 8 KV heads, as numbered
// and in this order: 26..60 nodes 161 and 143 us; 20..32 nodes 132 and 127 us;
// 8 nodes 112 and 113 us (the order takes a CTA about a microsecond: a load,
// two barriers, the comparisons).
constexpr int kTreeWindow = 128;
__device__ __forceinline__ int tree_longest_first(const TreeParams& p, int r, int* scratch) {
  const int w0 = r / kTreeWindow * kTreeWindow, n = min(kTreeWindow, p.num_reqs - w0), t = threadIdx.x;
  int len = 0;
  if (t < n) scratch[t] = len = __ldg(p.lens + w0 + t);
  __syncthreads();
  if (t < n) {
    int before = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) before += scratch[i] > len || (scratch[i] == len && i < t);
    if (before == r - w0) scratch[kTreeWindow] = w0 + t;
  }
  __syncthreads();
  return scratch[kTreeWindow];
}

// Blocks of 4 tokens: a TMA box of 4 rows is half of the 8-row atom that the
// 128-byte swizzle repeats in.  The pattern follows the shared-memory address,
// so a box at an odd multiple of 512 bytes lands as the atom's upper half, and
// the tile is laid out as from boxes of 16 rows.  A lane takes a block: its id,
// loaded a tile ahead, then a box per 64 elements of head_dim.  Measured on
// GB300, 64 requests of 509..4079 tokens, 26..60 nodes: 220 us, bound by the
// boxes (blocks of 16: 146); 16-byte asynchronous copies by the same warps 257.
__device__ __forceinline__ int quad_ids(const int32_t* trow, int ts, int nvalid) {
  const int lane = threadIdx.x & 31;
  return 4 * lane < nvalid ? __ldg(trow + ts / 4 + lane) : 0;
}

template <typename Tile, int ROWS>
__device__ __forceinline__ void quad_tile(const TreeParams& p, const CUtensorMap* map, int id, int h, int nvalid,
                                          uint32_t dst, uint32_t bar, uint64_t pol) {
  static_assert(ROWS <= 128, "a block per lane");
  const int lane = threadIdx.x & 31, nsub = (min(nvalid, ROWS) + 3) / 4;
  if (lane == 0) mbar_arrive_expect_tx(bar, nsub * Tile::NH * 512);
  __syncwarp();
  if (lane < nsub) {
    if (id < 0 || id >= p.num_blocks) {
      record_error(p.err, PA_DEVERR_BLOCK_ID);
      id = p.num_blocks;  // rows past the tensor map: TMA zero-fills
    }
#pragma unroll
    for (int hf = 0; hf < Tile::NH; ++hf)
      tma_load_4d_hint(dst + Tile::line(hf, 4 * lane), map, bar, 0, hf, h, id * 4, pol);
  }
}

// Which of the 64 keys from `rel` past the draft's start on (before it:
// negative) a row with this mask sees.
__device__ __forceinline__ uint64_t tree_window(uint64_t mask, int rel) {
  if (rel <= -64) return ~0ull;
  if (rel < 0) return (mask << -rel) | ((1ull << -rel) - 1);
  return rel < 64 ? mask >> rel : 0ull;
}

// 1 / l; a row that sees nothing (l = 0) is zero, a NaN among its scores stays one.
__device__ __forceinline__ float tree_inverse(float l) { return l > 0.f ? 1.f / l : l == 0.f ? 0.f : l; }

// P.V multiplies a masked node's V by exactly zero, which is NaN where V holds
// an infinity or a NaN (a padding node's stale slot).  So the non-finite
// elements of drafted V rows are replaced by zero in shared memory, the row's
// bit is noted, and a row that does see such a node adds the elements back at
// the end (tree_restore): they decide the result there whatever their weight.
// Returns true if v held a non-finite element.
template <typename T> __device__ __forceinline__ bool scrub8(uint4& v) {
  constexpr uint32_t E = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
  uint32_t* u = reinterpret_cast<uint32_t*>(&v);
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool lo = (u[i] & E) == E, hi = ((u[i] >> 16) & E) == E;
    if (lo) u[i] &= 0xFFFF0000u;
    if (hi) u[i] &= 0x0000FFFFu;
    any |= lo || hi;
  }
  return any;
}

// What the noted nodes `bits` (non-finite V, seen by the row) add to element d
// of the row: the sum of their non-finite elements, else 0.
template <typename T>
__device__ __forceinline__ float tree_restore(const TreeParams& p, int r, int h, int head_dim, int hist, uint64_t bits,
                                              int d) {
  float add = 0.f;
  while (bits) {
    const int j = __ffsll((long long)bits) - 1;
    bits &= bits - 1;
    const int t = hist + j;
    const int b = __ldg(p.tables + (size_t)r * p.maxblk + t / p.block_size);
    if (b < 0 || b >= p.num_blocks) continue;
    const T x = reinterpret_cast<const T*>(
        p.v_cache)[(((size_t)b * p.block_size + t % p.block_size) * p.kv_heads + h) * head_dim + d];
    const float f = static_cast<float>(x);
    if (!isfinite(f)) add += f;
  }
  return add;
}

}  // namespace pa
