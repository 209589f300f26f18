// Attention of a tree of drafted tokens over the paged cache, for sm_103a
// (pa_verify_tree): the choice of the kernel, and the log-sum-exp merge of the
// partitions.
//
// The attention itself is the tcgen05 kernels' TREE form.  Up to 128 rows per
// (request, KV head) take attn_tile.cu's (128-key tiles; one Q tile), more
// attn_tc.cu's (two Q tiles of 128 rows share every 64-key K/V tile).  Measured
// on GB300, 64 requests of 509..4079 tokens, 32/8 heads: 20..32 nodes 125 us on
// the first; 26..60 nodes 147 us on the second; before the requests ran in
// order of length 132 and 162 us, and the latter 215 us as two row tiles of
// the first (K and V once more through L2).  Before them a warp-MMA kernel took 347
// and 509 us.
#include <float.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "tree.cuh"

namespace pa {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// One warp per row of a request of several partitions: M = max_c m_c,
// out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c, partitions in order.
// blockIdx.y: request; 8 rows per CTA.
template <int D, typename T>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeParams p) {
  constexpr int V = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  TreeReq rq;
  if (tree_request(p, r, rq)) return;
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rq.n * p.q_heads || rq.ctx <= p.split_tokens) return;
  const int nsplit = partitions_of(rq.ctx, p.split_tokens);
  const size_t orow = (size_t)rq.qs * p.q_heads + row;
  const float* pm = p.part_m + orow * p.max_splits;
  const float* pl = p.part_l + orow * p.max_splits;
  const float* po = p.part_o + orow * p.max_splits * D + lane * V;
  float M = -INFINITY;
  for (int c = lane; c < nsplit; c += 32) M = fmaxf(M, pm[c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  float a[V], den = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = 0.f;
#pragma unroll 4
  for (int c = 0; c < nsplit; ++c) {
    // no smaller than the smallest normal number where the row sees a key: a value
    // that is not finite decides the row however little it weighs
    const float w = pm[c] == -INFINITY ? 0.f : fmaxf(exp2f(pm[c] - M), FLT_MIN);
    den += w * pl[c];
    const float* x = po + (size_t)c * D;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(x + i);
      if (w != 0.f) {  // a partition that the row sees nothing of holds no numbers
        a[i] += w * v.x;
        a[i + 1] += w * v.y;
      }
    }
  }
  const float inv = tree_inverse(den);
  T* o = reinterpret_cast<T*>(p.out) + orow * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(o + i) = Elem<T>::pack(a[i] * inv, a[i + 1] * inv);
}

template <int D, typename T>
cudaError_t launch_tree_dt(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int bsub, pa_dtype dt,
                           cudaStream_t stream) {
  const cudaError_t e = p.max_q_len * p.group <= 128 ? launch_tree_tile(kmap, vmap, p, D, bsub, dt, stream)
                                                     : launch_tree_pair(kmap, vmap, p, D, bsub, dt, stream);
  if (e != cudaSuccess || p.max_splits == 1) return e;
  const unsigned gx = (unsigned)(((int64_t)p.max_q_len * p.q_heads + 7) / 8);
  return launch_pdl(tree_merge_kernel<D, T>, dim3(gx, p.num_reqs), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_verify_tree(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int head_dim,
                               int bsub, pa_dtype dt, cudaStream_t stream) {
  if (head_dim == 128)
    return dt == PA_BF16 ? launch_tree_dt<128, __nv_bfloat16>(kmap, vmap, p, bsub, dt, stream)
                         : launch_tree_dt<128, __half>(kmap, vmap, p, bsub, dt, stream);
  if (head_dim == 64)
    return dt == PA_BF16 ? launch_tree_dt<64, __nv_bfloat16>(kmap, vmap, p, bsub, dt, stream)
                         : launch_tree_dt<64, __half>(kmap, vmap, p, bsub, dt, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
