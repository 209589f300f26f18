// Attention of a tree of drafted tokens over the paged cache, for sm_103a
// (pa_verify_tree): the warp-MMA kernel, and the log-sum-exp merge of the
// partitions.
//
// A CTA owns 64 rows (query, head of the group) of one (request, KV head,
// partition of the context) and walks its keys in tiles of 64: one producer
// warp gathers K and V from the blocks by TMA into a ring, four consumer warps
// of 16 rows each compute S = Q K^T and O += P V with mma.m16n8k16 (fp32) and
// an online softmax.  Only tiles that reach the drafted tokens are masked, by
// one 64-bit word per row.  A request of one partition is written to out; the
// partitions of a longer one leave unnormalised partials (o, m in log2 units,
// l) that the merge combines.
#include <float.h>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "tree.cuh"

namespace pa {

namespace {

constexpr int kTreeConsumers = 4;
constexpr int kTreeStages = 3;
constexpr int kTreeKeys = 64;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ uint8_t* align1024_tree(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

template <int D, int BSUB>
struct TreeSmem {
  using Tile = KvTile<D, BSUB, kTreeKeys>;
  static constexpr int STAGE_BYTES = 2 * Tile::BYTES;
  static constexpr int FULL_OFF = kTreeStages * STAGE_BYTES;
  static constexpr int EMPTY_OFF = FULL_OFF + kTreeStages * 8;
  static constexpr int ZERO_OFF = EMPTY_OFF + kTreeStages * 8;  // consumers' "V rows cleaned" barrier
  static constexpr int BAD_OFF = ZERO_OFF + 8;                  // drafted nodes with non-finite V (2 words)
  static constexpr int BYTES = BAD_OFF + 8 + 1024;
};

template <int D, int BSUB, typename T>
__global__ void __launch_bounds__((kTreeConsumers + 1) * 32)
    tree_mma_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const TreeParams p) {
  using L = TreeSmem<D, BSUB>;
  using Tile = typename L::Tile;
  constexpr int CW = kTreeConsumers, STAGES = kTreeStages;
  constexpr int KSTEPS = D / 16;
  constexpr int DT8 = D / 8;
  constexpr int ROWS = CW * 16;
  constexpr int LOADS = Tile::NH * 2;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024_tree(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::FULL_OFF);
  uint64_t* empty = reinterpret_cast<uint64_t*>(smem + L::EMPTY_OFF);
  uint64_t* zbar = reinterpret_cast<uint64_t*>(smem + L::ZERO_OFF);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::BAD_OFF);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  const int row_tiles = (p.max_q_len * G + ROWS - 1) / ROWS;
  const int r = blockIdx.y;
  const int row0 = (blockIdx.x % row_tiles) * ROWS;
  const int hc = blockIdx.x / row_tiles;
  const int h = hc % p.kv_heads, c = hc / p.kv_heads;

  TreeReq rq;
  const int code = tree_request(p, r, rq);
  const int rows = rq.n * G;
  const int k0 = c * p.split_tokens;
  if (code || row0 >= rows || k0 >= rq.ctx) {
    griddep_wait();
    if (code && blockIdx.x == 0 && threadIdx.x == 0) record_error(p.err, code);
    return;
  }
  const int kend = min(rq.ctx, k0 + p.split_tokens);
  const int ntiles = (kend - k0 + kTreeKeys - 1) / kTreeKeys;
  const bool direct = rq.ctx <= p.split_tokens;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), CW);
    }
    mbar_init(smem_u32(zbar), CW);
    bad[0] = bad[1] = 0;
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  __syncthreads();
  griddep_launch_dependents();

  if (warp == CW) {
    // ------------------------------------------------------------ producer
    const int32_t* trow = p.tables + (size_t)r * p.maxblk;
    const uint64_t pol = policy_evict_last();  // re-read by the other row tiles
    griddep_wait();
    bool failed = false;
    int j = 0;
    for (; j < ntiles; ++j) {
      const int s = j % STAGES;
      if (j >= STAGES && !mbar_wait(smem_u32(&empty[s]), ((j / STAGES) - 1) & 1)) {
        failed = true;
        break;
      }
      const int ts = k0 + j * kTreeKeys;
      const int nvalid = min(kTreeKeys, kend - ts);
      const int nsub = (nvalid + BSUB - 1) / BSUB;
      const uint32_t bar = smem_u32(&full[s]);
      const uint32_t kdst = smem_u32(smem + s * L::STAGE_BYTES);
      if (lane == 0) mbar_arrive_expect_tx(bar, nsub * LOADS * Tile::BOX_BYTES);
      __syncwarp();
      for (int i = lane; i < nsub * LOADS; i += 32) {
        const int sub = i / LOADS, rem = i % LOADS;
        const int isv = rem / Tile::NH, hf = rem % Tile::NH;
        const int tok = ts + sub * BSUB;
        int b = __ldg(trow + tok / p.block_size);
        if (b < 0 || b >= p.num_blocks) {
          record_error(p.err, PA_DEVERR_BLOCK_ID);
          b = p.num_blocks;  // rows past the tensor map: TMA zero-fills
        }
        tma_load_4d_hint(kdst + isv * Tile::BYTES + Tile::box(hf, sub), isv ? &vmap : &kmap, bar, 0, hf, h,
                         b * p.block_size + tok % p.block_size, pol);
      }
    }
    if (failed && lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
    for (int t = j - STAGES < 0 ? 0 : j - STAGES; t < j; ++t)  // loads in flight land before exit (bounded)
      mbar_wait(smem_u32(&full[t % STAGES]), (t / STAGES) & 1);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int ra = row0 + warp * 16 + (lane >> 2);
  const int rb = ra + 8;
  const int qia = ra / G, qib = rb / G;
  const uint64_t all_nodes = rq.n >= 64 ? ~0ull : (1ull << rq.n) - 1;
  const uint64_t maska = ra < rows ? __ldg(p.mask + rq.qs + qia) & all_nodes : 0;
  const uint64_t maskb = rb < rows ? __ldg(p.mask + rq.qs + qib) & all_nodes : 0;

  // Q A-fragments: rows ra/rb, d = 16ks + 2(lane%4) (+8)
  uint32_t qa[KSTEPS][4];
  {
    const T* q = reinterpret_cast<const T*>(p.q);
    const T* qra = q + ((size_t)(rq.qs + qia) * p.q_heads + h * G + ra % G) * D;
    const T* qrb = q + ((size_t)(rq.qs + qib) * p.q_heads + h * G + rb % G) * D;
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks) {
      const int d = ks * 16 + 2 * (lane & 3);
      qa[ks][0] = ra < rows ? __ldg(reinterpret_cast<const uint32_t*>(qra + d)) : 0u;
      qa[ks][1] = rb < rows ? __ldg(reinterpret_cast<const uint32_t*>(qrb + d)) : 0u;
      qa[ks][2] = ra < rows ? __ldg(reinterpret_cast<const uint32_t*>(qra + d + 8)) : 0u;
      qa[ks][3] = rb < rows ? __ldg(reinterpret_cast<const uint32_t*>(qrb + d + 8)) : 0u;
    }
  }

  griddep_wait();
  float acc[DT8][4];
#pragma unroll
  for (int i = 0; i < DT8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
  const float sl2 = p.scale_log2;
  const int mi = lane >> 3, rr = lane & 7;
  int cleaned = 0;  // tiles whose V rows were cleaned (phase of zbar)

  for (int j = 0; j < ntiles; ++j) {
    const int s = j % STAGES;
    if (!mbar_wait(smem_u32(&full[s]), (j / STAGES) & 1)) {
      if (lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
      return;
    }
    const int ts = k0 + j * kTreeKeys;
    const int nvalid = min(kTreeKeys, kend - ts);
    uint8_t* kt = smem + s * L::STAGE_BYTES;
    uint8_t* vt = kt + Tile::BYTES;
    const int first = max(0, rq.hist - ts);  // first drafted row of the tile
    if (nvalid < kTreeKeys || first < kTreeKeys) {
      // V rows past the keys become zero (p = 0 must not meet stale NaN);
      // drafted rows lose their non-finite elements.  The consumers take a
      // share each and meet on zbar.
      const int f0 = min(first, nvalid);
      const int nv = (kTreeKeys - f0) * Tile::NH * 8;
      for (int i = warp * 32 + lane; i < nv; i += CW * 32) {
        const int row = f0 + i / (Tile::NH * 8);
        const int rem = i % (Tile::NH * 8);
        uint4* at = reinterpret_cast<uint4*>(vt + Tile::line(rem >> 3, row) + ((rem & 7) << 4));
        if (row >= nvalid) {
          *at = make_uint4(0, 0, 0, 0);
        } else {
          uint4 v = *at;
          if (scrub8<T>(v)) {
            *at = v;
            const int node = ts + row - rq.hist;
            atomicOr(&bad[node >> 5], 1u << (node & 31));
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(zbar));
      if (!mbar_wait(smem_u32(zbar), cleaned & 1)) {
        if (lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
        return;
      }
      ++cleaned;
    }
    const uint32_t kts = smem_u32(kt), vts = smem_u32(vt);

    // S = Q K^T over 64 keys: 8 n-tiles of 8 keys
    float sc[8][4];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
    for (int nt = 0; nt < 8; nt += 2) {
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        uint32_t b[4];
        ldmatrix_x4(b, kts + Tile::offset(8 * (nt + (mi >> 1)) + rr, 2 * ks + (mi & 1)));
        mma_16816<T>(sc[nt], qa[ks], b[0], b[1]);
        mma_16816<T>(sc[nt + 1], qa[ks], b[2], b[3]);
      }
    }

    // mask + online softmax (rows ra: elements 0,1; rb: elements 2,3)
    const bool masked = first < kTreeKeys || nvalid < kTreeKeys;
    float mxa = -INFINITY, mxb = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[nt][e] *= sl2;
        sc[nt][2 + e] *= sl2;
        if (masked) {
          const int t = ts + nt * 8 + 2 * (lane & 3) + e;
          const int node = t - rq.hist;
          const bool in = t < kend;
          sc[nt][e] = in && (node < 0 || ((maska >> node) & 1)) ? sc[nt][e] : -INFINITY;
          sc[nt][2 + e] = in && (node < 0 || ((maskb >> node) & 1)) ? sc[nt][2 + e] : -INFINITY;
        }
        mxa = fmaxf(mxa, sc[nt][e]);
        mxb = fmaxf(mxb, sc[nt][2 + e]);
      }
    }
    mxa = fmaxf(mxa, __shfl_xor_sync(kAll, mxa, 1));
    mxa = fmaxf(mxa, __shfl_xor_sync(kAll, mxa, 2));
    mxb = fmaxf(mxb, __shfl_xor_sync(kAll, mxb, 1));
    mxb = fmaxf(mxb, __shfl_xor_sync(kAll, mxb, 2));
    const float mna = fmaxf(ma, mxa), mnb = fmaxf(mb, mxb);
    const float ua = mna == -INFINITY ? 0.f : mna;  // nothing seen so far: every p is 0
    const float ub = mnb == -INFINITY ? 0.f : mnb;
    const float ala = exp2f(ma - ua), alb = exp2f(mb - ub);
    ma = mna;
    mb = mnb;
    // P is rounded to the input type for the P.V MMA (both operands of an MMA
    // have one type); the denominators sum the same rounded values, so each
    // output row is an exact convex combination of V rows
    float suma = 0.f, sumb = 0.f;
    uint32_t pka[8], pkb[8];
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
      pka[nt] = Elem<T>::pack(exp2f(sc[nt][0] - ua), exp2f(sc[nt][1] - ua));
      pkb[nt] = Elem<T>::pack(exp2f(sc[nt][2] - ub), exp2f(sc[nt][3] - ub));
      suma += Elem<T>::sum2(pka[nt]);
      sumb += Elem<T>::sum2(pkb[nt]);
    }
    la = la * ala + suma;
    lb = lb * alb + sumb;
#pragma unroll
    for (int i = 0; i < DT8; ++i) {
      acc[i][0] *= ala;
      acc[i][1] *= ala;
      acc[i][2] *= alb;
      acc[i][3] *= alb;
    }

    // O += P V: 4 k-steps of 16 keys; P from the S accumulators in registers
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const uint32_t pa[4] = {pka[2 * kk], pkb[2 * kk], pka[2 * kk + 1], pkb[2 * kk + 1]};
#pragma unroll
      for (int nd = 0; nd < DT8; nd += 2) {
        uint32_t b[4];
        ldmatrix_x4_trans(b, vts + Tile::offset(16 * kk + rr + 8 * (mi & 1), nd + (mi >> 1)));
        mma_16816<T>(acc[nd], pa, b[0], b[1]);
        mma_16816<T>(acc[nd + 1], pa, b[2], b[3]);
      }
    }
    if (masked) fence_proxy_async_smem();  // cleaned rows were written here; TMA may refill them
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
  }

  la += __shfl_xor_sync(kAll, la, 1);
  la += __shfl_xor_sync(kAll, la, 2);
  lb += __shfl_xor_sync(kAll, lb, 1);
  lb += __shfl_xor_sync(kAll, lb, 2);
  const uint64_t noted = cleaned ? (uint64_t)bad[0] | ((uint64_t)bad[1] << 32) : 0;
  const uint64_t fixa = maska & noted, fixb = maskb & noted;
  if (fixa | fixb) {
#pragma unroll
    for (int i = 0; i < DT8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int d = i * 8 + 2 * (lane & 3) + e;
        acc[i][e] += tree_restore<T>(p, r, h, D, rq.hist, fixa, d);
        acc[i][2 + e] += tree_restore<T>(p, r, h, D, rq.hist, fixb, d);
      }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = x ? rb : ra;
    if (row >= rows) continue;
    const float l = x ? lb : la, m = x ? mb : ma;
    const size_t orow = (size_t)(rq.qs + (x ? qib : qia)) * p.q_heads + h * G + row % G;
    if (direct) {
      const float inv = tree_inverse(l);
      T* o = reinterpret_cast<T*>(p.out) + orow * D + 2 * (lane & 3);
#pragma unroll
      for (int i = 0; i < DT8; ++i)
        *reinterpret_cast<uint32_t*>(o + i * 8) = Elem<T>::pack(acc[i][2 * x] * inv, acc[i][2 * x + 1] * inv);
    } else {
      const size_t pr = orow * p.max_splits + c;
      float* o = p.part_o + pr * D + 2 * (lane & 3);
#pragma unroll
      for (int i = 0; i < DT8; ++i)
        *reinterpret_cast<float2*>(o + i * 8) = make_float2(acc[i][2 * x], acc[i][2 * x + 1]);
      if ((lane & 3) == 0) {
        p.part_m[pr] = m;
        p.part_l[pr] = l;
      }
    }
  }
}

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
  const int nsplit = (rq.ctx + p.split_tokens - 1) / p.split_tokens;
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
    const float w = pm[c] == -INFINITY ? 0.f : exp2f(pm[c] - M);
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

template <int D, int BSUB, typename T>
cudaError_t launch_mma_t(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, cudaStream_t stream) {
  using L = TreeSmem<D, BSUB>;
  auto kern = tree_mma_kernel<D, BSUB, T>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t row_tiles = ((int64_t)p.max_q_len * p.group + kTreeConsumers * 16 - 1) / (kTreeConsumers * 16);
  const int64_t gx = row_tiles * p.kv_heads * p.max_splits;
  if (gx > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(kern, dim3((unsigned)gx, p.num_reqs), dim3((kTreeConsumers + 1) * 32), L::BYTES, stream, kmap,
                    vmap, p);
}

template <int D, typename T>
cudaError_t launch_tree_dt(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int bsub,
                           cudaStream_t stream) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (bsub) {
    case 4: e = launch_mma_t<D, 4, T>(kmap, vmap, p, stream); break;
    default: {
      const pa_dtype dt = std::is_same<T, __half>::value ? PA_FP16 : PA_BF16;
      e = p.max_q_len * p.group <= 128 ? launch_tree_tile(kmap, vmap, p, D, bsub, dt, stream)
                                       : launch_tree_pair(kmap, vmap, p, D, bsub, dt, stream);
    }
  }
  if (e != cudaSuccess || p.max_splits == 1) return e;
  const unsigned gx = (unsigned)(((int64_t)p.max_q_len * p.q_heads + 7) / 8);
  return launch_pdl(tree_merge_kernel<D, T>, dim3(gx, p.num_reqs), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_verify_tree(const CUtensorMap& kmap, const CUtensorMap& vmap, const TreeParams& p, int head_dim,
                               int bsub, pa_dtype dt, cudaStream_t stream) {
  if (head_dim == 128)
    return dt == PA_BF16 ? launch_tree_dt<128, __nv_bfloat16>(kmap, vmap, p, bsub, stream)
                         : launch_tree_dt<128, __half>(kmap, vmap, p, bsub, stream);
  if (head_dim == 64)
    return dt == PA_BF16 ? launch_tree_dt<64, __nv_bfloat16>(kmap, vmap, p, bsub, stream)
                         : launch_tree_dt<64, __half>(kmap, vmap, p, bsub, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
