// Norm, rotation and cache write of new tokens in one pass, for sm_103a.
//
// Per head row x of D elements: x <- x * rsqrt(mean(x^2) + eps) * w (optional),
// then the first rot_dim elements are rotated pair by pair, (a, b) ->
// (a c - b s, b c + a s), with c, s read from a table at the token's position
// (of up to three axes); queries go to q_out, keys and values to their cache
// slots.  Everything between the one load and the one store is fp32.
//
// Bound by HBM: 2 bytes read and 2 written per element; what it takes to get
// there is bytes in flight and few instructions per element.
//  * A warp's work item is up to 2 KB of one token's query, key or value heads
//    (8 heads of 128): one bulk copy (cp.async.bulk) into the warp's own ring
//    in shared memory, kRopeStages of them, so loads in flight cost no registers
//    and no address arithmetic.  Warps share nothing and never meet.
//  * D/8 threads hold a head row, and each thread four whole pairs of it
//    (elements 4s.. and rot_dim/2 + 4s..; eight neighbours if interleaved), so
//    a rotation needs no other thread and the norm's sum is the only shuffle.
//    The thread keeps its four cosines and sines for the item's heads.
//  * The chain slot/position -> table row runs ahead of the items: positions
//    two items, cosines one.
// Measured on GB300, bf16, norms, 8192 tokens of 32/8 heads of 128 (205 MB): 35.3
// us, 0.86 of the copy rate.  2 KB items, 2 stages, 4 CTAs of 8 warps an SM; when
// that took 36.1: 3 stages 39.7, 4 with 3 CTAs 38.1, 1 KB items 52, 4 KB 38 to 46.
// The same from registers, a CTA per token: 50.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRopeStages = 2;
constexpr int kItemBytes = 2048;
constexpr int kRopeMaxWarps = 8;  // of a CTA
constexpr unsigned kAll = 0xffffffffu;

// A token's place: its slot and its positions on the axes.
struct Place {
  int slot, pos[3];
};

// PARTIAL: rot_dim < D.  Elements behind it are passed on, not turned by nothing (0
// times an infinite neighbour is NaN).  The case of the figures above takes 37.0 us
// with that choice, so the whole rotation goes without.
template <int D, typename T, bool INTER, bool PARTIAL>
__global__ void __launch_bounds__(32 * kRopeMaxWarps, 4) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPH = D / 8;                       // threads per head row
  constexpr int GROUPS = 32 / LPH;                 // head rows side by side
  constexpr int HEADS = kItemBytes / (2 * D);      // heads of an item
  constexpr int RPT = HEADS / GROUPS;              // rows of a thread
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nwarps = blockDim.x >> 5;
  uint8_t* ring = smem + warp * kRopeStages * kItemBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + nwarps * kRopeStages * kItemBytes) + warp * kRopeStages;
  if (lane == 0) {
    for (int s = 0; s < kRopeStages; ++s) mbar_init(smem_u32(&bars[s]), 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int sub = lane % LPH, group = lane / LPH;
  const int half = p.rot_dim / 2;
  const bool rotated = !PARTIAL || sub < p.rot_dim / 8;
  // this thread's two runs of four elements; behind rot_dim, eight neighbours
  const int lo = INTER || !rotated ? 8 * sub : 4 * sub;
  const int hi = INTER || !rotated ? 8 * sub + 4 : half + 4 * sub;
  // blocks of a token: queries, keys, values
  const int qb = (p.q_heads + HEADS - 1) / HEADS, kb = (p.kv_heads + HEADS - 1) / HEADS;
  const int bpt = qb + 2 * kb;
  // items of this warp: gw, gw + W, ... of num_tokens * bpt, as (token, block)
  const int W = gridDim.x * nwarps, gw = blockIdx.x * nwarps + warp;
  const int dt = W / bpt, db = W % bpt;
  auto advance = [&](int& t, int& b) {
    t += dt;
    b += db;
    if (b >= bpt) {
      b -= bpt;
      ++t;
    }
  };

  // the whole kernel after the one before it: its inputs may come from there,
  // and q_out may still be read there.  No early launch of the next kernel,
  // which may read q_out in its set-up.
  griddep_wait();

  // heads [h0, h0 + n) of block b's kind
  auto heads_of = [&](int b, int& h0) {
    const int all = b < qb ? p.q_heads : p.kv_heads;
    h0 = (b < qb ? b : b < qb + kb ? b - qb : b - qb - kb) * HEADS;
    return min(HEADS, all - h0);
  };
  auto issue = [&](int t, int b, int s) {
    int h0;
    const int n = heads_of(b, h0);
    const T* src = reinterpret_cast<const T*>(b < qb ? p.q : b < qb + kb ? p.k : p.v) +
                   (b < qb ? p.q_stride : b < qb + kb ? p.k_stride : p.v_stride) * (int64_t)t + (int64_t)h0 * D;
    fence_proxy_async_smem();  // this warp's reads of the stage before the copy's writes
    __syncwarp();
    if (lane == 0) {
      mbar_arrive_expect_tx(smem_u32(&bars[s]), n * D * 2);
      bulk_load(smem_u32(ring + s * kItemBytes), src, n * D * 2, smem_u32(&bars[s]));
    }
  };
  auto place_of = [&](int t) {
    Place w;
    w.slot = __ldg(p.slots + t);
#pragma unroll
    for (int a = 0; a < 3; ++a) w.pos[a] = a < p.num_axes ? __ldg(p.positions + (size_t)a * p.num_tokens + t) : 0;
    return w;
  };
  auto outside = [&](const Place& w) {
    bool bad = false;
#pragma unroll
    for (int a = 0; a < 3; ++a) bad |= w.pos[a] < 0 || w.pos[a] >= p.max_position;
    return bad;
  };
  // this thread's four cosines and sines at a place inside the table
  auto turn = [&](const Place& w, bool want, float4& c, float4& s) {
    c = make_float4(1.f, 1.f, 1.f, 1.f);
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!rotated || !want) return;
    const int j = 4 * sub;  // its pairs
    auto axis = [&](int jj) { return jj < p.sec_end[0] ? w.pos[0] : jj < p.sec_end[1] ? w.pos[1] : w.pos[2]; };
    if ((j >= p.sec_end[0] || j + 3 < p.sec_end[0]) && (j >= p.sec_end[1] || j + 3 < p.sec_end[1])) {
      const float* row = p.cos_sin + (size_t)axis(j) * p.rot_dim + j;  // all four turn by one axis
      c = __ldg(reinterpret_cast<const float4*>(row));
      s = __ldg(reinterpret_cast<const float4*>(row + half));
    } else {
      auto at = [&](int i) { return p.cos_sin + (size_t)axis(j + i) * p.rot_dim + j + i; };
      c = make_float4(__ldg(at(0)), __ldg(at(1)), __ldg(at(2)), __ldg(at(3)));
      s = make_float4(__ldg(at(0) + half), __ldg(at(1) + half), __ldg(at(2) + half), __ldg(at(3) + half));
    }
  };

  int t = gw / bpt, b = gw % bpt;  // the item at hand
  int ti = t, bi = b;              // the next to load
  for (int s = 0; s < kRopeStages; ++s) {
    if (ti < p.num_tokens) issue(ti, bi, s);
    advance(ti, bi);
  }
  int t1 = t, b1 = b;  // the item after this one
  advance(t1, b1);
  Place w{}, w1{};
  if (t < p.num_tokens) w = place_of(t);
  if (t1 < p.num_tokens) w1 = place_of(t1);
  float4 c4, s4;
  turn(w, t < p.num_tokens && b < qb + kb && !outside(w), c4, s4);

  for (int k = 0; t < p.num_tokens; ++k) {
    int t2 = t1, b2 = b1;
    advance(t2, b2);
    Place w2{};
    if (t2 < p.num_tokens) w2 = place_of(t2);
    float4 c4n, s4n;
    turn(w1, t1 < p.num_tokens && b1 < qb + kb && !outside(w1), c4n, s4n);

    const int s = k % kRopeStages;
    if (!mbar_wait(smem_u32(&bars[s]), (k / kRopeStages) & 1)) {
      if (lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
      // copies in flight land before exit (bounded)
      for (int j = k + 1; j < k + kRopeStages && t1 < p.num_tokens; ++j, advance(t1, b1))
        mbar_wait(smem_u32(&bars[j % kRopeStages]), (j / kRopeStages) & 1);
      return;
    }
    const bool skip = outside(w);
    if (b == 0 && lane == 0) {
      if (skip && w.slot >= 0) record_error(p.err, PA_DEVERR_POSITION);
      if (!skip && w.slot >= p.num_slots) record_error(p.err, PA_DEVERR_SLOT);
    }
    const bool is_q = b < qb, is_v = b >= qb + kb;
    if (!skip && (is_q || (w.slot >= 0 && w.slot < p.num_slots))) {
      int h0;
      const int n = heads_of(b, h0);
      const uint8_t* from = ring + s * kItemBytes;
      T* dst = is_q ? reinterpret_cast<T*>(p.q_out) + ((size_t)t * p.q_heads + h0) * D
                    : reinterpret_cast<T*>(is_v ? p.v_cache : p.k_cache) + ((size_t)w.slot * p.kv_heads + h0) * D;
      if (is_v) {
        for (int i = lane; i < n * (D / 8); i += 32)
          reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(from)[i];
      } else {
        const T* wt = reinterpret_cast<const T*>(is_q ? p.q_weight : p.k_weight);
        uint2 wx = make_uint2(0u, 0u), wy = wx;
        if (wt) {
          wx = __ldg(reinterpret_cast<const uint2*>(wt + lo));
          wy = __ldg(reinterpret_cast<const uint2*>(wt + hi));
        }
        // pair i of two packed runs: (a[i], b[i])
        auto pairs = [](const uint2& x, const uint2& y, float (&a)[4], float (&bb)[4]) {
          if constexpr (INTER) {
            a[0] = Elem<T>::lo(x.x), bb[0] = Elem<T>::hi(x.x), a[1] = Elem<T>::lo(x.y), bb[1] = Elem<T>::hi(x.y);
            a[2] = Elem<T>::lo(y.x), bb[2] = Elem<T>::hi(y.x), a[3] = Elem<T>::lo(y.y), bb[3] = Elem<T>::hi(y.y);
          } else {
            a[0] = Elem<T>::lo(x.x), a[1] = Elem<T>::hi(x.x), a[2] = Elem<T>::lo(x.y), a[3] = Elem<T>::hi(x.y);
            bb[0] = Elem<T>::lo(y.x), bb[1] = Elem<T>::hi(y.x), bb[2] = Elem<T>::lo(y.y), bb[3] = Elem<T>::hi(y.y);
          }
        };
        float wa[4], wb[4];
        pairs(wx, wy, wa, wb);
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int u = 0; u < RPT; ++u) {
          const int row = u * GROUPS + group;  // rows behind n hold an earlier item: not stored
          const T* src = reinterpret_cast<const T*>(from) + row * D;
          const uint2 x = *reinterpret_cast<const uint2*>(src + lo), y = *reinterpret_cast<const uint2*>(src + hi);
          float a[4], bb[4];
          pairs(x, y, a, bb);
          if (wt) {  // warp-uniform
            float sx = 0.f, sy = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) ffma2(sx, sy, a[i], bb[i], a[i], bb[i], sx, sy);
            float sum = sx + sy;
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
            const float f = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] *= f * wa[i];
              bb[i] *= f * wb[i];
            }
          }
          float za[4], zb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            za[i] = rotated ? a[i] * c[i] - bb[i] * sn[i] : a[i];
            zb[i] = rotated ? bb[i] * c[i] + a[i] * sn[i] : bb[i];
          }
          if (row < n) {
            T* to = dst + row * D;
            if constexpr (INTER) {
              *reinterpret_cast<uint2*>(to + lo) = make_uint2(Elem<T>::pack(za[0], zb[0]), Elem<T>::pack(za[1], zb[1]));
              *reinterpret_cast<uint2*>(to + hi) = make_uint2(Elem<T>::pack(za[2], zb[2]), Elem<T>::pack(za[3], zb[3]));
            } else {
              *reinterpret_cast<uint2*>(to + lo) = make_uint2(Elem<T>::pack(za[0], za[1]), Elem<T>::pack(za[2], za[3]));
              *reinterpret_cast<uint2*>(to + hi) = make_uint2(Elem<T>::pack(zb[0], zb[1]), Elem<T>::pack(zb[2], zb[3]));
            }
          }
        }
      }
    }
    if (ti < p.num_tokens) issue(ti, bi, s);
    advance(ti, bi);
    t = t1, b = b1, w = w1, c4 = c4n, s4 = s4n;
    t1 = t2, b1 = b2, w1 = w2;
  }
}

template <int D, typename T, bool INTER, bool PARTIAL>
cudaError_t launch_rot(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int HEADS = kItemBytes / (2 * D);
  auto kern = norm_rope_kernel<D, T, INTER, PARTIAL>;
  auto bytes = [](int warps) { return warps * kRopeStages * (kItemBytes + 8); };
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kRopeMaxWarps));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t bpt = (p.q_heads + HEADS - 1) / HEADS + 2 * ((p.kv_heads + HEADS - 1) / HEADS);
  const int64_t items = p.num_tokens * bpt, sms = num_sms() > 0 ? num_sms() : 1;
  // few items: two warps a CTA, so that they spread over the SMs; many: 32
  // warps an SM (128 KB of rings) that walk the items
  const int warps = items <= 2 * kRopeMaxWarps * sms ? 2 : kRopeMaxWarps;
  const int64_t want = (items + warps - 1) / warps, cap = 4 * sms;
  const unsigned grid = (unsigned)(warps == 2 || want < cap ? want : cap);
  return launch_pdl(kern, dim3(grid), dim3(32 * warps), bytes(warps), stream, p);
}

template <int D, typename T, bool INTER>
cudaError_t launch_t(const NormRopeParams& p, cudaStream_t stream) {
  return p.rot_dim < D ? launch_rot<D, T, INTER, true>(p, stream) : launch_rot<D, T, INTER, false>(p, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const bool b = dt == PA_BF16, i = p.interleaved != 0;
  if (head_dim == 128)
    return b ? (i ? launch_t<128, __nv_bfloat16, true>(p, stream) : launch_t<128, __nv_bfloat16, false>(p, stream))
             : (i ? launch_t<128, __half, true>(p, stream) : launch_t<128, __half, false>(p, stream));
  if (head_dim == 64)
    return b ? (i ? launch_t<64, __nv_bfloat16, true>(p, stream) : launch_t<64, __nv_bfloat16, false>(p, stream))
             : (i ? launch_t<64, __half, true>(p, stream) : launch_t<64, __half, false>(p, stream));
  return cudaErrorInvalidValue;
}

}  // namespace pa
