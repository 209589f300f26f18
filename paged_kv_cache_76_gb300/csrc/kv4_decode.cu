// Decode attention over a 4-bit paged cache (see kv4.cuh for the page), one
// query per request or a few causal ones, for sm_103a.
//
// A CTA of four warps owns one (request r, KV head h, partition c) unit: warp w
// takes the stages of 32 tokens w, w + 4, ..., every query head of the group on
// one read of K and V; the warps' parts are joined in shared memory and the
// partitions by the log-sum-exp merge.  The codes and the scales of a page are
// contiguous, so each comes by a bulk copy into the warp's own ring.
//
// A cache element is exact in fp16, so the products are fp16 MMAs whatever the
// type of q: a query row is brought to [2^13, 2^14) by a power of two (taken
// back in its softmax scale), where fp16 holds every bf16 or fp16 element that
// is not 2^-27 of the row's largest, and the weights are held up to 2^15, where
// one of 2^-29 of the largest is still a normal number: they are rounded by at
// most 2^-11 of themselves (less than bf16's 2^-9).  The denominator is the fp32
// sum of the unrounded weights.
//
// Per 16 tokens (m16n8k16, S^T = K Q^T and O^T += V^T P^T):
//   K: lane (g, c) = (lane / 4, lane % 4) reads D/4 consecutive elements of
//      tokens pi(g), pi(g) + 8, D/16 A fragments of both; which elements a
//      fragment takes is free as long as Q's B fragments take the same.
//   V: lane (g, c) reads D/8 elements of the four tokens that P's B fragments
//      hold for it.  An A fragment wants two tokens side by side, so the codes
//      of two tokens are interleaved before they are converted (four logical
//      instructions for 16 elements, where 16 fp16 pairs would take 16).
//   pi(i) = i ^ (i/2 & 1) puts neighbouring lanes' rows into different banks.
// Elements cost one conversion and one multiplication a pair (42 pairs per
// clock and SM measured for the two together).
//
// Tokens past the context: their K scores become -inf by selection, and their V
// scales 0 (codes are always finite), so nothing they hold reaches the output.
// A draft's later token that holds NaN must not reach the queries before it:
// the last q_len - 1 tokens' NaN scales are zeroed too and kept as bits, and
// the queries that do see such a token get their NaN at the end.
#include <float.h>

#include <type_traits>

#include "kv4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kStageTokens = 32;
constexpr int kMaxEntries = 1024;  // Block Table entries of a partition
constexpr float kRescale = 8.f;   // a reference is raised when a score passes it by more (log2 units)
constexpr float kShift = 7.f;     // weights are 2^(s - m + kShift) <= 2^15
constexpr unsigned kAll = 0xffffffffu;

template <int D, int NT, int STAGES>
struct Kv4DecodeSmem {
  // of a stage: codes of K, its scales, codes of V, its scales
  static constexpr int CODES = kStageTokens * Kv4Row<D>::CODES;
  static constexpr int SCALES = kStageTokens * Kv4Row<D>::SCALES;
  static constexpr int HALF = CODES + SCALES;
  static constexpr int STAGE = 2 * HALF;
  static constexpr int RING = STAGES * STAGE;  // of a warp; at the end its outputs [NT * 8][ROW]
  static constexpr int ROW = D + 4;            // floats, so that the lanes of a store spread over the banks
  static constexpr int BAR_OFF = kWarps * RING;
  static constexpr int NAN_OFF = BAR_OFF + kWarps * STAGES * 8;
  static constexpr int SUM_OFF = NAN_OFF + D / kKv4Group * 4;  // m, then l: [kWarps][NT * 8]
  static constexpr int TAB_OFF = SUM_OFF + 2 * kWarps * NT * 8 * 4;
  static_assert(NT * 8 * ROW * 4 <= RING, "a warp's outputs take its ring's place");
  static constexpr int bytes(int entries) { return TAB_OFF + entries * 4; }
};

template <int D, int NT, int STAGES, typename T>
__global__ void __launch_bounds__(kWarps * 32) kv4_decode_kernel(const Kv4DecodeParams p) {
  using L = Kv4DecodeSmem<D, NT, STAGES>;
  using R = Kv4Row<D>;
  constexpr int KSTEPS = D / 16;
  constexpr int NW = D / 32;  // words of K codes a lane reads per token; of V codes: D / 64

  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;
  uint8_t* ring = smem + warp * L::RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF) + warp * STAGES;
  uint32_t* nan = reinterpret_cast<uint32_t*>(smem + L::NAN_OFF);
  float* sums = reinterpret_cast<float*>(smem + L::SUM_OFF);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + L::TAB_OFF);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&bars[s]), 1);
    fence_mbar_init();
  }
  if (threadIdx.x < D / kKv4Group) nan[threadIdx.x] = 0;
  griddep_launch_dependents();

  const int r = blockIdx.y;
  const int h = blockIdx.x % p.kv_heads, c = blockIdx.x / p.kv_heads;
  const int col0 = blockIdx.z * NT * 8;
  const int cap = p.maxblk * p.block_size;
  int ctx = __ldg(p.lens + r);
  const bool bad_len = ctx < 0 || ctx > cap;
  ctx = min(max(ctx, 0), cap);
  const int nsplit = (ctx + p.split_tokens - 1) / p.split_tokens;
  const int G = p.group, NC = G * p.q_len, qh0 = h * G;
  if (c >= max(nsplit, 1)) {
    griddep_wait();
    if (bad_len && threadIdx.x == 0) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
    return;
  }
  const int tok0 = c * p.split_tokens, tok1 = min(tok0 + p.split_tokens, ctx);
  const int nstages = (tok1 - tok0 + kStageTokens - 1) / kStageTokens;  // of the CTA: warp w takes w, w + kWarps, ...
  const int mine = nstages > warp ? (nstages - warp + kWarps - 1) / kWarps : 0;
  const int blk0 = tok0 / p.block_size;

  // row of column n in q, out and the partials
  auto row_of = [&](int n) {
    const int qi = n / G;
    return (size_t)(r * p.q_len + qi) * p.q_heads + qh0 + (n - qi * G);
  };

  bool bad_id = false;
  uint32_t qf[NT][KSTEPS][2];
  float sl2[NT][2];  // softmax scale (log2 units) of the lane's two columns of each n-tile
  if (nstages > 0) {
    const int nblk = (tok1 - 1) / p.block_size - blk0 + 1;
    const int32_t* trow = p.tables + (size_t)r * p.maxblk + blk0;
    for (int i = threadIdx.x; i < nblk; i += kWarps * 32) {
      int b = __ldg(trow + i);
      if (b < 0 || b >= p.num_blocks) {
        bad_id = true;
        b = -1;
      }
      tab[i] = b;
    }
    // Q^T as the B operand: lane (g, c) holds column g of each n-tile, elements
    // D/4 c + 4 ks + {0, 1} and {2, 3}
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = col0 + nt * 8 + g;
      const uint2* src = reinterpret_cast<const uint2*>(static_cast<const T*>(p.q) + (n < NC ? row_of(n) : 0) * D + (D / 4) * c4);
      float x[KSTEPS][4];
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        const uint2 w = n < NC ? __ldg(src + ks) : make_uint2(0u, 0u);
        x[ks][0] = Elem<T>::lo(w.x), x[ks][1] = Elem<T>::hi(w.x);
        x[ks][2] = Elem<T>::lo(w.y), x[ks][3] = Elem<T>::hi(w.y);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(x[ks][e]));
      }
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      // 2^e <= top < 2^(e + 1); rows of zeros and of values that are not finite stay as they are
      int e = top > 0.f && top < INFINITY ? ilogbf(top) - 13 : 0;
      e = max(e, -126);
      const float down = ldexpf(1.f, -e);
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        qf[nt][ks][0] = Elem<__half>::pack(x[ks][0] * down, x[ks][1] * down);
        qf[nt][ks][1] = Elem<__half>::pack(x[ks][2] * down, x[ks][3] * down);
      }
      const float back = p.scale_log2 * ldexpf(1.f, e);
      // accumulators hold columns 2c, 2c + 1 of the tile
      sl2[nt][0] = __shfl_sync(kAll, back, 8 * c4);
      sl2[nt][1] = __shfl_sync(kAll, back, 8 * c4 + 4);
    }
  }
  griddep_wait();
  if (bad_len && threadIdx.x == 0) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
  if (bad_id) record_error(p.err, PA_DEVERR_BLOCK_ID);
  T* out = static_cast<T*>(p.out);
  const int ncols = min(NC - col0, NT * 8);  // of this CTA
  if (ctx == 0) {
    for (int i = threadIdx.x; i < ncols * D; i += kWarps * 32) out[row_of(col0 + i / D) * D + i % D] = Elem<T>::from(0.f);
    return;
  }
  __syncthreads();  // the table

  const int bs = p.block_size;
  const int bsh = p.block_shift;
  const int page = bs * R::BYTES;
  const uint64_t pol = policy_evict_first();
  // stage j: tokens [ts, ts + 32); lane 4i + {0, 1, 2, 3} brings page i's codes and scales of K, of V (pages that
  // hold tokens of the partition)
  auto issue = [&](int j) {  // the warp's j-th stage
    const int s = j % STAGES;
    const int ts = tok0 + kStageTokens * (j * kWarps + warp);
    const int npages = (min(kStageTokens, tok1 - ts) + bs - 1) >> bsh;
    const uint32_t bar = smem_u32(&bars[s]);
    const int i = lane >> 2;
    const bool has = i < npages, isv = lane & 2, part = lane & 1;
    const int b = has ? tab[((ts - tok0) >> bsh) + i] : -1;
    const int copies = __popc(__ballot_sync(kAll, b >= 0)) >> 1;  // pages, of K and of V
    fence_proxy_async_smem();  // this stage's earlier reads and writes before the copies
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(bar, copies * page);
    __syncwarp();
    if (has) {
      const int bytes = bs * (part ? R::SCALES : R::CODES);
      uint8_t* dst = ring + s * L::STAGE + (isv ? L::HALF : 0) + (part ? L::CODES : 0) + i * bytes;
      if (b >= 0) {
        const uint8_t* src = static_cast<const uint8_t*>(isv ? p.v_cache : p.k_cache) +
                             ((size_t)b * p.kv_heads + h) * page + (part ? bs * R::CODES : 0);
        bulk_load_hint(smem_u32(dst), src, bytes, bar, pol);
      } else {  // a bad block id: zeros
        for (int k = 0; k < bytes; k += 16) *reinterpret_cast<uint4*>(dst + k) = make_uint4(0, 0, 0, 0);
      }
    }
  };

  float m[NT][2], l[NT][2], acc[NT][KSTEPS][4];
  int lim[NT][2];  // tokens [0, lim) are visible to the lane's columns
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
      const int n = col0 + nt * 8 + 2 * c4 + e;
      lim[nt][e] = min(tok1, ctx - (p.q_len - 1 - (n < NC ? n / G : p.q_len - 1)));
    }
#pragma unroll
    for (int mt = 0; mt < KSTEPS; ++mt) acc[nt][mt][0] = acc[nt][mt][1] = acc[nt][mt][2] = acc[nt][mt][3] = 0.f;
  }
  const int causal0 = ctx - (p.q_len - 1);  // tokens from here on are hidden from some query (q_len 1: from ctx on)

  for (int j = 0; j < min(mine, STAGES); ++j) issue(j);
  const int pg = g ^ ((g >> 1) & 1);        // token row of this lane's K fragments
  const int t01[2] = {2 * c4 ^ (c4 & 1), (2 * c4 + 1) ^ (c4 & 1)};  // pi(2c), pi(2c + 1)

  bool failed = false;
  int j = 0;
  for (; j < mine; ++j) {
    const int s = j % STAGES;
    if (!mbar_wait(smem_u32(&bars[s]), (j / STAGES) & 1)) {
      failed = true;
      break;
    }
    const int ts = tok0 + kStageTokens * (j * kWarps + warp);
    uint8_t* kst = ring + s * L::STAGE;
    uint8_t* vst = kst + L::HALF;
    // where token t of the stage has its codes and scales
    auto code_at = [](int t) { return t * R::CODES; };
    auto scale_at = [](int t) { return L::CODES + t * R::SCALES; };
    __syncwarp();  // zeroed pages
    if (ts + kStageTokens > tok1) {
      const int t = lane;  // a token per lane
      if (ts + t >= tok1) {
#pragma unroll
        for (int i = 0; i < R::SCALES; i += 4) *reinterpret_cast<uint32_t*>(vst + scale_at(t) + i) = 0u;
      }
      __syncwarp();
    }
    if (ts + kStageTokens > causal0 && p.q_len > 1) {
      const int t = lane;
      if (ts + t >= causal0 && ts + t < tok1) {
#pragma unroll
        for (int i = 0; i < R::SCALES; ++i) {
          uint8_t* at = vst + scale_at(t) + i;
          if (*at >= kKv4FirstInf) {
            *at = 0;
            atomicOr(&nan[i], 1u << (ts + t - causal0));
          }
        }
      }
      __syncwarp();
    }

    // 16 tokens from tb on; `all`: every column sees all of them
    auto tile = [&](const int tb, const auto all_t) {
      constexpr bool all = decltype(all_t)::value;
      const int t0 = ts + tb + pg;  // this lane's score rows: tokens t0, t0 + 8
      float sacc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sacc[nt][0] = sacc[nt][1] = sacc[nt][2] = sacc[nt][3] = 0.f;
      {
        uint32_t w[2][NW], sc[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* src = kst + code_at(tb + pg + 8 * e) + c4 * (4 * NW);
          if constexpr (NW == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(src);
            w[e][0] = v.x, w[e][1] = v.y, w[e][2] = v.z, w[e][3] = v.w;
            sc[e] = *reinterpret_cast<const uint16_t*>(kst + scale_at(tb + pg + 8 * e) + 2 * c4);
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            w[e][0] = v.x, w[e][1] = v.y;
            sc[e] = kst[scale_at(tb + pg + 8 * e) + c4];
          }
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) {
          uint32_t x[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            kv4_unpack(w[e][i], x[e]);
            const uint32_t s2 = kv4_scale2(NW == 4 && i >= 2 ? sc[e] >> 8 : sc[e] & 0xFFu);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[e][k] = hmul2_u(x[e][k], s2);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a[4] = {x[0][2 * k], x[1][2 * k], x[0][2 * k + 1], x[1][2 * k + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_16816<__half>(sacc[nt], a, qf[nt][2 * i + k][0], qf[nt][2 * i + k][1]);
          }
        }
      }

      uint32_t pb0[NT], pb1[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float s0 = all || t0 < lim[nt][0] ? sacc[nt][0] * sl2[nt][0] : -INFINITY;
        const float s1 = all || t0 < lim[nt][1] ? sacc[nt][1] * sl2[nt][1] : -INFINITY;
        const float s2 = all || t0 + 8 < lim[nt][0] ? sacc[nt][2] * sl2[nt][0] : -INFINITY;
        const float s3 = all || t0 + 8 < lim[nt][1] ? sacc[nt][3] * sl2[nt][1] : -INFINITY;
        // m is raised to the column's maximum only when a score passes it by
        // more than kRescale, so most tiles need no maximum across lanes: a
        // vote says that no lane has such a score
        const bool up = fmaxf(s0, s2) > m[nt][0] + kRescale || fmaxf(s1, s3) > m[nt][1] + kRescale;
        if (__any_sync(kAll, up)) {
          float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kAll, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kAll, mx1, o));
          }
          const bool up0 = mx0 > m[nt][0] + kRescale, up1 = mx1 > m[nt][1] + kRescale;
          const float al0 = up0 ? ex2_approx(m[nt][0] - mx0) : 1.f;
          const float al1 = up1 ? ex2_approx(m[nt][1] - mx1) : 1.f;
          m[nt][0] = up0 ? mx0 : m[nt][0];
          m[nt][1] = up1 ? mx1 : m[nt][1];
          l[nt][0] *= al0;
          l[nt][1] *= al1;
#pragma unroll
          for (int mt = 0; mt < KSTEPS; ++mt) {
            acc[nt][mt][0] *= al0;
            acc[nt][mt][1] *= al1;
            acc[nt][mt][2] *= al0;
            acc[nt][mt][3] *= al1;
          }
        }
        // a column that has seen no token keeps m = -inf; its exponents then use 0
        const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kShift;
        const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kShift;
        const float p0 = ex2_approx(s0 - b0), p1 = ex2_approx(s1 - b1);
        const float p2 = ex2_approx(s2 - b0), p3 = ex2_approx(s3 - b1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        pb0[nt] = movmatrix_trans(Elem<__half>::pack(p0, p1));
        pb1[nt] = movmatrix_trans(Elem<__half>::pack(p2, p3));
      }

      {
        // V of tokens pi(2c), pi(2c+1) (pair 0) and those + 8 (pair 1), elements D/8 g ..
        uint32_t x[2][D / 16][2];  // [pair][element pair][element of it]: two tokens each
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t a[D / 64], b[D / 64];
          const uint8_t* sa = vst + code_at(tb + t01[0] + 8 * e) + g * (D / 16);
          const uint8_t* sb = vst + code_at(tb + t01[1] + 8 * e) + g * (D / 16);
          if constexpr (D == 128) {
            const uint2 va = *reinterpret_cast<const uint2*>(sa), vb = *reinterpret_cast<const uint2*>(sb);
            a[0] = va.x, a[1] = va.y, b[0] = vb.x, b[1] = vb.y;
          } else {
            a[0] = *reinterpret_cast<const uint32_t*>(sa);
            b[0] = *reinterpret_cast<const uint32_t*>(sb);
          }
          const int grp = D == 128 ? g : g >> 1;
          const uint32_t s2 = kv4_scale_pair(vst[scale_at(tb + t01[0] + 8 * e) + grp], vst[scale_at(tb + t01[1] + 8 * e) + grp]);
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const uint32_t lo = (a[i] & 0x0F0F0F0Fu) | ((b[i] << 4) & 0xF0F0F0F0u);
            const uint32_t hi = ((a[i] >> 4) & 0x0F0F0F0Fu) | (b[i] & 0xF0F0F0F0u);
            uint32_t y[4], z[4];
            kv4_unpack(lo, y);
            kv4_unpack(hi, z);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              x[e][4 * i + k][0] = hmul2_u(y[k], s2);
              x[e][4 * i + k][1] = hmul2_u(z[k], s2);
            }
          }
        }
#pragma unroll
        for (int mt = 0; mt < KSTEPS; ++mt) {
          const uint32_t a[4] = {x[0][mt][0], x[0][mt][1], x[1][mt][0], x[1][mt][1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816<__half>(acc[nt][mt], a, pb0[nt], pb1[nt]);
        }
      }
    };
    if (ts + kStageTokens <= min(tok1, causal0)) {
#pragma unroll
      for (int q = 0; q < kStageTokens / 16; ++q) tile(16 * q, std::true_type{});
    } else {
      const int tiles = (min(kStageTokens, tok1 - ts) + 15) >> 4;
#pragma unroll 1
      for (int q = 0; q < tiles; ++q) tile(16 * q, std::false_type{});
    }
    __syncwarp();
    if (j + STAGES < mine) issue(j + STAGES);
  }

  if (failed) {
    if (lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
    for (int k = j + 1; k < mine && k < j + STAGES; ++k)  // copies in flight land before the warp goes on
      mbar_wait(smem_u32(&bars[k % STAGES]), (k / STAGES) & 1);
  }

  // the warps' parts of each column: brought to the largest reference, added up in order
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[nt][e];
      x += __shfl_xor_sync(kAll, x, 4);
      x += __shfl_xor_sync(kAll, x, 8);
      x += __shfl_xor_sync(kAll, x, 16);
      if (g == 0) {
        const int n = nt * 8 + 2 * c4 + e;
        sums[warp * NT * 8 + n] = m[nt][e];
        sums[(kWarps + warp) * NT * 8 + n] = x;
      }
    }
  float* po = reinterpret_cast<float*>(ring);  // every copy into the ring has landed and been read
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      // the lane's D/8 elements of column n: D/8 g + 2 mt + {0, 1}
      float4* dst = reinterpret_cast<float4*>(po + (nt * 8 + 2 * c4 + e) * L::ROW + (D / 8) * g);
#pragma unroll
      for (int i = 0; i < KSTEPS / 2; ++i)
        dst[i] = make_float4(acc[nt][2 * i][e], acc[nt][2 * i][2 + e], acc[nt][2 * i + 1][e], acc[nt][2 * i + 1][2 + e]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < ncols * (D / 4); i += kWarps * 32) {
    const int n = i / (D / 4), d = 4 * (i % (D / 4));
    float f[kWarps], M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, f[w] = sums[w * NT * 8 + n]);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    const float ref = M == -INFINITY ? 0.f : M;  // no finite score: sums are zero or not numbers
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = ex2_approx(f[w] - ref);
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * L::RING) + n * L::ROW + d);
      o.x += a * x.x, o.y += a * x.y, o.z += a * x.z, o.w += a * x.w;
      sum += a * sums[(kWarps + w) * NT * 8 + n];
    }
    // a token behind causal0 that is not a number, for the columns that see it
    const int nsee = min(max(min(tok1, ctx - (p.q_len - 1 - (col0 + n) / G)) - causal0, 0), 31);
    if (nan[d / kKv4Group] & ((1u << nsee) - 1u)) o = make_float4(NAN, NAN, NAN, NAN);
    const size_t row = row_of(col0 + n);
    if (nsplit == 1) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a NaN sum stays one
      *reinterpret_cast<uint2*>(out + row * D + d) =
          make_uint2(Elem<T>::pack(o.x * inv, o.y * inv), Elem<T>::pack(o.z * inv, o.w * inv));
    } else {
      *reinterpret_cast<float4*>(p.part_o + (row * p.max_splits + c) * D + d) = o;
      if (d == 0) {
        p.part_m[row * p.max_splits + c] = M;
        p.part_l[row * p.max_splits + c] = sum;
      }
    }
  }
}

template <int D, int NT, typename T>
cudaError_t launch_t(const Kv4DecodeParams& p, cudaStream_t stream) {
  constexpr int STAGES = 3;
  using L = Kv4DecodeSmem<D, NT, STAGES>;
  auto kern = kv4_decode_kernel<D, NT, STAGES, T>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(kMaxEntries));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const dim3 grid((unsigned)(p.max_splits * p.kv_heads), p.num_seqs, (p.group * p.q_len + NT * 8 - 1) / (NT * 8));
  return launch_pdl(kern, grid, dim3(kWarps * 32), L::bytes(p.tab_entries), stream, p);
}

template <int D, typename T>
cudaError_t launch_nt(const Kv4DecodeParams& p, cudaStream_t stream) {
  return p.group * p.q_len <= 8 ? launch_t<D, 1, T>(p, stream) : launch_t<D, 2, T>(p, stream);
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  if (head_dim == 128)
    return dt == PA_BF16 ? launch_nt<128, __nv_bfloat16>(p, stream) : launch_nt<128, __half>(p, stream);
  return dt == PA_BF16 ? launch_nt<64, __nv_bfloat16>(p, stream) : launch_nt<64, __half>(p, stream);
}

}  // namespace pa
