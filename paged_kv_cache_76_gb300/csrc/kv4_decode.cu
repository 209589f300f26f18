// Decode attention over a 4-bit paged cache (see kv4.cuh for the page), one
// query per request or a few causal ones, for sm_103a.
//
// A CTA of four warps owns one (request r, KV head h, partition c) unit: warp w
// takes the tiles of 16 tokens w, w + 4, ..., every query head of the group on
// one read of K and V; the warps' parts are joined in shared memory and the
// partitions by the log-sum-exp merge, or, where all CTAs run at the same time
// and a list has 16 partitions at most, in a cluster: each CTA writes its parts to
// the ones that join them, all at once, and one barrier later every CTA has a
// share of the list's outputs to write.  No partials, no second kernel (1 request
// of 2048 tokens, 32/8 heads, in 16 partitions 5.0 -> 4.5 us, 16 in four 14 -> 11;
// 4 of <= 1501, 28/4 heads 5.3 -> 5.0, and a call from Python 8..10 -> 6.5).  Past
// that the CTAs of a cluster wait for one another in places that others could
// have (64 requests below 41 -> 46).
//
// At 4.5 bits an element the instructions that turn a tile into MMA operands
// take about as long as its bytes, so the kernel is built for few of them.  The
// tensor and 16-bit floating-point pipe is the one that counts: an MMA holds it
// for 8 cycles of a quarter SM, a conversion of a pair for 1.5, a multiplication
// for 1, so a tile costs 105 cycles of an SM if nothing waits, and its bytes 98.
// Measured on GB300, in us: 64 requests of 509..4079 tokens, 32/8 heads (floor
// 25), and 8 of 32768..131009, 64/8 heads (floor 116):
//   a warp per unit, bulk copies of pages into its ring      52   197
//   codes and scales copied apart, two tiles unrolled        48   178
//   a CTA's four warps share a unit                          51   179
//   16-byte asynchronous copies, block size a constant       46   162
//   shared memory at constant offsets, copies before q       41   144
// What was tried and left: loads straight into registers, a tile ahead (47 and
// 184: too few bytes under way; with a prefetch to L2 six tiles ahead 50 and
// 171); the batch's tiles shared out evenly over as many CTAs as run at a time
// (50 and 154: CTAs that hold ends of two lists take their latencies twice, and
// the merge has more to find out); five CTAs an SM at 96 registers (56 and 161);
// rings of 3 or 6 tiles (no difference); first partitions of all requests first
// (41 and 152); of 16 columns, Q's fragments in shared memory, which leaves four
// CTAs an SM instead of three (4 queries for each of the 64: 66 us either way).
// Over its active cycles an SM issues in 43 to 77 % of them at 64 requests: the last
// of its partitions run with few beside them.  A copy of a page by the bulk engine is issued lane by lane, 15
// instructions each, which is why 16-byte copies win: 334 instructions a tile
// against 378.
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
//   K: lane (g, c) = (lane / 4, lane % 4) holds D/4 consecutive elements of
//      tokens pi(g) and pi(g) + 8, D/16 A fragments of both; which elements a
//      fragment takes is free as long as Q's B fragments take the same.
//   V: lane (g, c) holds D/8 elements of the four tokens that P's B fragments
//      hold for it, pi(2c) = c, pi(2c + 1) = c + 4 and those + 8 (so that a
//      load's lanes have rows of either parity).  An A fragment wants two tokens
//      side by side, so the codes of two tokens are interleaved before they are
//      converted (four logical instructions for 16 elements, where 16 fp16 pairs
//      would take 16).
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
constexpr int kMaxCluster = kKv4Cluster;  // partitions that join their parts in one another's shared memory
constexpr int kTile = 16;
constexpr int kDepth = 4;  // tiles of a warp's ring
constexpr int kMaxEntries = 1024;  // Block Table entries of a partition
constexpr float kRescale = 8.f;    // a reference is raised when a score passes it by more (log2 units)
constexpr float kShift = 7.f;      // weights are 2^(s - m + kShift) <= 2^15
constexpr unsigned kAll = 0xffffffffu;

template <int D, int NT>
struct Kv4DecodeSmem {
  static constexpr int TILE = 2 * kTile * Kv4Row<D>::BYTES;  // K, then V
  static constexpr int RING = kDepth * TILE;                 // of a warp; at the end its outputs
  static constexpr int ROW = D + 4;  // floats of a column's outputs, so that the lanes of a store spread over the banks
  static constexpr int WARP = RING > NT * 8 * ROW * 4 ? RING : NT * 8 * ROW * 4;
  static constexpr int SUM_OFF = kWarps * WARP;             // m, then l: [kWarps][NT * 8]
  static constexpr int NAN_OFF = SUM_OFF + 2 * kWarps * NT * 8 * 4;
  static constexpr int BAD_OFF = NAN_OFF + D / kKv4Group * 4;  // bits: bad block ids of the table
  // from each partition of a cluster: m, then l, of every column; the outputs that this CTA joins
  static constexpr int PART_SUM_OFF = BAD_OFF + (kMaxEntries + 32) / 8;
  static constexpr int PART_OFF = (PART_SUM_OFF + 2 * kMaxCluster * NT * 8 * 4 + 15) & ~15;
  static constexpr int PART = (NT * 8 * D / 4 + kMaxCluster) * 16;
  // then the Block Table; a call without clusters has it in the parts' place
  static constexpr int bytes(int entries, bool cluster) {
    return (cluster ? PART_OFF + PART : PART_SUM_OFF) + entries * 4;
  }
};

// Shared memory at an address and a constant, after the wait that orders them
// (volatile: they stay behind it).
__device__ __forceinline__ uint4 lds4(uint32_t at, int off) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at + off));
  return v;
}
__device__ __forceinline__ uint2 lds2(uint32_t at, int off) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at + off));
  return v;
}
__device__ __forceinline__ uint32_t lds1(uint32_t at, int off) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + off));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t at, int off) {
  uint32_t v;
  asm volatile("{\n .reg .u16 t;\n ld.shared.u16 t, [%1];\n cvt.u32.u16 %0, t;\n}" : "=r"(v) : "r"(at + off));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t at, int off) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at + off));
  return v;
}
// The low four bits of every byte of a, the high four of b (one instruction;
// written as & and | it became two).
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(r) : "r"(0x0F0F0F0Fu), "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void cp_async16_at(uint32_t dst, int off, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + off), "l"(src) : "memory");
}

// JOIN: the partitions of a list are a cluster
template <int D, int NT, int BS, bool JOIN>
__global__ void __launch_bounds__(kWarps * 32, D == 128 && NT == 2 ? 3 : 4) kv4_decode_kernel(const Kv4DecodeParams p) {
  using L = Kv4DecodeSmem<D, NT>;
  using R = Kv4Row<D>;
  constexpr int KSTEPS = D / 16;
  constexpr int NW = D / 32;  // words of K codes a lane has per token; of V codes: D / 64
  constexpr int PAGE = BS * R::BYTES;

  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c4 = lane & 3;
  float* sums = reinterpret_cast<float*>(smem + L::SUM_OFF);
  uint32_t* nan = reinterpret_cast<uint32_t*>(smem + L::NAN_OFF);
  uint32_t* badbits = reinterpret_cast<uint32_t*>(smem + L::BAD_OFF);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + (JOIN ? L::PART_OFF + L::PART : L::PART_SUM_OFF));
  if (threadIdx.x < D / kKv4Group) nan[threadIdx.x] = 0;
  griddep_launch_dependents();

  const int r = blockIdx.y;
  // a list's partitions side by side where they are a cluster
  const int h = JOIN ? blockIdx.x / p.max_splits : blockIdx.x % p.kv_heads;
  const int c = JOIN ? blockIdx.x - h * p.max_splits : blockIdx.x / p.kv_heads;
  const int col0 = blockIdx.z * NT * 8;
  const int cap = p.maxblk * BS;
  int ctx = __ldg(p.lens + r);
  const bool bad_len = ctx < 0 || ctx > cap;
  ctx = min(max(ctx, 0), cap);
  const int nsplit = partitions_of(ctx, p.split_tokens);
  const int G = p.group, NC = G * p.q_len, qh0 = h * G;
  if (c >= max(nsplit, 1)) {
    griddep_wait();
    if (bad_len && threadIdx.x == 0) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
    return;
  }
  const bool joins = JOIN && nsplit > 1;
  if (joins) cluster_arrive();  // CTAs without tokens have left, and no one writes to them
  const int tok0 = c * p.split_tokens, tok1 = partition_end(tok0, p.split_tokens, ctx);
  const int ntiles = (tok1 - tok0 + kTile - 1) / kTile;  // of the CTA

  // row of column n in q, out and the partials
  auto row_of = [&](int n) {
    const int qi = n / G;
    return (size_t)(r * p.q_len + qi) * p.q_heads + qh0 + (n - qi * G);
  };

  // Q^T as the B operand: lane (g, c) holds column g of each n-tile, elements
  // D/4 c + 4 ks + {0, 1} and {2, 3}
  uint2 raw[KSTEPS];
  auto load_q = [&](int nt) {
    const int n = col0 + nt * 8 + g;
    const uint2* q2 = reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + (n < NC ? row_of(n) : 0) * D + (D / 4) * c4);
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks) raw[ks] = n < NC ? __ldg(q2 + ks) : make_uint2(0u, 0u);
  };
  if (NT == 1) load_q(0);  // beside the table; more columns would take too many registers that long
  bool bad_id = false;
  {
    const int nblk = (tok1 - tok0 + BS - 1) / BS;
    const int entries = (ntiles * kTile + BS - 1) / BS;
    const int32_t* trow = p.tables + (size_t)r * p.maxblk + tok0 / BS;
    // a bad block, and one behind the last, is read as block 0 and counts as zeros
    for (int i = threadIdx.x; i < (entries + 31 & ~31); i += kWarps * 32) {
      int b = i < nblk ? __ldg(trow + i) : 0;
      const bool bad = b < 0 || b >= p.num_blocks;
      const uint32_t bits = __ballot_sync(kAll, bad);
      if (lane == 0) badbits[i >> 5] = bits;
      if (i < entries) tab[i] = bad ? 0 : b;
      bad_id |= bad;
    }
  }
  griddep_wait();
  if (bad_len && threadIdx.x == 0) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
  if (bad_id) record_error(p.err, PA_DEVERR_BLOCK_ID);
  const int ncols = min(NC - col0, NT * 8);  // of this CTA
  if (ctx == 0) {
    uint16_t* out = static_cast<uint16_t*>(p.out);  // 0 in either type
    for (int i = threadIdx.x; i < ncols * D; i += kWarps * 32) out[row_of(col0 + i / D) * D + i % D] = 0;
    return;
  }
  const bool any_bad = __syncthreads_or(bad_id);  // and the table is complete

  // Where this lane's elements are in a tile: K of token pi(g) (+ 8), V of c and c + 4 (+ 8)
  auto code_at = [](int t) { return BS < kTile ? t / BS * PAGE + t % BS * R::CODES : t * R::CODES; };
  auto scale_at = [](int t) {
    return BS < kTile ? t / BS * PAGE + BS * R::CODES + t % BS * R::SCALES : kTile * R::CODES + t * R::SCALES;
  };
  constexpr int VOFF = kTile * R::BYTES;
  const int pg = (g >> 1) + 4 * (g & 1);
  constexpr int CODE4 = BS < 8 ? PAGE : 4 * R::CODES, SCALE4 = BS < 8 ? PAGE : 4 * R::SCALES;  // to the token 4 behind
  constexpr int CODE8 = BS < kTile ? 8 / BS * PAGE : 8 * R::CODES, SCALE8 = BS < kTile ? 8 / BS * PAGE : 8 * R::SCALES;
  const uint32_t ring_at = smem_u32(smem + warp * L::WARP);
  const uint32_t kcode = ring_at + code_at(pg) + c4 * (4 * NW), kscale = ring_at + scale_at(pg) + c4 * (NW / 2);
  const uint32_t vcode = ring_at + VOFF + code_at(c4) + g * (D / 16);
  const uint32_t vscale = ring_at + VOFF + scale_at(c4) + (D == 128 ? g : g >> 1);
  // A tile is 2 * R::BYTES vectors of 16 bytes, K's and then V's, copied as they
  // are in the pages (of blocks of 32: the tile's half of the codes, then of the
  // scales); this lane copies vectors lane, lane + 32, ...
  constexpr int VECS = R::BYTES, SLOTS = (2 * VECS + 31) / 32;
  constexpr int PV = BS < kTile ? PAGE / 16 : VECS;  // vectors of a page in a tile
  uint8_t* ring = smem + warp * L::WARP;
  const uint32_t ring0 = ring_at + 16 * lane;
  const uint32_t block_bytes = (uint32_t)p.kv_heads * PAGE;
  // Where the lane's vectors are in a block.  Of blocks of 16 a tile is a run of
  // K's bytes and one of V's: two addresses and constants.
  constexpr bool RUN = BS == kTile;
  const uint8_t* src[RUN ? 2 : SLOTS];
  if constexpr (RUN) {
    src[0] = static_cast<const uint8_t*>(p.k_cache) + (int64_t)h * PAGE + 16 * lane;
    src[1] = static_cast<const uint8_t*>(p.v_cache) + (int64_t)h * PAGE + 16 * lane - 16 * VECS;
  } else {
#pragma unroll
    for (int q = 0; q < SLOTS; ++q) {
      const int id = lane + 32 * q, i = id % VECS;
      const int codes = kTile * R::CODES / 16;  // vectors of them, blocks of 32
      const int off = BS <= kTile || i < codes ? (i % PV) * 16 : BS * R::CODES + (i - codes) * 16;
      src[q] = static_cast<const uint8_t*>(id < VECS ? p.k_cache : p.v_cache) + (int64_t)h * PAGE + off;
    }
  }
  // entry of the table that holds a token of tile j
  auto entry = [](int j, int token) { return BS >= kTile ? j * kTile / BS : j * (kTile / BS) + token / BS; };
  auto issue = [&](int j, uint32_t slot) {  // tile j of the CTA to a place of the ring
    if (j < ntiles) {
      const uint32_t dst = ring0 + slot * L::TILE;
      const uint32_t block = (uint32_t)tab[entry(j, 0)];  // the only one, of blocks of 16 and 32
      const uint64_t at_block = (uint64_t)block * block_bytes;
      const uint8_t* kv[2];
      if constexpr (RUN) kv[0] = src[0] + at_block, kv[1] = src[1] + at_block;
#pragma unroll
      for (int q = 0; q < SLOTS; ++q) {
        const int id = lane + 32 * q, v = id % VECS;
        const uint8_t* s;
        if constexpr (RUN) {
          s = (32 * q + 32 <= VECS ? kv[0] : 32 * q >= VECS ? kv[1] : id < VECS ? kv[0] : kv[1]) + 512 * q;
        } else {
          s = src[q] + (BS > kTile ? at_block : (uint64_t)(uint32_t)tab[entry(j, v / PV * BS)] * block_bytes);
          if (BS > kTile) s += (j * kTile & (BS - 1)) * (v < kTile * R::CODES / 16 ? R::CODES : R::SCALES);
        }
        if (32 * q + 32 <= 2 * VECS || id < 2 * VECS) cp_async16_at(dst, 512 * q, s);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) issue(warp + i * kWarps, i);
  uint32_t slot = 0;

  uint32_t qf[NT][KSTEPS][2];
  float sl2[NT][2];  // softmax scale (log2 units) of the lane's two columns of each n-tile
  auto convert_q = [&](auto type) {
    using T = decltype(type);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (NT > 1) load_q(nt);
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        const uint2 w = raw[ks];
        top = fmaxf(top, fmaxf(fmaxf(fabsf(Elem<T>::lo(w.x)), fabsf(Elem<T>::hi(w.x))),
                               fmaxf(fabsf(Elem<T>::lo(w.y)), fabsf(Elem<T>::hi(w.y)))));
      }
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
      // 2^e <= top < 2^(e + 1); rows of zeros and of values that are not finite stay as they are
      int e = (int)(__float_as_uint(top) >> 23) - 127;  // of a subnormal -127: it is brought up less
      e = top > 0.f && top < INFINITY ? max(e - 13, -126) : 0;
      const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
      for (int ks = 0; ks < KSTEPS; ++ks) {
        const uint2 w = raw[ks];
        qf[nt][ks][0] = Elem<__half>::pack(Elem<T>::lo(w.x) * down, Elem<T>::hi(w.x) * down);
        qf[nt][ks][1] = Elem<__half>::pack(Elem<T>::lo(w.y) * down, Elem<T>::hi(w.y) * down);
      }
      const float back = p.scale_log2 * __uint_as_float((uint32_t)(127 + e) << 23);
      // accumulators hold columns 2c, 2c + 1 of the tile
      sl2[nt][0] = __shfl_sync(kAll, back, 8 * c4);
      sl2[nt][1] = __shfl_sync(kAll, back, 8 * c4 + 4);
    }
  };
  if (p.bf16) convert_q(__nv_bfloat16{});  // while the first tiles come
  else convert_q(__half{});

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

  // 16 tokens from ts on; `all`: every column sees all of them
  auto compute = [&](const uint32_t x, const int j, const auto all_t) {  // x: the tile's place in the ring
    constexpr bool all = decltype(all_t)::value;
    const int ts = tok0 + j * kTile;
    auto bad_block = [&](int token) {
      const int i = entry(j, token);
      return badbits[i >> 5] >> (i & 31) & 1;
    };
    float sacc[NT][2][4];  // even and odd steps: a chain of half the length
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) sacc[nt][k][0] = sacc[nt][k][1] = sacc[nt][k][2] = sacc[nt][k][3] = 0.f;
    uint32_t kw[2][NW], ks[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (NW == 4) {
        const uint4 w = lds4(x + kcode, e * CODE8);
        kw[e][0] = w.x, kw[e][1] = w.y, kw[e][2] = w.z, kw[e][3] = w.w;
        ks[e] = lds_u16(x + kscale, e * SCALE8);
      } else {
        const uint2 w = lds2(x + kcode, e * CODE8);
        kw[e][0] = w.x, kw[e][1] = w.y;
        ks[e] = lds_u8(x + kscale, e * SCALE8);
      }
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      uint32_t y[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        kv4_unpack(kw[e][i], y[e]);
        uint32_t s2 = kv4_scale2(NW == 4 && i >= 2 ? ks[e] >> 8 : ks[e] & 0xFFu);
        if (!all && bad_block(pg + 8 * e)) s2 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[e][k] = hmul2_u(y[e][k], s2);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a[4] = {y[0][2 * k], y[1][2 * k], y[0][2 * k + 1], y[1][2 * k + 1]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<__half>(sacc[nt][k], a, qf[nt][2 * i + k][0], qf[nt][2 * i + k][1]);
      }
    }

    const int t0 = ts + pg;  // the lane's score rows: tokens t0, t0 + 8
    uint32_t pb0[NT], pb1[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float s0 = all || t0 < lim[nt][0] ? (sacc[nt][0][0] + sacc[nt][1][0]) * sl2[nt][0] : -INFINITY;
      const float s1 = all || t0 < lim[nt][1] ? (sacc[nt][0][1] + sacc[nt][1][1]) * sl2[nt][1] : -INFINITY;
      const float s2 = all || t0 + 8 < lim[nt][0] ? (sacc[nt][0][2] + sacc[nt][1][2]) * sl2[nt][0] : -INFINITY;
      const float s3 = all || t0 + 8 < lim[nt][1] ? (sacc[nt][0][3] + sacc[nt][1][3]) * sl2[nt][1] : -INFINITY;
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

    uint32_t vs2[2];  // scales of the two tokens of each pair
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint32_t vs[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        vs[i] = lds_u8(x + vscale, e * SCALE8 + i * SCALE4);
        if constexpr (!all) {
          const int t = ts + c4 + 4 * i + 8 * e;
          if (t >= causal0 && t < tok1 && vs[i] >= kKv4FirstInf) {
            vs[i] = 0;
            atomicOr(&nan[D == 128 ? g : g >> 1], 1u << (t - causal0));
          }
          if (t >= tok1 || bad_block(c4 + 4 * i + 8 * e)) vs[i] = 0;
        }
      }
      vs2[e] = kv4_scale_pair(vs[0], vs[1]);
    }
    uint32_t va[2][2][D / 64];  // [e][token of the pair]
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (D == 128) {
          const uint2 w = lds2(x + vcode, e * CODE8 + i * CODE4);
          va[e][i][0] = w.x, va[e][i][1] = w.y;
        } else {
          va[e][i][0] = lds1(x + vcode, e * CODE8 + i * CODE4);
        }
      }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      uint32_t u[2][4], z[2][4];  // even and odd elements of the word, two tokens each
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t a = va[e][0][i], b = va[e][1][i];
        kv4_unpack(low_halves(a, b << 4), u[e]);
        kv4_unpack(low_halves(a >> 4, b), z[e]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[e][k] = hmul2_u(u[e][k], vs2[e]);
          z[e][k] = hmul2_u(z[e][k], vs2[e]);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t a[4] = {u[0][k], z[0][k], u[1][k], z[1][k]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<__half>(acc[nt][4 * i + k], a, pb0[nt], pb1[nt]);
      }
    }
  };

  const int nfull = any_bad ? 0 : min(max(min(tok1, causal0) - tok0, 0) / kTile, ntiles);  // seen whole by every column
  for (int j = warp; j < ntiles; j += kWarps) {
    cp_async_wait<kDepth - 2>();
    __syncwarp();  // every lane's part of tile j is there, and every lane is done with the one before
    issue(j + (kDepth - 1) * kWarps, slot == 0 ? kDepth - 1 : slot - 1);
    const uint32_t x = slot * L::TILE;
    slot = slot + 1 == kDepth ? 0 : slot + 1;
    if (j < nfull) compute(x, j, std::true_type{});
    else compute(x, j, std::false_type{});
  }
  cp_async_wait_all();
  __syncwarp();  // the ring becomes the outputs' place

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
  float* po = reinterpret_cast<float*>(ring);
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
  // a cluster's outputs are joined by all of its CTAs, `per` vectors of four each
  float* parts = reinterpret_cast<float*>(smem + L::PART_SUM_OFF);
  const int per = joins ? (ncols * (D / 4) + nsplit - 1) / nsplit : 0;
  if (joins) cluster_wait();  // every CTA has begun
  auto put_out = [&](size_t row, int d, float4 o, float sum) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a NaN sum stays one
    o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + row * D + d) =
        p.bf16 ? make_uint2(Elem<__nv_bfloat16>::pack(o.x, o.y), Elem<__nv_bfloat16>::pack(o.z, o.w))
               : make_uint2(Elem<__half>::pack(o.x, o.y), Elem<__half>::pack(o.z, o.w));
  };
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
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * L::WARP) + n * L::ROW + d);
      o.x += a * x.x, o.y += a * x.y, o.z += a * x.z, o.w += a * x.w;
      sum += a * sums[(kWarps + w) * NT * 8 + n];
    }
    // a token behind causal0 that is not a number, for the columns that see it
    const int nsee = min(max(min(tok1, ctx - (p.q_len - 1 - (col0 + n) / G)) - causal0, 0), 31);
    if (nan[d / kKv4Group] & ((1u << nsee) - 1u)) o = make_float4(NAN, NAN, NAN, NAN);
    const size_t row = row_of(col0 + n);
    if (nsplit == 1) {
      put_out(row, d, o, sum);
    } else if (joins) {
      const int to = i / per;
      cluster_st4(smem_u32(smem + L::PART_OFF) + (c * per + i - to * per) * 16, to, o);
      const int w = d / 4;  // a lane per CTA: the column's sums
      if (w < nsplit) {
        cluster_st(smem_u32(parts + c * NT * 8 + n), w, M);
        cluster_st(smem_u32(parts + (kMaxCluster + c) * NT * 8 + n), w, sum);
      }
    } else {
      *reinterpret_cast<float4*>(p.part_o + (row * p.max_splits + c) * D + d) = o;
      if (d == 0) {
        p.part_m[row * p.max_splits + c] = M;
        p.part_l[row * p.max_splits + c] = sum;
      }
    }
  }
  if (!joins) return;

  // this CTA's outputs, from the parts that the partitions have written to it
  cluster_sync();
  for (int j = threadIdx.x; j < per; j += kWarps * 32) {
    const int i = c * per + j;
    if (i >= ncols * (D / 4)) break;
    const int n = i / (D / 4), d = 4 * (i % (D / 4));
    float M = -INFINITY;
    for (int w = 0; w < nsplit; ++w) M = fmaxf(M, parts[w * NT * 8 + n]);
    const float ref = M == -INFINITY ? 0.f : M;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll 4
    for (int w = 0; w < nsplit; ++w) {
      const float a = ex2_approx(parts[w * NT * 8 + n] - ref);
      const float4 x = *reinterpret_cast<const float4*>(smem + L::PART_OFF + (w * per + j) * 16);
      o.x += a * x.x, o.y += a * x.y, o.z += a * x.z, o.w += a * x.w;
      sum += a * parts[(kMaxCluster + w) * NT * 8 + n];
    }
    put_out(row_of(col0 + n), d, o, sum);
  }
}

template <int D, int NT, int BS>
cudaError_t launch_t(const Kv4DecodeParams& p, cudaStream_t stream) {
  using L = Kv4DecodeSmem<D, NT>;
  static_assert(L::bytes(kMaxEntries + 4, false) <= 48 * 1024 && L::bytes(kKv4ClusterEntries + 4, true) <= 48 * 1024,
                "no attribute needed");
  const dim3 grid((unsigned)(p.max_splits * p.kv_heads), p.num_seqs, (p.group * p.q_len + NT * 8 - 1) / (NT * 8));
  const int smem = L::bytes(p.tab_entries + 4, p.cluster);
  if (p.cluster) {
    auto kern = kv4_decode_kernel<D, NT, BS, true>;
    static bool attr_set[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      if (dev < 64) attr_set[dev] = true;
    }
    return launch_pdl_cluster(kern, p.max_splits, grid, dim3(kWarps * 32), smem, stream, p);
  }
  return launch_pdl(kv4_decode_kernel<D, NT, BS, false>, grid, dim3(kWarps * 32), smem, stream, p);
}

template <int D, int BS>
cudaError_t launch_nt(const Kv4DecodeParams& p, cudaStream_t stream) {
  return p.group * p.q_len <= 8 ? launch_t<D, 1, BS>(p, stream) : launch_t<D, 2, BS>(p, stream);
}

template <int D>
cudaError_t launch_bs(const Kv4DecodeParams& p, cudaStream_t stream) {
  switch (p.block_size) {
    case 4: return launch_nt<D, 4>(p, stream);
    case 8: return launch_nt<D, 8>(p, stream);
    case 16: return launch_nt<D, 16>(p, stream);
    default: return launch_nt<D, 32>(p, stream);
  }
}

}  // namespace

cudaError_t launch_kv4_decode(const Kv4DecodeParams& p, int head_dim, cudaStream_t stream) {
  return head_dim == 128 ? launch_bs<128>(p, stream) : launch_bs<64>(p, stream);
}

}  // namespace pa
