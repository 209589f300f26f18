// Chunked prefill over a 4-bit paged cache (see kv4.cuh for the page) on the
// 5th-generation tensor cores, sm_103a.
//
// The decomposition is attn_tc.cu's: a CTA owns two tiles of 128 rows (query,
// head of the group) of one (request, KV head) and walks the keys they see 64
// at a time; S_x = Q_x K^T into one of two tensor-memory buffers per tile, the
// softmax in registers, P over the same buffer, O_x += P_x V with P from tensor
// memory.  What differs:
//
//  * K and V tiles are not loaded but made: pages come by bulk copy (their codes
//    to one place and their scales to another, so that a token is found by its
//    number whatever the block size), and a warp writes the fp16 tile in the
//    128-byte-swizzled layout that the MMAs read (exact: kv4.cuh).  Three warps
//    make K tiles in turn and three V tiles; a warp's next pages come while the
//    others work.  A lane takes the 16 elements of a scale at a time; lanes of
//    the second half-row store their two 16-byte pieces in the other order, so
//    that a store's eight lanes meet eight banks.
//  * All operands are fp16 whatever the type of q (see kv4_decode.cu): a row of
//    Q is brought to [2^13, 2^14) by a power of two that its softmax takes back.
//  * V rows behind the last key are zeros; a V group that is not a number becomes
//    zeros too, and the first such token of each group of elements is kept, so
//    that the rows that see it get their NaN at the end and no other row does.
//  * A context may be cut into partitions of split_tokens keys, a unit each,
//    where there are few units; a merge joins them.
//
// Measured on GB300 in us, a chunk of 2048 queries over 34816 tokens, 64/8 heads
// (floor 1179 at the measured bf16 rate), and eight chunks of 257..768 over 509..
// 4079 tokens more, 32/8 (floor 97):
//   one warp makes K, one V                                4508   413
//   three each, codes and scales apart                     2193   234
//   a lane's addresses worked out once, scales as zeros    1752   198
//   Q and outputs by whole lines, longest requests first   1752   180
//   two partitions where rounds of units fill the SMs      1639   180
//   Q and the first table entries before the barriers      1638   180
// What is left: about 9 us to start and end a unit of 256 rows (barriers and
// tensor memory 1, table and first pages 1.8, their tile and Q 2.5, outputs 3),
// with nothing under them, a fifth of the second case; the MMAs of a tile at the
// measured rate are 0.66 us of its 0.79.
// Tried and left: CTAs that take over further units (by cluster launch control),
// whose makers are a unit ahead of the softmax (1680 and 183: the counters across
// units take registers that the softmax has not, 3 % of every tile, as much as the
// overlap gives; asked for at a unit's start instead of its end 1688 and 194, as
// units are then held by busy CTAs while others have none); partitions joined in a
// cluster, through the places of the K and V tiles (up to five, 64 KB and more a
// CTA: four short chunks 22.6 in two, and where units go in rounds 1667 instead of
// 1638 and worse).
//
// Warps: 0, 1 MMA issuers of tiles A, B; 2..7 make K and V; 8..11 softmax of
// tile A, 12..15 of tile B.  Every wait is bounded.
#include <float.h>
#include <limits.h>

#include "kv4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRows = 128;  // rows per Q tile
constexpr int kKeys = 64;   // keys per K/V tile
constexpr int kStages = 4;  // of K and of V, fp16
constexpr int kMakers = 3;  // warps that make K tiles, and V tiles, in turn
constexpr int kThreads = 32 * 16;
constexpr int kSoftmaxWarp0 = 8;
constexpr uint32_t kTmem = 512;
constexpr unsigned kAll = 0xffffffffu;
constexpr float kRescale = 8.f;
constexpr float kShift = 7.f;  // weights are 2^(s - m + kShift) <= 2^15

template <int D>
struct Kv4PrefillSmem {
  using Tile = KvTile<D, 16, kKeys>;
  static constexpr int QHALF = kRows * 128;
  static constexpr int QTILE = D / 64 * QHALF;
  static constexpr int RAW = kKeys * Kv4Row<D>::BYTES;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * QTILE;
  static constexpr int V_OFF = K_OFF + kStages * Tile::BYTES;
  static constexpr int RAW_OFF = V_OFF + kStages * Tile::BYTES;  // a tile per maker: its codes, then its scales
  static constexpr int BAR_OFF = RAW_OFF + 2 * kMakers * RAW;
  static constexpr int NBARS = 4 * kStages + 2 * kMakers + 16;
  static constexpr int SLOT_OFF = BAR_OFF + NBARS * 8;
  static constexpr int NAN_OFF = SLOT_OFF + 8;
  static constexpr int SCALE_OFF = NAN_OFF + D / kKv4Group * 4;  // softmax scale of each row
  static constexpr int BYTES = SCALE_OFF + 2 * kRows * 4 + 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(kMakers <= kStages, "the last tile of every maker is still the last of its stage at the end");
};

// barrier indices
constexpr int B_KFULL = 0;                      // [kStages] the producer warp wrote K_j
constexpr int B_KEMPTY = B_KFULL + kStages;     // [kStages] one commit per issuer after S_x(j)
constexpr int B_VFULL = B_KEMPTY + kStages;
constexpr int B_VEMPTY = B_VFULL + kStages;     // [kStages] one commit per issuer after P.V_x(j)
constexpr int B_RAW = B_VEMPTY + kStages;       // [maker] its pages landed
constexpr int B_SFULL = B_RAW + 2 * kMakers;    // [2 Q tiles][2 S buffers]
constexpr int B_PFULL = B_SFULL + 4;            // [2][2] four softmax warps
constexpr int B_OFULL = B_PFULL + 4;            // [2][2] P.V_x(j) complete
constexpr int B_QFULL = B_OFULL + 4;            // [2]
constexpr int B_MMADONE = B_QFULL + 2;
constexpr int B_BEGUN = B_MMADONE + 1;          // tile A's first P is there (its B_PFULL may be a phase further by the time B looks)
static_assert(B_BEGUN + 1 == 4 * kStages + 2 * kMakers + 16, "barrier count");

__device__ __forceinline__ void st_shared4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Named barriers of the start: of the warps that are no softmax warps, and of warp
// 0 and those.
constexpr int kSetUpBar = 1, kReadyBar = 2;
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int threads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

struct Unit {
  int r, h, row0, part, qs, chunk, p0, rows, k0, kend, ntiles;
  int code;  // error of a refused request
};

// Units are numbered (request, partition), then row tile in reverse, then head:
// the last row tiles of a chunk see the most keys.
__device__ __forceinline__ Unit unit_of(const Kv4PrefillParams& p, int u) {
  Unit w{};
  const int per_z = p.row_tiles * p.kv_heads;
  const int z = u / per_z, rem = u - z * per_z, rt = rem / p.kv_heads;
  w.h = rem - rt * p.kv_heads;
  w.row0 = (p.row_tiles - 1 - rt) * 2 * kRows;
  w.r = z / p.max_splits;
  w.part = z - w.r * p.max_splits;
  w.qs = __ldg(p.q_start + w.r);
  const int qe = __ldg(p.q_start + w.r + 1), ctx = __ldg(p.lens + w.r);
  w.chunk = qe - w.qs;
  w.p0 = ctx - w.chunk;
  if (w.qs < 0 || qe < w.qs || qe > p.total_q || w.chunk > p.max_q_len || ctx < w.chunk || ctx > p.maxblk * p.block_size) {
    w.code = PA_DEVERR_QUERY_RANGE;
    return w;
  }
  w.rows = w.chunk * p.group;
  if (w.row0 >= w.rows) return w;
  const int last_row = min(w.row0 + 2 * kRows, w.rows) - 1;
  w.k0 = w.part * p.split_tokens;
  w.kend = partition_end(w.k0, p.split_tokens, w.p0 + last_row / p.group + 1);
  if (w.k0 < w.kend) w.ntiles = (w.kend - w.k0 + kKeys - 1) / kKeys;
  return w;
}

// Where units outnumber the SMs the last ones decide when the kernel ends, so
// requests of one partition run longest first: the request of index r in that
// order, ties by number, among the kWindow around it.  Every thread calls it.
constexpr int kWindow = 128;
__device__ __forceinline__ int longest_first(const Kv4PrefillParams& p, int r, int* scratch) {
  const int w0 = r / kWindow * kWindow, n = min(kWindow, p.num_reqs - w0), t = threadIdx.x;
  int len = 0;
  if (t < n) scratch[t] = len = __ldg(p.lens + w0 + t);
  __syncthreads();
  if (t < n) {
    int before = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) before += scratch[i] > len || (scratch[i] == len && i < t);
    if (before == r - w0) scratch[kWindow] = w0 + t;
  }
  __syncthreads();
  return scratch[kWindow];
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const Kv4PrefillParams p) {
  using L = Kv4PrefillSmem<D>;
  using Tile = typename L::Tile;
  using R = Kv4Row<D>;
  constexpr int KSTEPS = D / 16;
  constexpr int PSTEPS = kKeys / 16;
  constexpr int ROW_BYTES = 2 * D;  // of a row of Q
  constexpr uint32_t O_COL = 4 * kKeys;
  constexpr uint32_t IDESC_S = idesc_f16<__half>(kRows, kKeys, false);
  constexpr uint32_t IDESC_O = idesc_f16<__half>(kRows, D, true);

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::SLOT_OFF);
  int* first_nan = reinterpret_cast<int*>(smem + L::NAN_OFF);  // per group of elements: its first V token that is NaN
  float* scales = reinterpret_cast<float*>(smem + L::SCALE_OFF);
  auto bar = [&](int i) { return smem_u32(&bars[i]); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  int u = blockIdx.x;
  if (p.longest_first) {
    __shared__ int longest[kWindow + 1];
    const int per_r = p.row_tiles * p.kv_heads, r = u / per_r;
    u += (longest_first(p, r, longest) - r) * per_r;
  }
  const Unit w = unit_of(p, u);
  if (w.code || w.ntiles == 0) {
    griddep_wait();
    if (w.code && w.h == 0 && w.row0 == 0 && w.part == 0 && threadIdx.x == 0) record_error(p.err, w.code);
    return;
  }
  const int tiles = w.row0 + kRows < w.rows ? 2 : 1;  // Q tiles with rows

  if (threadIdx.x < D / kKv4Group) first_nan[threadIdx.x] = INT_MAX;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(B_KFULL + i), 1);
      mbar_init(bar(B_KEMPTY + i), tiles);
      mbar_init(bar(B_VFULL + i), 1);
      mbar_init(bar(B_VEMPTY + i), tiles);
    }
    for (int i = 0; i < 2 * kMakers; ++i) mbar_init(bar(B_RAW + i), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(B_SFULL + i), 1);
      mbar_init(bar(B_PFULL + i), 4);
      mbar_init(bar(B_OFULL + i), 1);
    }
    mbar_init(bar(B_QFULL), 4);
    mbar_init(bar(B_QFULL + 1), 4);
    mbar_init(bar(B_MMADONE), tiles);
    mbar_init(bar(B_BEGUN), 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmem);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  // Barriers and tensor memory take about a microsecond: the softmax warps load Q
  // meanwhile and meet warp 0 behind it, the makers have their first table entries.
  tc_fence_before();
  if (warp == 0) named_arrive(kReadyBar, 32 + 32 * (kThreads / 32 - kSoftmaxWarp0));

  if (warp >= 2 && warp < kSoftmaxWarp0) {
    // ------------------------------------------------------------ K and V
    // warps 2, 4, 6 make K tiles, 3, 5, 7 V tiles, every kMakers-th each
    const int maker = warp - 2, isv = maker & 1, first = maker >> 1;
    const uint8_t* cache = static_cast<const uint8_t*>(isv ? p.v_cache : p.k_cache);
    uint8_t* codes = smem + L::RAW_OFF + maker * L::RAW;
    uint8_t* raw_scales = codes + kKeys * R::CODES;
    uint8_t* tile0 = smem + (isv ? L::V_OFF : L::K_OFF);
    const int full0 = isv ? B_VFULL : B_KFULL, empty0 = isv ? B_VEMPTY : B_KEMPTY;
    const uint32_t rawbar = bar(B_RAW + maker);
    const int32_t* trow = p.tables + (size_t)w.r * p.maxblk;
    const int bs = p.block_size, bsh = p.block_shift, page = bs * R::BYTES;
    const uint64_t pol = p.row_tiles == 1 ? policy_evict_first() : policy_evict_last();  // other row tiles re-read them
    // pages of tile j: lane 2i their i-th's codes, lane 2i + 1 its scales
    auto entry = [&](int j) {
      const int ts = w.k0 + j * kKeys, npages = (min(kKeys, w.kend - ts) + bs - 1) >> bsh;
      return (lane >> 1) < npages ? __ldg(trow + (ts >> bsh) + (lane >> 1)) : -1;
    };
    auto issue = [&](int j, int b) {
      const int ts = w.k0 + j * kKeys;
      const int npages = (min(kKeys, w.kend - ts) + bs - 1) >> bsh;
      const int i = lane >> 1, part = lane & 1;
      const bool mine = i < npages;
      if (mine && (b < 0 || b >= p.num_blocks)) {
        record_error(p.err, PA_DEVERR_BLOCK_ID);
        b = -1;
      }
      const int pages = __popc(__ballot_sync(kAll, b >= 0)) >> 1;
      if (lane == 0) mbar_arrive_expect_tx(rawbar, pages * page);
      __syncwarp();
      if (mine) {
        const int bytes = bs * (part ? R::SCALES : R::CODES);
        uint8_t* dst = (part ? raw_scales : codes) + i * bytes;
        if (b >= 0) {
          bulk_load_hint(smem_u32(dst), cache + ((size_t)b * p.kv_heads + w.h) * page + (part ? bs * R::CODES : 0), bytes,
                         rawbar, pol);
        } else {  // a bad block id: zeros
          for (int k = 0; k < bytes; k += 16) *reinterpret_cast<uint4*>(dst + k) = make_uint4(0, 0, 0, 0);
        }
      }
      __syncwarp();  // the zeros before other lanes read them
    };
    const int b0 = first < w.ntiles ? entry(first) : -1;
    named_sync(kSetUpBar, 32 * kSoftmaxWarp0);
    griddep_wait();
    if (first < w.ntiles) issue(first, b0);
    bool failed = false;
    int n = 0;  // tiles made
    for (int j = first; j < w.ntiles; j += kMakers, ++n) {
      const int s = j % kStages;
      if (!__all_sync(kAll, mbar_wait(rawbar, n & 1) &&
                                (j < kStages || mbar_wait(bar(empty0 + s), (j / kStages - 1) & 1)))) {
        failed = true;
        break;
      }
      const int ts = w.k0 + j * kKeys;
      const int nvalid = min(kKeys, w.kend - ts);
      if (nvalid < kKeys) {
        // rows behind the last key: their scales, which the copies are done with, become zeros
        for (int row = nvalid + lane; row < kKeys; row += 32) {
          uint32_t* at = reinterpret_cast<uint32_t*>(raw_scales + row * R::SCALES);
#pragma unroll
          for (int i = 0; i < R::SCALES / 4; ++i) at[i] = 0u;
        }
        __syncwarp();
      }
      // The lane's row in step i is row0 + STEP i, so in the swizzle its 16-byte
      // piece c is at c ^ (row % 8): row0 and a bit that alternates.
      constexpr int PER_ROW = D / kKv4Group, STEP = 32 / PER_ROW;  // rows of a step: 4, or 8 of 64 elements
      const int g = lane % PER_ROW, row0 = lane / PER_ROW, flip = g >> 2;
      const uint32_t place = smem_u32(tile0 + s * Tile::BYTES) + row0 * 128;
      uint32_t at0[2], at1[2];  // of the first and the second store, even and odd steps
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int sw = (row0 + STEP * e) & 7, c = 2 * g + flip;
        at0[e] = place + (c >> 3) * Tile::HALF + (((c & 7) ^ sw) << 4);
        at1[e] = place + (c >> 3) * Tile::HALF + (((c & 7 ^ 1) ^ sw) << 4);
      }
      const uint8_t* code = codes + row0 * R::CODES + 8 * g;
      const uint8_t* scale = raw_scales + row0 * R::SCALES + g;
#pragma unroll
      for (int i = 0; i < kKeys / STEP; ++i) {
        const uint2 c = *reinterpret_cast<const uint2*>(code + i * STEP * R::CODES);
        uint32_t byte = scale[i * STEP * R::SCALES];
        if (isv && byte >= kKv4FirstInf) {
          byte = 0;
          atomicMin(&first_nan[g], ts + row0 + i * STEP);
        }
        const uint32_t s2 = kv4_scale2(byte);
        uint32_t x[8];
        kv4_unpack(flip ? c.y : c.x, *reinterpret_cast<uint32_t(*)[4]>(&x[0]));
        kv4_unpack(flip ? c.x : c.y, *reinterpret_cast<uint32_t(*)[4]>(&x[4]));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = hmul2_u(x[e], s2);
        st_shared4(at0[i & 1] + i * STEP * 128, make_uint4(x[0], x[1], x[2], x[3]));
        st_shared4(at1[i & 1] + i * STEP * 128, make_uint4(x[4], x[5], x[6], x[7]));
      }
      fence_proxy_async_smem();  // the tile before the MMAs, the pages before the next copies over them
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(full0 + s));
      if (j + kMakers < w.ntiles) issue(j + kMakers, entry(j + kMakers));
    }
    if (failed) {
      if (lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
      mbar_wait(rawbar, n & 1);  // copies in flight land before exit (bounded)
    }
  } else if (warp < 2) {
    // ------------------------------------------------------------ MMA issuers
    named_sync(kSetUpBar, 32 * kSoftmaxWarp0);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int x = warp;
    if (x < tiles) {
      bool ok = true;
      const uint32_t kbase = smem_u32(smem + L::K_OFF), vbase = smem_u32(smem + L::V_OFF);
      const uint32_t qa = smem_u32(smem + L::Q_OFF + x * L::QTILE);
      const uint32_t sd = tmem + 2 * x * kKeys, od = tmem + O_COL + x * D;
      auto issue_pv = [&](int t) -> bool {
        const int pb = t & 1, vst = t % kStages;
        if (!__all_sync(kAll, mbar_wait(bar(B_PFULL + 2 * x + pb), (t >> 1) & 1) &&
                                  mbar_wait(bar(B_VFULL + vst), (t / kStages) & 1)))
          return false;
        if (x == 0 && t == 0 && lane == 0) mbar_arrive(bar(B_BEGUN));
        tc_fence_after();
        const uint32_t vb = vbase + vst * Tile::BYTES;
#pragma unroll
        for (int kk = 0; kk < PSTEPS; ++kk)
          tc_mma_f16_ts_warp(od, sd + pb * kKeys + kk * 8, smem_desc_sw128(vb + kk * 2048, Tile::HALF, 1024), IDESC_O,
                             (t > 0 || kk > 0) ? 1u : 0u);
        tc_commit_warp(bar(B_OFULL + 2 * x + pb));
        tc_commit_warp(bar(B_VEMPTY + vst));
        return true;
      };
      ok = __all_sync(kAll, mbar_wait(bar(B_QFULL + x), 0));
      // tile B starts half a key tile behind tile A, so that the two softmaxes alternate
      if (ok && x == 1) ok = __all_sync(kAll, mbar_wait(bar(B_BEGUN), 0));
      for (int j = 0; ok && j < w.ntiles; ++j) {
        const int s = j % kStages, b = j & 1;
        // S_x(j) overwrites P_x(j - 2)
        ok = __all_sync(kAll, mbar_wait(bar(B_KFULL + s), (j / kStages) & 1) &&
                                  (j < 2 || mbar_wait(bar(B_OFULL + 2 * x + b), ((j - 2) >> 1) & 1)));
        if (!ok) break;
        tc_fence_after();
        const uint32_t kb = kbase + s * Tile::BYTES;
#pragma unroll
        for (int ks = 0; ks < KSTEPS; ++ks)
          tc_mma_f16_warp(sd + b * kKeys, smem_desc_sw128(qa + (ks >> 2) * L::QHALF + (ks & 3) * 32, 16, 1024),
                          smem_desc_sw128(kb + (ks >> 2) * Tile::HALF + (ks & 3) * 32, 16, 1024), IDESC_S,
                          ks > 0 ? 1u : 0u);
        tc_commit_warp(bar(B_SFULL + 2 * x + b));
        tc_commit_warp(bar(B_KEMPTY + s));
        if (j > 0) ok = issue_pv(j - 1);
      }
      if (ok) ok = issue_pv(w.ntiles - 1);
      if (!ok && lane == 0) record_error(p.err, PA_DEVERR_TIMEOUT);
      tc_commit_warp(bar(B_MMADONE));
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int x = (warp - kSoftmaxWarp0) >> 2;
    const int quarter = warp & 3, row = quarter * 32 + lane;
    if (x >= tiles) named_sync(kReadyBar, 32 + 32 * (kThreads / 32 - kSoftmaxWarp0));
    if (x < tiles) {
      const int grow = w.row0 + x * kRows + row;
      const int lim = grow < w.rows ? w.p0 + grow / G : -1;  // last key this row sees
      // The warp's 32 rows of Q -> shared memory (K-major, 128-byte swizzle), a row
      // by D/8 neighbouring lanes: a row per thread would touch 32 lines a load
      // (measured: 5 us for the tile instead of 1)
      constexpr int PIECES = D / 8, AT_ONCE = 32 / PIECES;  // 16-byte pieces of a row; rows a load takes
      const int piece = lane % PIECES, row_in = lane / PIECES;
      // row of q and out, in heads, of the warp's row `lane`; -1: a padding row.  The
      // others' come by shuffles: a division each would cost more than the loads
      auto own_row = [&](const Unit& w) {
        const int n = w.row0 + x * kRows + row, i = n / G;
        return n < w.rows ? (w.qs + i) * p.q_heads + w.h * G + (n - i * G) : -1;
      };
      uint8_t* qt = smem + L::Q_OFF + x * L::QTILE;
      {
        constexpr int BATCH = 8;
        const int own = own_row(w);
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += BATCH * AT_ONCE) {
          uint4 v[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int at = __shfl_sync(kAll, own, r0 + i * AT_ONCE + row_in);
            v[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + (int64_t)at * D) + piece)
                           : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int r = r0 + i * AT_ONCE + row_in, tr = quarter * 32 + r;
            const uint32_t e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            float top = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, fmaxf(fabsf(Elem<T>::lo(e[k])), fabsf(Elem<T>::hi(e[k]))));
#pragma unroll
            for (int o = 1; o < PIECES; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
            int ex = (int)(__float_as_uint(top) >> 23) - 127;  // 2^ex <= top; of a subnormal -127: it is brought up less
            ex = top > 0.f && top < INFINITY ? max(ex - 13, -126) : 0;
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            uint32_t y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = Elem<__half>::pack(Elem<T>::lo(e[k]) * down, Elem<T>::hi(e[k]) * down);
            *reinterpret_cast<uint4*>(qt + (piece >> 3) * L::QHALF + tr * 128 + (((piece & 7) ^ (tr & 7)) << 4)) =
                make_uint4(y[0], y[1], y[2], y[3]);
            // a masked score is -inf and must stay so: not below the smallest normal number
            if (piece == 0) scales[x * kRows + tr] = fmaxf(p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23), FLT_MIN);
          }
        }
        fence_proxy_async_smem();
        named_sync(kReadyBar, 32 + 32 * (kThreads / 32 - kSoftmaxWarp0));
        if (lane == 0) mbar_arrive(bar(B_QFULL + x));
      }
      tc_fence_after();
      const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16, tmem = *tmem_slot;
      const uint32_t scol0 = tmem + lane_addr + 2 * x * kKeys, ocol = tmem + lane_addr + O_COL + x * D;
      const float sl2 = scales[x * kRows + row];
      griddep_wait();  // before writing outputs

      bool ok = true;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < w.ntiles; ++j) {
        const int sb = j & 1;
        const uint32_t scol = scol0 + sb * kKeys;
        if (!__all_sync(kAll, mbar_wait(bar(B_SFULL + 2 * x + sb), (j >> 1) & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int nvis = lim - (w.k0 + j * kKeys) + 1;  // keys of this tile the row sees
        float sv[kKeys];
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) tmem_ld32(scol + 32 * c, *reinterpret_cast<float(*)[32]>(&sv[32 * c]));
        tmem_wait_ld();
        // raw scores meet the scale's sign before the maximum
        if (p.negative) {
#pragma unroll
          for (int e = 0; e < kKeys; ++e) sv[e] = -sv[e];
        }
        if (!__all_sync(kAll, nvis >= kKeys) || j == w.ntiles - 1) {
          const int n = min(nvis, w.kend - (w.k0 + j * kKeys));
#pragma unroll
          for (int e = 0; e < kKeys; ++e) sv[e] = e < n ? sv[e] : -INFINITY;
        }
        float ma = -INFINITY, mb = -INFINITY, mc = -INFINITY, md = -INFINITY;
#pragma unroll
        for (int e = 0; e < kKeys; e += 8) {
          ma = fmax3(ma, sv[e], sv[e + 1]);
          mb = fmax3(mb, sv[e + 2], sv[e + 3]);
          mc = fmax3(mc, sv[e + 4], sv[e + 5]);
          md = fmax3(md, sv[e + 6], sv[e + 7]);
        }
        const float mx = fmax3(ma, mb, fmaxf(mc, md)) * sl2;
        const bool raise = mx > m + kRescale;
        const float alpha = (raise && m != -INFINITY) ? ex2_approx(m - mx) : 1.f;
        const bool rescale = __any_sync(kAll, alpha != 1.f);
        if (raise) {
          l = m == -INFINITY ? 0.f : l * alpha;
          m = mx;
        }
        const float neg_m = m == -INFINITY ? 0.f : kShift - m;
        float sx[4] = {0.f, 0.f, 0.f, 0.f}, sy[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kKeys / 32; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float a0, a1;
            ffma2(a0, a1, sv[32 * c + e], sv[32 * c + e + 1], sl2, sl2, neg_m, neg_m);
            const float p0 = ex2_approx(a0), p1 = ex2_approx(a1);
            const int k = (e >> 1) & 3;
            fadd2(sx[k], sy[k], sx[k], sy[k], p0, p1);
            pk[e >> 1] = Elem<__half>::pack(p0, p1);
          }
          tmem_st16u(scol + 16 * c, pk);
        }
        if (rescale) {
          // O_x before P.V_x(j) starts, once P.V_x(j - 1) has completed
          if (!mbar_wait(bar(B_OFULL + 2 * x + ((j - 1) & 1)), ((j - 1) >> 1) & 1)) ok = false;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            float ov[16];
            tmem_ld16(ocol + 16 * c, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] *= alpha;
            tmem_st16u(ocol + 16 * c, *reinterpret_cast<const uint32_t(*)[16]>(ov));
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PFULL + 2 * x + sb));
        l += ((sx[0] + sy[0]) + (sx[1] + sy[1])) + ((sx[2] + sy[2]) + (sx[3] + sy[3]));
        if (!__all_sync(kAll, ok)) {
          ok = false;
          break;
        }
      }
      const int last = w.ntiles - 1;
      // the unit's last P.V, and (for first_nan) the V makers' last arrivals
      if (ok) ok = mbar_wait(bar(B_OFULL + 2 * x + (last & 1)), (last >> 1) & 1);
      for (int j = max(last - kMakers + 1, 0); j <= last; ++j)
        ok = ok && mbar_wait(bar(B_VFULL + j % kStages), (j / kStages) & 1);
      if (__all_sync(kAll, ok)) {
        tc_fence_after();
        // the unit once more: kept through the loop above, its fields would spill
        int again = u;
        asm volatile("" : "+r"(again));
        const Unit w = unit_of(p, again);
        const int own = own_row(w);
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
        // O through the Q tile's place (its MMAs have completed), 256 bytes of each
        // of the warp's rows at a time, so that a store's lanes write whole rows
        uint8_t* mine = smem + L::Q_OFF + x * L::QTILE + quarter * (L::QTILE / 4);
        const bool whole = p.max_splits == 1;
        auto put = [&](int c, uint4 v) {  // 16-byte piece c of this thread's row
          *reinterpret_cast<uint4*>(mine + lane * ROW_BYTES + ((c ^ (lane & 7)) << 4)) = v;
        };
        auto get = [&](int r, int c) { return *reinterpret_cast<const uint4*>(mine + r * ROW_BYTES + ((c ^ (r & 7)) << 4)); };
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float ov[32];
          tmem_ld32(ocol + 32 * c, ov);  // warp-collective
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            if (first_nan[2 * c + k] <= lim) {
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[16 * k + e] = NAN;
            }
          }
          if (whole) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              put(4 * c + q, make_uint4(Elem<T>::pack(ov[8 * q] * inv, ov[8 * q + 1] * inv),
                                        Elem<T>::pack(ov[8 * q + 2] * inv, ov[8 * q + 3] * inv),
                                        Elem<T>::pack(ov[8 * q + 4] * inv, ov[8 * q + 5] * inv),
                                        Elem<T>::pack(ov[8 * q + 6] * inv, ov[8 * q + 7] * inv)));
          } else {
            // 32 fp32 columns: a quarter of the row (half, of 64 elements)
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q)
              put(q, make_uint4(__float_as_uint(ov[4 * q]), __float_as_uint(ov[4 * q + 1]), __float_as_uint(ov[4 * q + 2]),
                                __float_as_uint(ov[4 * q + 3])));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // four rows a store, 128 bytes each
              const int r = 4 * i + (lane >> 3), at8 = lane & 7;
              const int at = __shfl_sync(kAll, own, r);
              if (at >= 0)
                reinterpret_cast<uint4*>(p.part_o + ((size_t)at * p.max_splits + w.part) * D + 32 * c)[at8] = get(r, at8);
            }
          }
        }
        if (whole) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 32 / AT_ONCE; ++i) {
            const int r = i * AT_ONCE + row_in;
            const int at = __shfl_sync(kAll, own, r);
            if (at >= 0) reinterpret_cast<uint4*>(static_cast<T*>(p.out) + (int64_t)at * D)[piece] = get(r, piece);
          }
        } else if (own >= 0) {
          const size_t pr = (size_t)own * p.max_splits + w.part;
          p.part_m[pr] = m;
          p.part_l[pr] = l;
        }
        tc_fence_before();
      } else if (lane == 0) {
        record_error(p.err, PA_DEVERR_TIMEOUT);
      }
    }
  }

  if (warp == 0 && lane == 0) mbar_wait(bar(B_MMADONE), 0);  // the issuers' tcgen05 ops done (bounded)
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kTmem);
  }
}

// One warp per row: the partitions its row tile has keys of, in order.
// blockIdx.y: request; 8 rows per CTA.
template <int D, typename T>
__global__ void __launch_bounds__(256) kv4_prefill_merge_kernel(const Kv4PrefillParams p) {
  constexpr int V = D / 32;
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.y, lane = threadIdx.x & 31;
  const int qs = __ldg(p.q_start + r), qe = __ldg(p.q_start + r + 1), ctx = __ldg(p.lens + r);
  const int chunk = qe - qs, p0 = ctx - chunk, G = p.group;
  if (qs < 0 || qe < qs || qe > p.total_q || chunk > p.max_q_len || ctx < chunk || ctx > p.maxblk * p.block_size) return;
  const int64_t at = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);  // (query, head)
  if (at >= (int64_t)chunk * p.q_heads) return;
  const int qi = (int)(at / p.q_heads), head = (int)(at - (int64_t)qi * p.q_heads);
  const int rows = chunk * G, grow = qi * G + head % G;
  const int last_row = min((grow / (2 * kRows) + 1) * 2 * kRows, rows) - 1;  // of the row's tiles
  const int nsplit = partitions_of(p0 + last_row / G + 1, p.split_tokens);
  const size_t orow = (size_t)(qs + qi) * p.q_heads + head;
  const float* pm = p.part_m + orow * p.max_splits;
  const float* pl = p.part_l + orow * p.max_splits;
  const float* po = p.part_o + orow * p.max_splits * D + lane * V;
  float M = -INFINITY;
  for (int c = lane; c < nsplit; c += 32) M = fmaxf(M, pm[c]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  if (M == -INFINITY) M = 0.f;  // no finite score: sums are zero or not numbers
  float a[V], den = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = 0.f;
#pragma unroll 4
  for (int c = 0; c < nsplit; ++c) {
    const float f = exp2f(pm[c] - M);
    den += f * pl[c];
    const float* x = po + (size_t)c * D;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(x + i);
      a[i] += f * v.x;
      a[i + 1] += f * v.y;
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  T* o = static_cast<T*>(p.out) + orow * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(o + i) = Elem<T>::pack(a[i] * inv, a[i + 1] * inv);
}

template <int D, typename T>
cudaError_t launch_t(const Kv4PrefillParams& p, cudaStream_t stream) {
  using L = Kv4PrefillSmem<D>;
  auto kern = kv4_prefill_kernel<D, T>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 64 && !attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t units = (int64_t)p.row_tiles * p.kv_heads * p.num_reqs * p.max_splits;
  if (units > INT32_MAX) return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(kern, dim3((unsigned)units), dim3(kThreads), L::BYTES, stream, p);
  if (e != cudaSuccess || p.max_splits == 1) return e;
  const unsigned gx = (unsigned)(((int64_t)p.max_q_len * p.q_heads + 7) / 8);
  return launch_pdl(kv4_prefill_merge_kernel<D, T>, dim3(gx, p.num_reqs), dim3(256), 0, stream, p);
}

}  // namespace

cudaError_t launch_kv4_prefill(const Kv4PrefillParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  if (head_dim == 128) return dt == PA_BF16 ? launch_t<128, __nv_bfloat16>(p, stream) : launch_t<128, __half>(p, stream);
  return dt == PA_BF16 ? launch_t<64, __nv_bfloat16>(p, stream) : launch_t<64, __half>(p, stream);
}

}  // namespace pa
