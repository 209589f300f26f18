// Writing a 4-bit paged cache and reading it back (see kv4.cuh for the page).
//
// One thread takes the 16 elements of a scale, of K and of V: their largest
// magnitude, the scale and the codes need no other thread, and neighbouring
// threads read and write neighbouring 32-byte pieces.  Both kernels are bound by
// memory: the write reads 2 bytes an element and writes 9/16.
#include "kv4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// 16 elements (two vectors) as floats.
template <typename T>
__device__ __forceinline__ void to_floats(const uint4 (&v)[2], float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = Elem<T>::lo(w[j]);
      x[8 * i + 2 * j + 1] = Elem<T>::hi(w[j]);
    }
  }
}

// Scale byte and codes of one group.
//
// The quotient x / s is taken as x * (1 / s) and one Newton step on its
// remainder: exact wherever x / s is representable, which is what decides a
// tie between two levels (x has at most 11 significant bits and s four, so
// every other quotient is at least 2^-12 of itself away from one).
__device__ __forceinline__ uint2 encode16(const float (&x)[16], uint32_t& byte) {
  float top = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    top = fmaxf(top, fabsf(x[i]));
    nan |= x[i] != x[i];
  }
  byte = nan ? kKv4NanScale : kv4_scale_byte(top);
  if (byte == 0 || byte == kKv4NanScale) return make_uint2(0u, 0u);
  const float s = kv4_scale(byte), r = __frcp_rn(s);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float y[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float q = x[i + e] * r;
      // a quotient that overflowed is far above the largest level: no step from it
      y[e] = fabsf(q) < 64.f ? fmaf(fmaf(-q, s, x[i + e]), r, q) : q;
    }
    w[i >> 3] |= kv4_pack2(y[0], y[1]) << ((i & 7) * 4);
  }
  return make_uint2(w[0], w[1]);
}

// Group i: its token, its place in the token's row of all heads, and where its
// codes and its scale are in either cache.
struct Place {
  uint32_t token, at;
  int32_t slot;
  int64_t codes, scale;
};
template <int D>
__device__ __forceinline__ Place place_of(uint32_t i, const int32_t* slots, uint32_t per_token, int64_t num_slots,
                                          int kv_heads, int block_shift) {
  constexpr uint32_t GROUPS = D / kKv4Group;
  Place w;
  w.token = i / per_token;
  w.at = i - w.token * per_token;
  w.slot = __ldg(slots + w.token);
  const uint32_t h = w.at / GROUPS, g = w.at % GROUPS;
  const uint32_t b = (uint32_t)w.slot >> block_shift, o = (uint32_t)w.slot & ((1u << block_shift) - 1u);
  const int64_t page = ((int64_t)b * kv_heads + h) * ((int64_t)Kv4Row<D>::BYTES << block_shift);
  w.codes = page + o * Kv4Row<D>::CODES + 8 * g;
  w.scale = page + (Kv4Row<D>::CODES << block_shift) + o * GROUPS + g;
  return w;
}

template <int D, typename T>
__global__ void __launch_bounds__(256) quantize_and_cache_kernel(const Kv4WriteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t per_token = p.kv_heads * (D / kKv4Group), total = (uint32_t)p.num_tokens * per_token;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const Place w = place_of<D>(i, p.slots, per_token, p.num_slots, p.kv_heads, p.block_shift);
  if (w.slot < 0) return;  // padding token
  if (w.slot >= p.num_slots) {
    if (w.at == 0) record_error(p.err, PA_DEVERR_SLOT);
    return;
  }
  const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + w.token * p.k_stride + w.at * kKv4Group);
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + w.token * p.v_stride + w.at * kKv4Group);
  const uint4 xk[2] = {__ldg(k), __ldg(k + 1)}, xv[2] = {__ldg(v), __ldg(v + 1)};
  float x[16];
  uint32_t byte;
  to_floats<T>(xk, x);
  uint2 codes = encode16(x, byte);
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k_cache) + w.codes) = codes;
  static_cast<uint8_t*>(p.k_cache)[w.scale] = (uint8_t)byte;
  to_floats<T>(xv, x);
  codes = encode16(x, byte);
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_cache) + w.codes) = codes;
  static_cast<uint8_t*>(p.v_cache)[w.scale] = (uint8_t)byte;
}

template <int D, typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const Kv4ReadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t per_token = p.kv_heads * (D / kKv4Group), total = (uint32_t)p.num_tokens * per_token;
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const Place w = place_of<D>(i, p.slots, per_token, p.num_slots, p.kv_heads, p.block_shift);
  const bool has = w.slot >= 0 && w.slot < p.num_slots;
  if (w.slot >= p.num_slots && w.at == 0) record_error(p.err, PA_DEVERR_SLOT);
  uint2 codes[2] = {make_uint2(0, 0), make_uint2(0, 0)};
  uint32_t byte[2] = {0, 0};
  if (has) {
    codes[0] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.k_cache) + w.codes);
    codes[1] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.v_cache) + w.codes);
    byte[0] = static_cast<const uint8_t*>(p.k_cache)[w.scale];
    byte[1] = static_cast<const uint8_t*>(p.v_cache)[w.scale];
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const uint32_t s = kv4_scale2(byte[e]);
    uint32_t r[8];
    kv4_unpack(codes[e].x, *reinterpret_cast<uint32_t(*)[4]>(&r[0]));
    kv4_unpack(codes[e].y, *reinterpret_cast<uint32_t(*)[4]>(&r[4]));
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = from_half2<T>(hmul2_u(r[k], s));
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(e ? p.v : p.k) + (int64_t)i * kKv4Group);
    dst[0] = make_uint4(r[0], r[1], r[2], r[3]);
    dst[1] = make_uint4(r[4], r[5], r[6], r[7]);
  }
}

// Tokens of a launch: groups are counted in 32 bits.
int64_t tokens_at_once(int kv_heads, int head_dim) { return INT32_MAX / (kv_heads * (head_dim / kKv4Group)); }

}  // namespace

cudaError_t launch_quantize_and_cache(const Kv4WriteParams& all, int head_dim, pa_dtype dt, cudaStream_t stream) {
  const int64_t most = tokens_at_once(all.kv_heads, head_dim);
  cudaError_t e = cudaSuccess;
  for (int64_t t = 0; t < all.num_tokens && e == cudaSuccess; t += most) {
    Kv4WriteParams p = all;
    p.num_tokens = all.num_tokens - t < most ? all.num_tokens - t : most;
    p.k = static_cast<const uint16_t*>(all.k) + t * all.k_stride;
    p.v = static_cast<const uint16_t*>(all.v) + t * all.v_stride;
    p.slots = all.slots + t;
    const dim3 grid((unsigned)((p.num_tokens * p.kv_heads * (head_dim / kKv4Group) + 255) / 256)), block(256);
    if (head_dim == 128)
      e = dt == PA_BF16 ? launch_pdl(quantize_and_cache_kernel<128, __nv_bfloat16>, grid, block, 0, stream, p)
                        : launch_pdl(quantize_and_cache_kernel<128, __half>, grid, block, 0, stream, p);
    else
      e = dt == PA_BF16 ? launch_pdl(quantize_and_cache_kernel<64, __nv_bfloat16>, grid, block, 0, stream, p)
                        : launch_pdl(quantize_and_cache_kernel<64, __half>, grid, block, 0, stream, p);
  }
  return e;
}

cudaError_t launch_dequantize_kv4(const Kv4ReadParams& all, int head_dim, pa_dtype dt, cudaStream_t stream) {
  const int64_t most = tokens_at_once(all.kv_heads, head_dim), row = (int64_t)all.kv_heads * head_dim;
  cudaError_t e = cudaSuccess;
  for (int64_t t = 0; t < all.num_tokens && e == cudaSuccess; t += most) {
    Kv4ReadParams p = all;
    p.num_tokens = all.num_tokens - t < most ? all.num_tokens - t : most;
    p.k = static_cast<uint16_t*>(all.k) + t * row;
    p.v = static_cast<uint16_t*>(all.v) + t * row;
    p.slots = all.slots + t;
    const dim3 grid((unsigned)((p.num_tokens * p.kv_heads * (head_dim / kKv4Group) + 255) / 256)), block(256);
    if (head_dim == 128)
      e = dt == PA_BF16 ? launch_pdl(dequantize_kernel<128, __nv_bfloat16>, grid, block, 0, stream, p)
                        : launch_pdl(dequantize_kernel<128, __half>, grid, block, 0, stream, p);
    else
      e = dt == PA_BF16 ? launch_pdl(dequantize_kernel<64, __nv_bfloat16>, grid, block, 0, stream, p)
                        : launch_pdl(dequantize_kernel<64, __half>, grid, block, 0, stream, p);
  }
  return e;
}

}  // namespace pa
