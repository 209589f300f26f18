// Writing a 4-bit paged cache and reading it back (see kv4.cuh for the page).
//
// One thread takes the 16 elements of one scale: its largest magnitude, the
// scale, and the codes need no other thread, and neighbouring threads read and
// write neighbouring 32-byte pieces.  Both kernels are bound by memory: the
// write reads 2 bytes an element and writes 9/16.
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

template <int D, typename T>
__global__ void __launch_bounds__(256) quantize_and_cache_kernel(const Kv4WriteParams p) {
  constexpr int GROUPS = D / kKv4Group;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t per_token = (int64_t)p.kv_heads * GROUPS;
  const int64_t total = 2 * p.num_tokens * per_token;
  const int64_t page = (int64_t)p.block_size * Kv4Row<D>::BYTES;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / per_token;  // K of token 0, V of token 0, K of token 1, ...
    const int at = (int)(i - row * per_token);
    const int64_t tok = row >> 1;
    const bool isv = row & 1;
    const int32_t slot = __ldg(p.slots + tok);
    if (slot < 0) continue;  // padding token
    if (slot >= p.num_slots) {
      if (at == 0) record_error(p.err, PA_DEVERR_SLOT);
      continue;
    }
    const T* src = static_cast<const T*>(isv ? p.v : p.k) + tok * (isv ? p.v_stride : p.k_stride) + at * kKv4Group;
    const uint4 v[2] = {__ldg(reinterpret_cast<const uint4*>(src)), __ldg(reinterpret_cast<const uint4*>(src) + 1)};
    float x[16];
    to_floats<T>(v, x);
    uint32_t byte;
    const uint2 codes = encode16(x, byte);
    const int h = at / GROUPS, g = at - h * GROUPS;
    const int b = slot / p.block_size, o = slot - b * p.block_size;
    uint8_t* dst = static_cast<uint8_t*>(isv ? p.v_cache : p.k_cache) + ((int64_t)b * p.kv_heads + h) * page;
    *reinterpret_cast<uint2*>(dst + o * Kv4Row<D>::CODES + 8 * g) = codes;
    dst[p.block_size * Kv4Row<D>::CODES + o * GROUPS + g] = (uint8_t)byte;
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(256) dequantize_kernel(const Kv4ReadParams p) {
  constexpr int GROUPS = D / kKv4Group;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t per_token = (int64_t)p.kv_heads * GROUPS;
  const int64_t total = 2 * p.num_tokens * per_token;
  const int64_t page = (int64_t)p.block_size * Kv4Row<D>::BYTES;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / per_token;
    const int at = (int)(i - row * per_token);
    const int64_t tok = row >> 1;
    const bool isv = row & 1;
    const int32_t slot = __ldg(p.slots + tok);
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot >= p.num_slots) {
      if (at == 0) record_error(p.err, PA_DEVERR_SLOT);
    } else if (slot >= 0) {
      const int h = at / GROUPS, g = at - h * GROUPS;
      const int b = slot / p.block_size, o = slot - b * p.block_size;
      const uint8_t* src = static_cast<const uint8_t*>(isv ? p.v_cache : p.k_cache) + ((int64_t)b * p.kv_heads + h) * page;
      const uint2 codes = *reinterpret_cast<const uint2*>(src + o * Kv4Row<D>::CODES + 8 * g);
      const uint32_t s = kv4_scale2(src[p.block_size * Kv4Row<D>::CODES + o * GROUPS + g]);
      uint32_t r[8];
      kv4_unpack(codes.x, *reinterpret_cast<uint32_t(*)[4]>(&r[0]));
      kv4_unpack(codes.y, *reinterpret_cast<uint32_t(*)[4]>(&r[4]));
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = from_half2<T>(hmul2_u(r[e], s));
      out[0] = make_uint4(r[0], r[1], r[2], r[3]);
      out[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(isv ? p.v : p.k) + (tok * per_token + at) * kKv4Group);
    dst[0] = out[0];
    dst[1] = out[1];
  }
}

}  // namespace

cudaError_t launch_quantize_and_cache(const Kv4WriteParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  const int64_t total = 2 * p.num_tokens * p.kv_heads * (head_dim / kKv4Group);
  if (total == 0) return cudaSuccess;
  const dim3 grid(copy_grid(total)), block(256);
  if (head_dim == 128)
    return dt == PA_BF16 ? launch_pdl(quantize_and_cache_kernel<128, __nv_bfloat16>, grid, block, 0, stream, p)
                         : launch_pdl(quantize_and_cache_kernel<128, __half>, grid, block, 0, stream, p);
  return dt == PA_BF16 ? launch_pdl(quantize_and_cache_kernel<64, __nv_bfloat16>, grid, block, 0, stream, p)
                       : launch_pdl(quantize_and_cache_kernel<64, __half>, grid, block, 0, stream, p);
}

cudaError_t launch_dequantize_kv4(const Kv4ReadParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  const int64_t total = 2 * p.num_tokens * p.kv_heads * (head_dim / kKv4Group);
  if (total == 0) return cudaSuccess;
  const dim3 grid(copy_grid(total)), block(256);
  if (head_dim == 128)
    return dt == PA_BF16 ? launch_pdl(dequantize_kernel<128, __nv_bfloat16>, grid, block, 0, stream, p)
                         : launch_pdl(dequantize_kernel<128, __half>, grid, block, 0, stream, p);
  return dt == PA_BF16 ? launch_pdl(dequantize_kernel<64, __nv_bfloat16>, grid, block, 0, stream, p)
                       : launch_pdl(dequantize_kernel<64, __half>, grid, block, 0, stream, p);
}

}  // namespace pa
