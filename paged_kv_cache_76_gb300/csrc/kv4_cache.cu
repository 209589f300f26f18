// Writing a 4-bit paged cache and reading it back (see kv4.cuh for the page).
//
// One thread takes the 16 elements of a scale, of K and of V: their largest
// magnitude, the scale and the codes need no other thread, and neighbouring
// threads read and write neighbouring 32-byte pieces.  Both kernels are bound by
// memory.  Measured on GB300: 8192 tokens (8 heads of 128, views of a fused
// projection's rows) written to scattered slots 8.9 us (43 MB: 4.8 TB/s), a pool
// of 10304 read back 8.1 (54 MB: 6.6 TB/s); 64 tokens 1.5.
#include "kv4.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

// Threads of a CTA (64: 9.3 us and 10.8 for the sizes above; 256: 9.35 and 8.3); of
// those that write an SM holds twelve (eleven, in 44 registers: 9.0).
constexpr int kThreads = 128;

// 32 bytes at once, where they are aligned: two accesses of 16 each take half of
// every sector (the read below 12.5 us instead of 8.3; the write the same either way).
__device__ __forceinline__ void ld_32(const void* p, uint4 (&v)[2]) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                 "=r"(v[1].w)
               : "l"(p));
}
__device__ __forceinline__ void st_32(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
               "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

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

// Largest magnitude of a group: positive 16-bit floats order as their bits do,
// infinities and NaN last, so it is a maximum of pairs of integers.
template <typename T>
__device__ __forceinline__ float largest(const uint4 (&v)[2]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m = __vmaxu2(m, __vmaxu2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu));
    m = __vmaxu2(m, __vmaxu2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
  }
  m = __vmaxu2(m, m >> 16);
  return Elem<T>::lo(m & 0xFFFFu);
}

// Scale byte and codes of one group.
//
// The quotient x / s is taken as x * (1 / s) and one Newton step on its
// remainder: exact wherever x / s is representable, which is what decides a
// tie between two levels (x has at most 11 significant bits and s four, so
// every other quotient is at least 2^-12 of itself away from one).  Quotients
// beyond 6 become the level 6, the nearest, by the conversion's saturation: up to
// 6.4 where s is rounded down at three bits, below 9 for the smallest scales
// (2^-17 apart, so the first stands for up to 1.5 times itself), any that fp32
// holds above the largest.
template <typename T>
__device__ __forceinline__ uint2 encode16(const uint4 (&v)[2], uint32_t& byte) {
  byte = kv4_scale_byte(largest<T>(v));
  if (byte == 0 || byte == kKv4NanScale) return make_uint2(0u, 0u);
  float x[16];
  to_floats<T>(v, x);
  const float s = kv4_scale(byte), r = __frcp_rn(s);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float q0, q1, y0, y1;
    fmul2(q0, q1, x[i], x[i + 1], r, r);
    ffma2(y0, y1, q0, q1, -s, -s, x[i], x[i + 1]);
    ffma2(y0, y1, y0, y1, r, r, q0, q1);
    w[i >> 3] |= kv4_pack2(y0, y1) << ((i & 7) * 4);
  }
  return make_uint2(w[0], w[1]);
}

// Where group `at` of a token's row of all heads has its codes and its scale in a cache.
struct Place {
  int64_t codes, scale;
};
template <int D>
__device__ __forceinline__ Place place_of(uint32_t at, int32_t slot, int kv_heads, int block_shift) {
  constexpr uint32_t GROUPS = D / kKv4Group;
  const uint32_t h = at / GROUPS, g = at % GROUPS;
  const uint32_t b = (uint32_t)slot >> block_shift, o = (uint32_t)slot & ((1u << block_shift) - 1u);
  const int64_t page = ((int64_t)b * kv_heads + h) * ((int64_t)Kv4Row<D>::BYTES << block_shift);
  return Place{page + o * Kv4Row<D>::CODES + 8 * g, page + (Kv4Row<D>::CODES << block_shift) + o * GROUPS + g};
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 12) quantize_and_cache_kernel(const Kv4WriteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t per_token = p.kv_heads * (D / kKv4Group), total = (uint32_t)p.num_tokens * per_token;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const uint32_t token = i / per_token, at = i - token * per_token;
  // k and v do not wait for the slot
  const uint4* k = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k) + token * p.k_stride + at * kKv4Group);
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + token * p.v_stride + at * kKv4Group);
  const int32_t slot = __ldg(p.slots + token);
  uint4 xk[2], xv[2];
  if (p.wide) {
    ld_32(k, xk);
    ld_32(v, xv);
  } else {
    xk[0] = __ldg(k), xk[1] = __ldg(k + 1);
    xv[0] = __ldg(v), xv[1] = __ldg(v + 1);
  }
  if (slot < 0) return;  // padding token
  if (slot >= p.num_slots) {
    if (at == 0) record_error(p.err, PA_DEVERR_SLOT);
    return;
  }
  const Place w = place_of<D>(at, slot, p.kv_heads, p.block_shift);
  uint32_t byte;
  uint2 codes = encode16<T>(xk, byte);
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.k_cache) + w.codes) = codes;
  static_cast<uint8_t*>(p.k_cache)[w.scale] = (uint8_t)byte;
  codes = encode16<T>(xv, byte);
  *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_cache) + w.codes) = codes;
  static_cast<uint8_t*>(p.v_cache)[w.scale] = (uint8_t)byte;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const Kv4ReadParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t per_token = p.kv_heads * (D / kKv4Group), total = (uint32_t)p.num_tokens * per_token;
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const uint32_t token = i / per_token, at = i - token * per_token;
  const int32_t slot = __ldg(p.slots + token);
  const bool has = slot >= 0 && slot < p.num_slots;
  if (slot >= p.num_slots && at == 0) record_error(p.err, PA_DEVERR_SLOT);
  const Place w = place_of<D>(at, has ? slot : 0, p.kv_heads, p.block_shift);
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
    T* dst = static_cast<T*>(e ? p.v : p.k) + (int64_t)i * kKv4Group;
    if (p.wide) {
      st_32(dst, r);
    } else {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
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
    p.wide = ((reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 31u) == 0 &&
             p.k_stride % 16 == 0 && p.v_stride % 16 == 0;
    const dim3 grid((unsigned)((p.num_tokens * p.kv_heads * (head_dim / kKv4Group) + kThreads - 1) / kThreads)),
        block(kThreads);
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
    p.wide = ((reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.v)) & 31u) == 0;
    const dim3 grid((unsigned)((p.num_tokens * p.kv_heads * (head_dim / kKv4Group) + kThreads - 1) / kThreads)),
        block(kThreads);
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
