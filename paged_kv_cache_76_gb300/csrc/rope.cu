// Norm, rotation and cache write of new tokens in one pass, for sm_103a.
//
// Per head row x of D elements: x <- x * rsqrt(mean(x^2) + eps) * w (optional),
// then the first rot_dim elements are rotated pair by pair, (a, b) ->
// (a c - b s, b c + a s), with c, s read from a table at the token's position
// (of up to three axes); queries go to q_out, keys and values to their cache
// slots.  Everything between the one load and the one store is fp32.
//
// Bound by HBM: 2 bytes read and 2 written per element, about 7 operations.
// D/8 threads hold a head row, 8 consecutive elements each (one 16-byte
// vector): a warp reads whole 128-byte lines, the norm's sum is a shuffle
// reduction over the row's threads, and the partner of a half-split pair is 8
// elements that one other thread of the row holds (one shuffle per 32-bit
// register).  A thread keeps its 8 cosines and sines over all heads of its
// token, so the table costs rot_dim * 4 bytes per token and CTA, not per head.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

template <typename T> __device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = Elem<T>::lo(u[i]);
    x[2 * i + 1] = Elem<T>::hi(u[i]);
  }
}
template <typename T> __device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Elem<T>::pack(x[0], x[1]), Elem<T>::pack(x[2], x[3]), Elem<T>::pack(x[4], x[5]),
                    Elem<T>::pack(x[6], x[7]));
}

// Heads of a token in the order queries, keys, values; a CTA takes one token
// and the heads group, group + ROWS, ... of its share (blockIdx.y of
// gridDim.y shares).
template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPH = D / 8;                 // threads per head row
  constexpr int ROWS = kRopeThreads / LPH;   // head rows in flight
  const int sub = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const int half = p.rot_dim / 2;
  const int e0 = sub * 8;  // this thread's first element
  const bool rotated = e0 < p.rot_dim;
  const int heads = p.q_heads + 2 * p.kv_heads;
  // the thread of the same row that holds the partners (half-split pairs)
  const int mate = (threadIdx.x & 31) + (e0 < half ? half / 8 : rotated ? -(half / 8) : 0);

  // the whole kernel after the one before it: its inputs may come from there,
  // and q_out may still be read there.  No early launch of the next kernel,
  // which may read q_out in its set-up.
  griddep_wait();

  for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    const int slot = __ldg(p.slots + t);
    int pos[3];
    bool bad_pos = false;
#pragma unroll
    for (int a = 0; a < 3; ++a) {
      pos[a] = a < p.num_axes ? __ldg(p.positions + (size_t)a * p.num_tokens + t) : 0;
      bad_pos |= pos[a] < 0 || pos[a] >= p.max_position;
    }
    if (bad_pos) {  // CTA-uniform
      if (slot >= 0 && threadIdx.x == 0) record_error(p.err, PA_DEVERR_POSITION);
      continue;
    }
    const bool write_kv = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0) record_error(p.err, PA_DEVERR_SLOT);

    // y_i = x_i * c_i + partner_i * s_i
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (rotated) {
        const int e = e0 + i;
        const int j = p.interleaved ? e >> 1 : (e < half ? e : e - half);
        const int ax = j < p.sec_end[0] ? 0 : (j < p.sec_end[1] ? 1 : 2);
        const float* row = p.cos_sin + (size_t)(ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2]) * p.rot_dim;
        const bool first = p.interleaved ? (e & 1) == 0 : e < half;
        c[i] = __ldg(row + j);
        s[i] = first ? -__ldg(row + half + j) : __ldg(row + half + j);
      }
    }

    for (int h0 = blockIdx.y * ROWS; h0 < heads; h0 += gridDim.y * ROWS) {
      const int hh = h0 + group;
      const bool is_q = hh < p.q_heads, is_k = !is_q && hh < p.q_heads + p.kv_heads;
      const bool is_v = !is_q && !is_k && hh < heads;
      const int h = is_q ? hh : is_k ? hh - p.q_heads : hh - p.q_heads - p.kv_heads;
      const bool live = hh < heads && (is_q || write_kv);
      const T* src = reinterpret_cast<const T*>(is_q ? p.q : is_k ? p.k : p.v) +
                     (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) * (int64_t)t + (int64_t)h * D + e0;
      const uint4 raw = live ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
      T* dst = is_q ? reinterpret_cast<T*>(p.q_out) + ((size_t)t * p.q_heads + h) * D + e0
                    : reinterpret_cast<T*>(is_k ? p.k_cache : p.v_cache) + ((size_t)slot * p.kv_heads + h) * D + e0;
      // partner elements (before the norm: the factor is the row's, the weight the partner's)
      uint4 other;
      other.x = __shfl_sync(kAll, raw.x, mate);
      other.y = __shfl_sync(kAll, raw.y, mate);
      other.z = __shfl_sync(kAll, raw.z, mate);
      other.w = __shfl_sync(kAll, raw.w, mate);
      float x[8], y[8];
      unpack8<T>(raw, x);
      unpack8<T>(other, y);
      const T* w = reinterpret_cast<const T*>(is_q ? p.q_weight : is_k ? p.k_weight : nullptr);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      if (w) {
        const float f = rsqrtf(sum * (1.f / D) + p.eps);
        float wx[8], wy[8];
        unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w + e0)), wx);
        const int ey = p.interleaved || !rotated ? e0 : e0 < half ? e0 + half : e0 - half;
        unpack8<T>(__ldg(reinterpret_cast<const uint4*>(w + ey)), wy);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= f * wx[i];
          y[i] *= f * wy[i];
        }
      }
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = x[i] * c[i] + (p.interleaved ? x[i ^ 1] : y[i]) * s[i];
      if (live) *reinterpret_cast<uint4*>(dst) = is_v ? raw : pack8<T>(z);
    }
  }
}

template <int D, typename T>
cudaError_t launch_t(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int ROWS = kRopeThreads / (D / 8);
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int shares = (heads + ROWS - 1) / ROWS;
  // few tokens: a CTA per share of the heads, so that the loads of a token
  // are all in flight at once
  const int sms = num_sms() > 0 ? num_sms() : 1;
  const int gy = (int64_t)p.num_tokens * shares <= 4 * (int64_t)sms ? shares : 1;
  const int64_t cap = 8 * (int64_t)sms;  // 8 CTAs of 256 threads per SM
  const unsigned gx = (unsigned)(p.num_tokens < cap ? p.num_tokens : cap);
  return launch_pdl(norm_rope_kernel<D, T>, dim3(gx, gy), dim3(kRopeThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (head_dim == 128) return dt == PA_BF16 ? launch_t<128, __nv_bfloat16>(p, stream) : launch_t<128, __half>(p, stream);
  if (head_dim == 64) return dt == PA_BF16 ? launch_t<64, __nv_bfloat16>(p, stream) : launch_t<64, __half>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
