// Norm, rotation and cache write of new tokens in one pass, for sm_103a.
//
// Per head row x of D elements: x <- x * rsqrt(mean(x^2) + eps) * w (optional),
// then the first rot_dim elements are rotated pair by pair, (a, b) ->
// (a c - b s, b c + a s), with c, s read from a table at the token's position
// (of up to three axes); queries go to q_out, keys and values to their cache
// slots.  Everything between the one load and the one store is fp32.
//
// Bound by HBM: 2 bytes read and 2 written per element.  D/8 threads hold a
// head row, and each thread holds four whole pairs of it (elements 4s.. and
// rot_dim/2 + 4s.., two 8-byte vectors; eight neighbours if interleaved), so a
// rotation needs no other thread, the norm's sum is the only shuffle, and the
// thread keeps its four cosines and sines over all heads of its token.  The
// rows of a token that a thread takes are loaded together, before any is used,
// and a CTA's next token while it works on this one's.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr unsigned kAll = 0xffffffffu;

// Heads of a token in the order queries, keys, values; a CTA takes a token and
// the rows group + ROWS * (share, share + shares, ...) of it, kRopeRows of them
// at a time.
constexpr int kRopeRows = 4;

template <int D, typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPH = D / 8;                // threads per head row
  constexpr int ROWS = kRopeThreads / LPH;  // head rows in flight
  const int sub = threadIdx.x % LPH, group = threadIdx.x / LPH;
  const int half = p.rot_dim / 2;
  const bool rotated = sub < p.rot_dim / 8;
  // this thread's two runs of four elements; behind rot_dim, eight neighbours
  const int lo = INTER || !rotated ? 8 * sub : 4 * sub;
  const int hi = INTER || !rotated ? 8 * sub + 4 : half + 4 * sub;
  const int heads = p.q_heads + 2 * p.kv_heads;
  const int share0 = blockIdx.y * ROWS + group, step = gridDim.y * ROWS;

  // the whole kernel after the one before it: its inputs may come from there,
  // and q_out may still be read there.  No early launch of the next kernel,
  // which may read q_out in its set-up.
  griddep_wait();

  // token t's slot and positions
  auto place = [&](int t, int& slot, int (&pos)[3]) {
    slot = __ldg(p.slots + t);
#pragma unroll
    for (int a = 0; a < 3; ++a) pos[a] = a < p.num_axes ? __ldg(p.positions + (size_t)a * p.num_tokens + t) : 0;
  };
  int slot_next, pos_next[3];
  if (blockIdx.x < p.num_tokens) place(blockIdx.x, slot_next, pos_next);

  for (int t = blockIdx.x; t < p.num_tokens; t += gridDim.x) {
    const int slot = slot_next;
    const int pos[3] = {pos_next[0], pos_next[1], pos_next[2]};
    if (t + (int)gridDim.x < p.num_tokens) place(t + gridDim.x, slot_next, pos_next);
    bool bad_pos = false;
#pragma unroll
    for (int a = 0; a < 3; ++a) bad_pos |= pos[a] < 0 || pos[a] >= p.max_position;
    if (bad_pos) {  // CTA-uniform
      if (slot >= 0 && threadIdx.x == 0) record_error(p.err, PA_DEVERR_POSITION);
      continue;
    }
    const bool write_kv = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0) record_error(p.err, PA_DEVERR_SLOT);

    float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (rotated) {
      const int j = 4 * sub;  // this thread's pairs
      auto axis = [&](int jj) { return jj < p.sec_end[0] ? pos[0] : jj < p.sec_end[1] ? pos[1] : pos[2]; };
      const bool one = (j >= p.sec_end[0] || j + 3 < p.sec_end[0]) && (j >= p.sec_end[1] || j + 3 < p.sec_end[1]);
      if (one) {  // all four turn by one axis
        const float* row = p.cos_sin + (size_t)axis(j) * p.rot_dim + j;
        const float4 cv = __ldg(reinterpret_cast<const float4*>(row));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half));
        c[0] = cv.x, c[1] = cv.y, c[2] = cv.z, c[3] = cv.w;
        s[0] = sv.x, s[1] = sv.y, s[2] = sv.z, s[3] = sv.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* row = p.cos_sin + (size_t)axis(j + i) * p.rot_dim + j + i;
          c[i] = __ldg(row);
          s[i] = __ldg(row + half);
        }
      }
    }

    for (int h0 = share0; h0 - group < heads; h0 += step * kRopeRows) {
      uint2 x[kRopeRows], y[kRopeRows];
#pragma unroll
      for (int u = 0; u < kRopeRows; ++u) {
        const int hh = h0 + u * step;
        x[u] = y[u] = make_uint2(0u, 0u);
        if (hh < p.q_heads || (hh < heads && write_kv)) {
          const bool is_q = hh < p.q_heads, is_k = hh < p.q_heads + p.kv_heads;
          const int h = is_q ? hh : is_k ? hh - p.q_heads : hh - p.q_heads - p.kv_heads;
          const T* src = reinterpret_cast<const T*>(is_q ? p.q : is_k ? p.k : p.v) +
                         (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) * (int64_t)t + (int64_t)h * D;
          x[u] = __ldg(reinterpret_cast<const uint2*>(src + lo));
          y[u] = __ldg(reinterpret_cast<const uint2*>(src + hi));
        }
      }
#pragma unroll
      for (int u = 0; u < kRopeRows; ++u) {
        const int hh = h0 + u * step;
        if (hh - group >= heads) break;  // CTA-uniform
        const bool is_q = hh < p.q_heads, is_k = !is_q && hh < p.q_heads + p.kv_heads;
        const int h = is_q ? hh : is_k ? hh - p.q_heads : hh - p.q_heads - p.kv_heads;
        // pair i: (a[i], b[i])
        float a[4], b[4];
        if constexpr (INTER) {
          a[0] = Elem<T>::lo(x[u].x), b[0] = Elem<T>::hi(x[u].x), a[1] = Elem<T>::lo(x[u].y), b[1] = Elem<T>::hi(x[u].y);
          a[2] = Elem<T>::lo(y[u].x), b[2] = Elem<T>::hi(y[u].x), a[3] = Elem<T>::lo(y[u].y), b[3] = Elem<T>::hi(y[u].y);
        } else {
          a[0] = Elem<T>::lo(x[u].x), a[1] = Elem<T>::hi(x[u].x), a[2] = Elem<T>::lo(x[u].y), a[3] = Elem<T>::hi(x[u].y);
          b[0] = Elem<T>::lo(y[u].x), b[1] = Elem<T>::hi(y[u].x), b[2] = Elem<T>::lo(y[u].y), b[3] = Elem<T>::hi(y[u].y);
        }
        if (p.q_weight || p.k_weight) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += a[i] * a[i] + b[i] * b[i];
#pragma unroll
          for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
          const T* w = reinterpret_cast<const T*>(is_q ? p.q_weight : is_k ? p.k_weight : nullptr);
          if (w) {
            const float f = rsqrtf(sum * (1.f / D) + p.eps);
            const uint2 wx = __ldg(reinterpret_cast<const uint2*>(w + lo)), wy = __ldg(reinterpret_cast<const uint2*>(w + hi));
            const float wl[4] = {Elem<T>::lo(wx.x), Elem<T>::hi(wx.x), Elem<T>::lo(wx.y), Elem<T>::hi(wx.y)};
            const float wh[4] = {Elem<T>::lo(wy.x), Elem<T>::hi(wy.x), Elem<T>::lo(wy.y), Elem<T>::hi(wy.y)};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] *= f * (INTER ? (i < 2 ? wl[2 * i] : wh[2 * i - 4]) : wl[i]);
              b[i] *= f * (INTER ? (i < 2 ? wl[2 * i + 1] : wh[2 * i - 3]) : wh[i]);
            }
          }
        }
        uint2 xo = x[u], yo = y[u];  // values: as they are
        if (is_q || is_k) {
          float za[4], zb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            za[i] = a[i] * c[i] - b[i] * s[i];
            zb[i] = b[i] * c[i] + a[i] * s[i];
          }
          if constexpr (INTER) {
            xo = make_uint2(Elem<T>::pack(za[0], zb[0]), Elem<T>::pack(za[1], zb[1]));
            yo = make_uint2(Elem<T>::pack(za[2], zb[2]), Elem<T>::pack(za[3], zb[3]));
          } else {
            xo = make_uint2(Elem<T>::pack(za[0], za[1]), Elem<T>::pack(za[2], za[3]));
            yo = make_uint2(Elem<T>::pack(zb[0], zb[1]), Elem<T>::pack(zb[2], zb[3]));
          }
        }
        if (is_q || (hh < heads && write_kv)) {
          T* dst = is_q ? reinterpret_cast<T*>(p.q_out) + ((size_t)t * p.q_heads + h) * D
                        : reinterpret_cast<T*>(is_k ? p.k_cache : p.v_cache) + ((size_t)slot * p.kv_heads + h) * D;
          *reinterpret_cast<uint2*>(dst + lo) = xo;
          *reinterpret_cast<uint2*>(dst + hi) = yo;
        }
      }
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
  return p.interleaved ? launch_pdl(norm_rope_kernel<D, T, true>, dim3(gx, gy), dim3(kRopeThreads), 0, stream, p)
                       : launch_pdl(norm_rope_kernel<D, T, false>, dim3(gx, gy), dim3(kRopeThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, pa_dtype dt, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (head_dim == 128) return dt == PA_BF16 ? launch_t<128, __nv_bfloat16>(p, stream) : launch_t<128, __half>(p, stream);
  if (head_dim == 64) return dt == PA_BF16 ? launch_t<64, __nv_bfloat16>(p, stream) : launch_t<64, __half>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
