// The second half of pa_decode_accumulate, for sm_103a: the logits that the
// partition pass of decode stored become attention weights, and each cached
// token's score grows by the sum of its weights over the query group.
//
//   scores_out[row][g][t] = scores[row][g][t] + sum_h 2^(s_h,t - M_h) / L_h
//
// with s in log2 units, M_h the largest partition reference and L_h the
// partitions' sums brought to it (what the log-sum-exp merge divides by).  One
// thread owns a token and adds its heads in order, so the result is the same
// bits on every run; nothing is atomic.
//
// Bound by memory: 4 * group bytes of logits (just written, mostly still in
// L2) and 8 bytes of score per token and KV head, beside the 4 * head_dim
// bytes of K and V that the partition pass reads.
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr int kAccThreads = 256;
constexpr int kAccTokens = 2048;  // tokens of a CTA
constexpr int kMaxGroup = 16;
constexpr unsigned kAll = 0xffffffffu;

__global__ void __launch_bounds__(kAccThreads) accumulate_kernel(const AccumulateParams p) {
  __shared__ float s_m[kMaxGroup], s_inv[kMaxGroup];
  griddep_wait();
  griddep_launch_dependents();
  const int r = blockIdx.z, h = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int ctx = __ldg(p.lens + r);
  ctx = ctx < 0 ? 0 : min(ctx, p.cap);
  const int row = p.score_rows ? __ldg(p.score_rows + r) : r;
  const int t0 = blockIdx.x * kAccTokens;
  if (row < 0 || t0 >= ctx) {
    if (row >= p.num_rows && t0 == 0 && tid == 0) record_error(p.err, PA_DEVERR_SCORE_ROW);
    return;
  }
  bool twice = false;  // an earlier request has this row: it alone keeps score
  if (p.score_rows)
    for (int i = tid; i < r; i += kAccThreads) twice |= __ldg(p.score_rows + i) == row;
  if (__syncthreads_or(twice) || row >= p.num_rows) {
    if (tid == 0) record_error(p.err, PA_DEVERR_SCORE_ROW);
    return;
  }
  if (ctx > p.score_len) {
    if (tid == 0) record_error(p.err, PA_DEVERR_CONTEXT_LEN);
    ctx = p.score_len;
  }
  const int nsplit = (min(__ldg(p.lens + r), p.cap) + p.split_tokens - 1) / p.split_tokens;
  const int G = p.group;
  for (int g = warp; g < G; g += kAccThreads / 32) {
    const size_t prow = ((size_t)r * p.q_heads + h * G + g) * p.max_splits;
    float M = -INFINITY;
    for (int c = lane; c < nsplit; c += 32) M = fmaxf(M, p.part_m[prow + c]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    if (M == -INFINITY) M = 0.f;
    float l = 0.f;
    for (int c = lane; c < nsplit; c += 32) l += exp2f(p.part_m[prow + c] - M) * p.part_w[prow + c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
    if (lane == 0) {
      s_m[g] = M;
      s_inv[g] = l > 0.f ? 1.f / l : 0.f;
    }
  }
  __syncthreads();
  const int t1 = min(t0 + kAccTokens, ctx);
  const size_t at = ((size_t)row * p.kv_heads + h) * p.score_len;
  const float* lg = p.logits + ((size_t)r * p.kv_heads + h) * p.cap * G;
  for (int t = t0 + tid; t < t1; t += kAccThreads) {
    float w = 0.f;
    for (int g = 0; g < G; ++g) w += exp2f(lg[(size_t)t * G + g] - s_m[g]) * s_inv[g];
    p.scores_out[at + t] = p.scores[at + t] + w;
  }
}

}  // namespace

cudaError_t launch_accumulate(const AccumulateParams& p, cudaStream_t stream) {
  const unsigned chunks = (unsigned)(((int64_t)p.cap + kAccTokens - 1) / kAccTokens);
  return launch_pdl(accumulate_kernel, dim3(chunks, p.kv_heads, p.num_seqs), dim3(kAccThreads), 0, stream, p);
}

}  // namespace pa
