// Expected attention mass of each candidate page of a query:
//   S[h, p]  = scale * (q_h . kbar_p),  kbar_p the page's mean key
//   mass[p]  = sum_h softmax_p(S[h, :])[p]
// over the complete pages before the query's own one.
#include <math_constants.h>

#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

struct ScoreArgs {
  const __nv_bfloat16* digests;
  const int32_t* table;
  const int32_t* seq_lens;
  const __nv_bfloat16* q_c;
  const __nv_bfloat16* q_r;
  float* scores;
  int* status;
  int num_pages, max_pages, max_seq_len, s_q, H, width;
  float scale_log2;
};

__device__ float block_reduce(float v, bool is_max, float* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = is_max ? fmaxf(v, u) : v + u;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  v = buf[0];
  for (int w = 1; w < 8; ++w) v = is_max ? fmaxf(v, buf[w]) : v + buf[w];
  return v;
}

__global__ void __launch_bounds__(256) page_scores_kernel(const ScoreArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  extern __shared__ float smem[];
  __shared__ float q[kDqk], buf[8];
  float* s = smem;
  float* mass = smem + a.width;
  const int b = blockIdx.y, i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int T = __ldg(a.seq_lens + b);
  if (T < 0 || T > a.max_seq_len) {
    if (tid == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    T = T < 0 ? 0 : a.max_seq_len;
  }
  const int L = T - a.s_q + 1 + i, P = L > 0 ? (L - 1) / kPage : 0;
  for (int p = tid; p < P; p += 256) mass[p] = 0.0f;
  for (int h = 0; h < a.H; ++h) {
    const size_t row = (static_cast<size_t>(b) * a.s_q + i) * a.H + h;
    __syncthreads();
    for (int c = tid; c < kDqk; c += 256)
      q[c] = __bfloat162float(c < kDc ? a.q_c[row * kDc + c] : a.q_r[row * kDr + c - kDc]);
    __syncthreads();
    float m = -CUDART_INF_F;
    for (int p = warp; p < P; p += 8) {
      const int page = lookup_page(a.table, a.max_pages, a.num_pages, b, p * kPage);
      float dot = 0.0f;
      if (page >= 0)
        for (int c = lane; c < kDqk; c += 32)
          dot = fmaf(q[c], __bfloat162float(a.digests[static_cast<size_t>(page) * kDqk + c]), dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (page < 0 && lane == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
      const float v = page >= 0 ? dot * a.scale_log2 : -CUDART_INF_F;
      if (lane == 0) s[p] = v;
      m = fmaxf(m, v);
    }
    m = block_reduce(m, true, buf);
    if (m == -CUDART_INF_F) m = 0.0f;
    float sum = 0.0f;
    for (int p = tid; p < P; p += 256) sum += s[p] = exp2f(s[p] - m);
    sum = block_reduce(sum, false, buf);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    for (int p = tid; p < P; p += 256) mass[p] = fmaf(s[p], inv, mass[p]);
  }
  __syncthreads();
  float* out = a.scores + (static_cast<size_t>(b) * a.s_q + i) * a.width;
  for (int p = tid; p < a.width; p += 256) {
    const bool ok = p < P && lookup_page(a.table, a.max_pages, a.num_pages, b, p * kPage) >= 0;
    out[p] = ok ? mass[p] : -CUDART_INF_F;
  }
}

}  // namespace

cudaError_t launch_page_scores(const PageScoresLaunch& L) {
  ScoreArgs a{static_cast<const __nv_bfloat16*>(L.digests), L.table, L.seq_lens,
              static_cast<const __nv_bfloat16*>(L.q_c), static_cast<const __nv_bfloat16*>(L.q_r), L.scores, L.status,
              L.num_pages, L.max_pages, L.max_seq_len, L.s_q, L.H, L.width, L.scale * kLog2e};
  const size_t smem = 2 * sizeof(float) * static_cast<size_t>(L.width);
  if (smem > 200 * 1024) return cudaErrorNotSupported;
  const cudaError_t e = cudaFuncSetAttribute(page_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e != cudaSuccess) return e;
  return launch_dependent(page_scores_kernel, dim3(L.s_q, L.B), dim3(256), smem, L.stream, a);
}

}  // namespace mla
