// Selection of the pages a query reads: its first n_sink pages, its newest
// n_recent ones (its own among them) and, up to k pages, those with the highest
// score, the lower index first among equals; in position order.
//
// Every page gets a 32-bit key in the order of its score (pages that are always
// taken rank above every score, NaN below); the k-th largest key is found two
// bits at a time by counting, and one ordered pass writes the pages above it
// and as many equal to it, from the front, as are still wanted.
#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct SelectArgs {
  const int32_t* table;
  const int32_t* seq_lens;
  const float* scores;
  int32_t* sel_table;
  int32_t* sel_pages;
  int32_t* sel_lens;
  int* status;
  int max_pages, max_seq_len, width, s_q, k, n_sink, n_recent;
};

// Key of a score: unsigned order = score order, -0 = +0, NaN lowest.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  if (v != v) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kThreads) page_select_kernel(const SelectArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ int cnt[2][kWarps][4];
  __shared__ int base[kWarps][2];
  const int b = blockIdx.y, i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int T = __ldg(a.seq_lens + b);
  if (T < 0 || T > a.max_seq_len) {
    if (tid == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    T = T < 0 ? 0 : a.max_seq_len;
  }
  const int L = T - a.s_q + 1 + i;
  const int n = L > 0 ? (L - 1) / kPage + 1 : 0;  // pages the query sees
  const int take = min(n, a.k);
  const size_t q = static_cast<size_t>(b) * a.s_q + i;
  const float* sc = a.scores + q * a.width;
  auto key = [&](int p) -> uint32_t {
    if (n <= a.k || p < a.n_sink || p >= n - a.n_recent) return 0xffffffffu;
    return score_key(__ldg(sc + p));
  };
  // the take-th largest key
  uint32_t thr = 0xffffffffu;
  int above = 0;  // keys above thr
  if (n > a.k) {
    thr = 0u;
    int round = 0;
    for (int bit = 30; bit >= 0; bit -= 2, ++round) {
      int c[4] = {0, 0, 0, 0};
      for (int p = tid; p < n; p += kThreads) {
        const uint32_t u = key(p);
#pragma unroll
        for (int d = 1; d < 4; ++d) c[d] += u >= (thr | (static_cast<uint32_t>(d) << bit));
      }
#pragma unroll
      for (int d = 1; d < 4; ++d) {
        c[d] = __reduce_add_sync(0xffffffffu, c[d]);
        if (lane == 0) cnt[round & 1][warp][d] = c[d];
      }
      __syncthreads();
      int t[4] = {0, 0, 0, 0};
      for (int w = 0; w < kWarps; ++w)
#pragma unroll
        for (int d = 1; d < 4; ++d) t[d] += cnt[round & 1][w][d];
      const uint32_t d = t[3] >= take ? 3u : t[2] >= take ? 2u : t[1] >= take ? 1u : 0u;
      thr |= d << bit;
    }
    int c = 0;
    for (int p = tid; p < n; p += kThreads) c += key(p) > thr;
    c = __reduce_add_sync(0xffffffffu, c);
    __syncthreads();
    if (lane == 0) cnt[0][warp][0] = c;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) above += cnt[0][w][0];
  }
  const int ties = take - above;  // pages equal to thr that are taken, lowest first
  // ordered pass: slot = pages above before p + min(ties, equal ones before p)
  int32_t* out = a.sel_table + q * a.k;
  int32_t* out_pages = a.sel_pages ? a.sel_pages + q * a.k : nullptr;
  int gt0 = 0, eq0 = 0;
  for (int p0 = 0; p0 < n; p0 += kThreads) {
    const int p = p0 + tid;
    const uint32_t u = p < n ? key(p) : 0u;
    const bool gt = p < n && u > thr, eq = p < n && u == thr;
    const uint32_t mg = __ballot_sync(0xffffffffu, gt), me = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) {
      base[warp][0] = __popc(mg);
      base[warp][1] = __popc(me);
    }
    __syncthreads();
    int g = gt0, e = eq0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        g += base[w][0];
        e += base[w][1];
      }
      gt0 += base[w][0];
      eq0 += base[w][1];
    }
    const uint32_t below = (1u << lane) - 1;
    g += __popc(mg & below);
    e += __popc(me & below);
    if (gt || (eq && e < ties)) {
      const int slot = g + min(e, ties);
      out[slot] = p < a.max_pages ? __ldg(a.table + static_cast<size_t>(b) * a.max_pages + p) : -1;
      if (out_pages) out_pages[slot] = p;
    }
  }
  for (int s = take + tid; s < a.k; s += kThreads) {
    out[s] = -1;
    if (out_pages) out_pages[s] = -1;
  }
  if (tid == 0) a.sel_lens[q] = n > 0 ? (take - 1) * kPage + (L - 1) % kPage + 1 : 0;
}

}  // namespace

cudaError_t launch_page_select(const PageSelectLaunch& L) {
  SelectArgs a{L.table, L.seq_lens, L.scores, L.sel_table, L.sel_pages, L.sel_lens, L.status,
               L.max_pages, L.max_seq_len, L.width, L.s_q, L.k_pages, L.n_sink, L.n_recent};
  return launch_dependent(page_select_kernel, dim3(L.s_q, L.B), dim3(kThreads), 0, L.stream, a);
}

}  // namespace mla
