// Selection of the pages a query reads: its first n_sink pages, its newest
// n_recent ones (its own among them) and, up to k pages, those with the highest
// score, the lower index first among equals; in position order.
//
// One CTA a query. Every candidate gets a 32-bit key in the order of its score
// (NaN lowest). The key of the last page taken is found two bits at a time, over
// the bits in which candidates differ, by counting the keys at or above each of
// three thresholds: one barrier a step, and the search ends when a threshold has
// exactly the wanted count at or above it. A thread holds consecutive pages in
// registers, so one scan over the threads gives each page its place. Latency is
// all there is to it (0.4 MB for 256 queries of up to 512 pages, 6.5 us);
// counting in histograms would meet its worst case, equal digits, whenever many
// scores are equal.
#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

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

// kItems consecutive pages a thread; a query of more than kItems * kThreads
// pages is walked in rounds of that many, its keys read again each time.
template <int kThreads, int kItems>
__global__ void __launch_bounds__(kThreads) page_select_kernel(const SelectArgs a) {
  constexpr int kWarps = kThreads / 32, kRound = kThreads * kItems;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  __shared__ uint32_t sums[3][3];
  __shared__ uint2 range[kWarps];
  __shared__ int2 scan[2][kWarps];
  const int b = blockIdx.y, i = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const size_t q = static_cast<size_t>(b) * a.s_q + i;
  const float* sc = a.scores + q * a.width;
  const int32_t* row = a.table + static_cast<size_t>(b) * a.max_pages;
  int T = __ldg(a.seq_lens + b);
  if (T < 0 || T > a.max_seq_len) {
    if (tid == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    T = T < 0 ? 0 : a.max_seq_len;
  }
  const int L = T - a.s_q + 1 + i;
  const int n = L > 0 ? (L - 1) / kPage + 1 : 0;  // pages the query sees
  const int take = min(n, a.k);
  const bool all = n <= a.k;
  const int lo = all ? n : a.n_sink, hi = all ? n : n - a.n_recent;  // candidates; the others are taken
  const int rounds = (n + kRound - 1) / kRound;
  uint32_t u[kItems];
  int held = -1;  // round whose keys u holds
  auto load = [&](int r) {
    if (held == r) return;
    held = r;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int p = r * kRound + tid * kItems + j;
      u[j] = p >= lo && p < hi ? score_key(__ldg(sc + p)) : 0u;
    }
  };
  // Keys at or above each of three thresholds, none of them zero, over the CTA.
  // Three buffers in turn: one in use, one being read by late warps, one cleared
  // for the next. Two counts share a word where a query's pages fit 16 bits.
  constexpr bool kWide = kRound > 8192;  // the instance that takes any number of pages
  int step = 0;
  auto count3 = [&](uint32_t t1, uint32_t t2, uint32_t t3) {
    uint32_t c1 = 0, c2 = 0, c3 = 0;
    for (int r = 0; r < rounds; ++r) {
      load(r);
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        c1 += (u[j] >= t1 ? 1u : 0u) + (!kWide && u[j] >= t2 ? 0x10000u : 0u);
        if (kWide) c2 += u[j] >= t2 ? 1u : 0u;
        c3 += u[j] >= t3 ? 1u : 0u;
      }
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    if (kWide) c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    uint32_t* buf = sums[step % 3];
    uint32_t* next = sums[(step + 1) % 3];
    ++step;
    if (lane == 0) {
      atomicAdd(buf, c1);
      if (kWide) atomicAdd(buf + 1, c2);
      atomicAdd(buf + 2, c3);
    }
    if (tid < 3) next[tid] = 0u;
    __syncthreads();
    return kWide ? make_int3(buf[0], buf[1], buf[2]) : make_int3(buf[0] & 0xffffu, buf[0] >> 16, buf[2]);
  };
  const int want = take - (all ? take : a.n_sink + a.n_recent);  // candidates to take
  uint32_t thr = 0xffffffffu;  // candidates above it are taken, and `ties` equal to it
  int ties = 0;
  if (want > 0) {
    uint32_t any = 0u, every = 0xffffffffu;
    for (int r = 0; r < rounds; ++r) {
      load(r);
#pragma unroll
      for (int j = 0; j < kItems; ++j) {
        const int p = r * kRound + tid * kItems + j;
        any |= u[j];
        every &= p >= lo && p < hi ? u[j] : 0xffffffffu;
      }
    }
    any = __reduce_or_sync(0xffffffffu, any);
    every = __reduce_and_sync(0xffffffffu, every);
    if (lane == 0) range[warp] = make_uint2(any, every);
    if (tid < 3) sums[0][tid] = 0u;
    __syncthreads();
    any = __reduce_or_sync(0xffffffffu, lane < kWarps ? range[lane].x : 0u);
    every = __reduce_and_sync(0xffffffffu, lane < kWarps ? range[lane].y : 0xffffffffu);
    const uint32_t vary = any ^ every;  // bits in which candidates differ; the others need no search
    thr = every;
    int bit = 30;
    bool exact = false;  // exactly `want` keys are at or above thr
    for (; bit >= 0 && !exact; bit -= 2) {
      if ((vary >> bit & 3u) == 0u) continue;
      const uint32_t base2 = thr & ~(3u << bit);
      const uint32_t t1 = base2 | (1u << bit), t2 = base2 | (2u << bit), t3 = base2 | (3u << bit);
      const int3 c = count3(t1, t2, t3);
      const int at = c.z >= want ? c.z : c.y >= want ? c.y : c.x >= want ? c.x : -1;
      if (at >= 0) thr = c.z >= want ? t3 : c.y >= want ? t2 : t1;
      exact = at == want;
    }
    if (exact) {
      --thr;  // every key at or above the old one is above this one; it is at least 1 there
    } else {
      const int above = thr == 0xffffffffu ? 0 : count3(thr + 1, thr + 1, thr + 1).x;
      ties = want - above;
    }
  }
  // one ordered pass: a page's place is the number of pages taken before it
  int32_t* out = a.sel_table + q * a.k;
  int32_t* out_pages = a.sel_pages ? a.sel_pages + q * a.k : nullptr;
  int base = 0, base_eq = 0;  // taken for certain, and equal to thr, in the rounds before
  for (int r = 0; r < rounds; ++r) {
    if (want > 0) load(r);
    int sure = 0, eq = 0;
    uint32_t is_sure = 0, is_eq = 0;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int p = r * kRound + tid * kItems + j;
      const bool cand = p >= lo && p < hi;
      const bool s = p < n && (!cand || (want > 0 && u[j] > thr));
      const bool e = cand && want > 0 && ties > 0 && u[j] == thr;
      is_sure |= static_cast<uint32_t>(s) << j;
      is_eq |= static_cast<uint32_t>(e) << j;
    }
    sure = __popc(is_sure);
    eq = __popc(is_eq);
    int is = sure, ie = eq;  // inclusive scans over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, is, o), y = __shfl_up_sync(0xffffffffu, ie, o);
      if (lane >= o) {
        is += x;
        ie += y;
      }
    }
    int2* buf = scan[r & 1];
    if (lane == 31) buf[warp] = make_int2(is, ie);
    __syncthreads();
    int s0 = base + is - sure, e0 = base_eq + ie - eq;  // before this thread's pages
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        s0 += buf[w].x;
        e0 += buf[w].y;
      }
      base += buf[w].x;
      base_eq += buf[w].y;
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
      const int p = r * kRound + tid * kItems + j;
      const bool s = (is_sure >> j) & 1, e = (is_eq >> j) & 1;
      if (s || (e && e0 < ties)) {
        const int slot = s0 + min(e0, ties);
        out[slot] = __ldg(row + p);
        if (out_pages) out_pages[slot] = p;
      }
      s0 += s;
      e0 += e;
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
  const dim3 grid(L.s_q, L.B);
  // Keys in registers up to 16,384 pages (a million tokens); longer queries read
  // theirs again in each step. Few keys a thread keep a step short, few warps its
  // barrier (2,048 pages: 6.7 us with 512 threads, 8.7 with eight keys each on 512,
  // 9.7 with sixteen on 256, 10.2 with four on 1,024).
  if (L.width <= 256) return launch_dependent(page_select_kernel<128, 2>, grid, dim3(128), 0, L.stream, a);
  if (L.width <= 1024) return launch_dependent(page_select_kernel<256, 4>, grid, dim3(256), 0, L.stream, a);
  if (L.width <= 2048) return launch_dependent(page_select_kernel<512, 4>, grid, dim3(512), 0, L.stream, a);
  if (L.width <= 4096) return launch_dependent(page_select_kernel<512, 8>, grid, dim3(512), 0, L.stream, a);
  if (L.width <= 8192) return launch_dependent(page_select_kernel<1024, 8>, grid, dim3(1024), 0, L.stream, a);
  return launch_dependent(page_select_kernel<1024, 16>, grid, dim3(1024), 0, L.stream, a);
}

}  // namespace mla
