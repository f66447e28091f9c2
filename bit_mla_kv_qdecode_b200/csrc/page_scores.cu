// Expected attention mass of each candidate page of a query, on the tensor cores:
//   S[h, p]  = scale * (q_h . kbar_p),  kbar_p the page's mean key
//   mass[p]  = sum_h exp(S[h, p]) / sum_p' exp(S[h, p'])
// over the complete pages p before the query's own one.
//
// A cluster of C CTAs takes one query; tile t of 128 pages goes to CTA t mod C.
// Heads are the MMA's M side (one TMEM lane a head), pages its N side, so a
// head's maximum and sum run along its lane's own columns, with no exchange
// between lanes; only the last sum, over heads, crosses lanes. A CTA keeps the
// logits of two tiles in tensor memory: up to 2 * C tiles (262,144 tokens at 16
// CTAs) the statistics of the whole query are known before any logit is read
// again, and none goes through memory. A longer query's tiles are computed
// twice, first for the statistics. (Pages as the M side, with the statistics
// reduced across lanes, took 3.7 us a tile of 128 heads for them instead of 1.1.)
//
// Precision. The tensor cores' fp32 accumulation truncates, in proportion to
// the sum so far and to the steps: with one accumulator for all 576 channels
// the scores of pages that hold most of the mass were off by 2e-6. A logit is
// therefore summed in three accumulators of 192 channels each, added in fp32.
// The first is the tile's own; the other two are scratch that every tile uses
// and that is free again once the statistics pass has added the three up.
//
// Digests are gathered by the block table with 16-byte asynchronous copies into
// the swizzled operand layout, 64 channels of 128 pages a stage; the query's
// heads come with nine tiled loads and stay for all tiles. (TMA's gather of four
// rows a request moved 10 GB/s an SM at 128 bytes a row, these copies 38 with the
// four stages that 128 heads leave room for, 48 where HBM is the limit.)
// Warp roles:
//   warps 0-7   a quarter of the heads and half of a tile's pages each:
//               statistics, later weights and their sum over the heads
//   warps 8-11  copies (eight were 2 % slower: fewer registers for the others)
//   warps 12-14 MMA issue, one accumulator each (a stage costs its issuing
//               thread 380 ns of waits and issue, its MMAs 130); tensor memory
// The CTAs' statistics meet in distributed shared memory, in rank order, so
// results do not depend on timing. Every wait is bounded; one that runs out
// sets MLA_ERR_TIMEOUT and leaves the scores undefined.
#include <math_constants.h>

#include <algorithm>
#include <mutex>

#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace mla {
namespace {

constexpr int kSoftWarps = 8, kCopyWarps = 4;
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kMaxCluster = 16;
constexpr int kAccs = 3;                           // accumulators of a logit, a warp that issues for each
constexpr int kMmaWarp = kSoftWarps + kCopyWarps;  // the first of them
constexpr int kThreads = (kMmaWarp + kAccs) * 32;
constexpr int kTile = 128;                         // pages of a tile
constexpr int kCopyPages = kTile / kCopyWarps;     // of them a copying warp takes
constexpr int kBlockCh = 64;                       // channels of one operand stage (128 B a row)
constexpr int kBlocks = kDqk / kBlockCh;           // 9: eight of the content, one of the RoPE part
constexpr int kStageBytes = kTile * kBlockCh * 2;  // 16 KB
constexpr int kMaxStages = 12;
constexpr int kHeld = 2;                           // tiles whose logits tensor memory holds
constexpr uint32_t kScratchCol = kHeld * kTile;
constexpr uint32_t kTmemCols = 512;
static_assert(kAccs == 3 && kHeld == 2 && kBlocks % kAccs == 0 && (kHeld + kAccs - 1) * kTile <= static_cast<int>(kTmemCols), "accumulators");
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kSmemLimit = 232448;

struct ScoreArgs {
  const __nv_bfloat16* digests;  // [num_pages][576]
  const int32_t* table;
  const int32_t* seq_lens;
  float* scores;
  int* status;
  int num_pages, max_pages, max_seq_len, s_q, H, width;
  int q_block, stages;  // bytes of a query block in shared memory; operand stages of the ring
  float scale_log2;
};

struct Maps {
  CUtensorMap q_c;  // bf16 [B * s_q * H][512], box 64 x H
  CUtensorMap q_r;  // bf16 [B * s_q * H][64], box 64 x H
};

struct Misc {
  uint64_t full[kMaxStages], empty[kMaxStages], q_full[kBlocks], t_full[kHeld], t_empty[kHeld], scratch_empty;
  float2 half[kScoreHeads];               // (maximum, sum) of each head over one half of the CTA's pages
  union {
    float2 part[kMaxCluster][kScoreHeads];  // over each CTA's pages, written by the CTAs
    float mass[2][4][kTile];                // later: a tile's weights, summed over a quarter of the heads
  };
  uint32_t ok[2][kTile / 32];   // a tile's pages that count
  uint32_t tmem;
  int abort;
};
// Shared memory: query blocks, ring, Misc. A query block holds the heads there
// are, in whole groups of eight rows; the MMA reads 128 rows, those past the heads
// from whatever follows (their lanes are not used), which the ring's size covers.
constexpr int kMinStages = 4;
constexpr int kSmemFixed = static_cast<int>(sizeof(Misc)) + 1024;
static_assert(kBlocks * kScoreHeads * 128 + kMinStages * kStageBytes + kSmemFixed <= kSmemLimit, "shared memory budget");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Arrive on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tma_load_2d(void* dst, const void* tmap, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(ptx::smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

// K-major operand of 128-byte rows in the 128-byte swizzle: 8-row groups 1,024 B apart.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftThreads) : "memory"); }

// Fold (top, sum) of another part into (m, l): sums of 2^(x - maximum).
__device__ __forceinline__ void fold(float& m, float& l, float top, float sum) {
  const float up = fmaxf(m, top);
  if (up == -CUDART_INF_F) return;
  l = fmaf(l, exp2_approx(m - up), sum * exp2_approx(top - up));
  m = up;
}

// Sum each of 16 columns over the warp's lanes; lane l returns column l & 15's.
__device__ __forceinline__ float sum_columns(float (&v)[16], int lane) {
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int k = 0; k < s; ++k) {
      const float keep = up ? v[s + k] : v[k], give = up ? v[k] : v[s + k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, give, s);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// kTwice: a CTA may have more tiles than it can hold, and goes over them twice.
template <bool kTwice>
__global__ void __launch_bounds__(kThreads, 1) page_scores_kernel(const ScoreArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* qbuf = smem;
  uint8_t* ring = qbuf + kBlocks * a.q_block;
  Misc& m = *reinterpret_cast<Misc*>(ring + a.stages * kStageBytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  int C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const int unit = blockIdx.x / C, b = unit / a.s_q, i = unit - b * a.s_q;

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      ptx::mbar_init(&m.full[s], kCopyWarps * 32);
      ptx::mbar_init(&m.empty[s], 1);
    }
    for (int k = 0; k < kBlocks; ++k) ptx::mbar_init(&m.q_full[k], 1);
    for (int t = 0; t < kHeld; ++t) {
      ptx::mbar_init(&m.t_full[t], kAccs);
      ptx::mbar_init(&m.t_empty[t], kSoftWarps);
    }
    ptx::mbar_init(&m.scratch_empty, kSoftWarps);
    m.abort = 0;
    ptx::fence_mbar_init_cluster();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&m.tmem, kTmemCols);
    ptx::tmem_relinquish();
  }
  if (tid == kSoftThreads) {
    ptx::prefetch_tmap(&maps.q_c);
    ptx::prefetch_tmap(&maps.q_r);
  }
  ptx::tc_fence_before();
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // waited for before the first remote store
  ptx::tc_fence_after();
  const uint32_t tmem = m.tmem;
  ptx::griddep_wait();

  // the copying warps' first table entries come along with the length
  const int copy_page = kCopyPages * (warp - kSoftWarps) + lane % kCopyPages;  // of a tile: the page this lane looks up
  auto table_at = [&](int p) { return p < a.max_pages ? __ldg(a.table + static_cast<size_t>(b) * a.max_pages + p) : -1; };
  int entry = -1;
  if (warp >= kSoftWarps && warp < kMmaWarp) entry = table_at(rank * kTile + copy_page);
  int T = __ldg(a.seq_lens + b);
  if (T < 0 || T > a.max_seq_len) {
    if (tid == 0 && rank == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    T = T < 0 ? 0 : a.max_seq_len;
  }
  const int L = T - a.s_q + 1 + i, P = L > 0 ? (L - 1) / kPage : 0;
  const int tiles = (P + kTile - 1) / kTile;
  const int mine = a.num_pages > 0 && tiles > rank ? (tiles - 1 - rank) / C + 1 : 0;
  volatile int* abort_flag = &m.abort;
  auto give_up = [&] {
    *abort_flag = 1;
    record_error(a.status, MLA_ERR_TIMEOUT);
  };
  // A whole warp waits; when one lane's wait runs out, all of them leave together.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort_flag, kWaitLimitNs));
    if (!ok) give_up();
    return ok;
  };
  auto page_ok = [&](int p) { return p < P && page_valid(table_at(p), a.num_pages); };
  auto tile_of = [&](int n) { return rank + (n < mine ? n : n - mine) * C; };  // n counts over both sweeps

  // Copy the digests of this CTA's tiles into the ring. Eight lanes take one
  // page's 128 bytes of a stage, a warp kCopyPages pages. `entry` is the lane's table
  // entry of the next tile.
  auto produce = [&](int n0, int n1) {
    const int w = warp - kSoftWarps, sub = lane >> 3, chunk = lane & 7;
    for (int n = n0; n < n1; ++n) {
      // pages that are none read page 0; their logits are masked
      const bool ok = tile_of(n) * kTile + copy_page < P && page_valid(entry, a.num_pages);
      const int mine_page = ok ? entry : 0;
      const uint8_t* src[kCopyPages / 4];
#pragma unroll
      for (int j = 0; j < kCopyPages / 4; ++j) {
        const int page = __shfl_sync(0xffffffffu, mine_page, 4 * j + sub);
        src[j] = reinterpret_cast<const uint8_t*>(a.digests + static_cast<size_t>(page) * kDqk) + 16 * chunk;
      }
      if (n + 1 < 2 * mine) entry = table_at(tile_of(n + 1) * kTile + copy_page);
      for (int k = 0; k < kBlocks; ++k) {
        const int it = n * kBlocks + k, round = it / a.stages, s = it - round * a.stages;
        if (round > 0 && !warp_wait(&m.empty[s], (round - 1) & 1)) return;
        const uint32_t dst = ptx::smem_u32(ring + s * kStageBytes) + kCopyPages * w * 128;
#pragma unroll
        for (int j = 0; j < kCopyPages / 4; ++j) {
          const int r = 4 * j + sub;
          cp_async16(dst + r * 128 + ((chunk ^ (r & 7)) << 4), src[j] + k * (kBlockCh * 2));
        }
        cp_async_arrive(&m.full[s]);
      }
    }
  };

  // Accumulator e takes channel blocks e, e + 3 and e + 6.
  auto issue = [&](int n0, int n1) {
    constexpr uint32_t idesc = ptx::idesc_bf16_f32(kScoreHeads, kTile, 0, 0);
    const int e = warp - kMmaWarp;
    for (int n = n0; n < n1; ++n) {
      const int buf = n % kHeld;
      const uint32_t d = tmem + (e == 0 ? buf * kTile : kScratchCol + (e - 1) * kTile);
      bool ok = true;
      if (e == 0 && n >= kHeld) ok = ptx::mbar_wait(&m.t_empty[buf], (n / kHeld - 1) & 1, abort_flag, kWaitLimitNs);
      if (e > 0 && n > 0) ok = ptx::mbar_wait(&m.scratch_empty, (n - 1) & 1, abort_flag, kWaitLimitNs);
      for (int k = e; ok && k < kBlocks; k += kAccs) {
        const int it = n * kBlocks + k, round = it / a.stages, s = it - round * a.stages;
        ok = ptx::mbar_wait(&m.full[s], round & 1, abort_flag, kWaitLimitNs) &&
             (n > 0 || ptx::mbar_wait(&m.q_full[k], 0, abort_flag, kWaitLimitNs));
        if (!ok) break;
        ptx::fence_proxy_async_smem();  // the copies were generic-proxy writes, seen through the barrier
        ptx::tc_fence_after();
        const uint64_t dq = smem_desc_sw128(ptx::smem_u32(qbuf + k * a.q_block));
        const uint64_t dp = smem_desc_sw128(ptx::smem_u32(ring + s * kStageBytes));
#pragma unroll
        for (int j = 0; j < kBlockCh / 16; ++j)  // 32 B of each row a step
          ptx::mma_ss(d, dq + 2 * j, dp + 2 * j, idesc, (k != e) | (j != 0));
        ptx::mma_commit(&m.empty[s]);
      }
      if (!ok) {
        give_up();
        return;
      }
      ptx::mma_commit(&m.t_full[buf]);
    }
  };

  const int quad = warp & 3, group = (warp >> 2) & 1;  // 32 heads and 64 pages of a tile
  const bool heads = 32 * quad < a.H;                  // the warp has any
  const uint32_t my_cols = tmem + (static_cast<uint32_t>(quad) << 21) + 64 * group;
  float top = -CUDART_INF_F, sum = 0.0f;  // this lane's head over the warp's pages
  float refs[kHeld][4] = {};              // of the held tiles: what each 16 columns' exponents are relative to

  // 16 columns of a tile's logits, in powers of two: the three accumulators,
  // fetched, and their sum, scaled.
  auto fetch = [&](int buf, int c, uint32_t (&r)[kAccs][16]) {
    ptx::tmem_ld16(my_cols + buf * kTile + c, r[0]);
    ptx::tmem_ld16(my_cols + kScratchCol + c, r[1]);
    ptx::tmem_ld16(my_cols + kScratchCol + kTile + c, r[2]);
  };
  auto add_up = [&](const uint32_t (&r)[kAccs][16], float (&v)[16]) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      v[k] = (__uint_as_float(r[0][k]) + __uint_as_float(r[1][k]) + __uint_as_float(r[2][k])) * a.scale_log2;
  };
  // Which of 32 pages of tile n count; bad table entries are flagged.
  auto pages_ok = [&](int n, int half) {
    const int p = tile_of(n) * kTile + 64 * group + 32 * half + lane;
    const bool ok = page_ok(p);
    if (p < P && !ok) record_error(a.status, MLA_ERR_INVALID_ARG);
    return __ballot_sync(0xffffffffu, ok);
  };
  auto release = [&](uint64_t* bar) {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
  };

  // ---- first sweep: logits and statistics ----
  if (warp < kSoftWarps) {
    for (int n = 0; n < mine; ++n) {
      const int buf = n % kHeld;
      const uint32_t ok0 = pages_ok(n, 0), ok1 = pages_ok(n, 1);
      if (!kTwice && quad == 0 && lane < 2) m.ok[n][2 * group + lane] = lane == 0 ? ok0 : ok1;
      if (!warp_wait(&m.t_full[buf], (n / kHeld) & 1)) break;
      ptx::tc_fence_after();
      if (heads) {
        uint32_t r[kAccs][16];
        fetch(buf, 0, r);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 16 * q;
          float v[16];
          ptx::tmem_ld_wait();
          add_up(r, v);
          if (q < 3) fetch(buf, c + 16, r);  // on its way while these columns are worked on
          const uint32_t mask = (q < 2 ? ok0 : ok1) >> (c & 16) & 0xffffu;
          if (mask != 0xffffu) {
#pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = (mask >> k) & 1 ? v[k] : -CUDART_INF_F;
          }
          float up = top;
#pragma unroll
          for (int k = 0; k < 16; ++k) up = fmaxf(up, v[k]);
          const float ref = up == -CUDART_INF_F ? 0.0f : up;
          float s0 = sum * exp2_approx(top - ref), s1 = 0.0f;
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            s0 += v[k] = exp2_approx(v[k] - ref);
            s1 += v[k + 1] = exp2_approx(v[k + 1] - ref);
          }
          if (!kTwice) {
            ptx::tmem_st16(my_cols + buf * kTile + c, v);
            if (n == 0) refs[0][q] = ref;
            if (n == 1) refs[1][q] = ref;
          }
          sum = s0 + s1;
          top = up;
        }
        if (!kTwice) ptx::tmem_st_wait();
      }
      if (kTwice) release(&m.t_empty[buf]);
      release(&m.scratch_empty);
    }
    // the halves' statistics, then every CTA's in every CTA's memory
    const int h = 32 * quad + lane;
    if (group == 1) m.half[h] = make_float2(top, sum);
    soft_sync();
    if (group == 0) fold(top, sum, m.half[h].x, m.half[h].y);
    } else if (warp < kMmaWarp) {
    if (tid == kSoftThreads && mine > 0) {
      for (int k = 0; k < kBlocks; ++k) {  // rows past the heads keep what they hold: their lanes are not read
        ptx::mbar_arrive_expect_tx(&m.q_full[k], a.H * kBlockCh * 2);
        tma_load_2d(qbuf + k * a.q_block, k < 8 ? &maps.q_c : &maps.q_r, k < 8 ? k * kBlockCh : 0, unit * a.H,
                    &m.q_full[k]);
      }
    }
    __syncwarp();
    if (mine > 0) produce(0, mine);
  } else if (lane == 0) {
    issue(0, mine);
  }
  ptx::griddep_launch_dependents();
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA runs
  const int h = 32 * quad + lane;
  if (warp < 4 && h < a.H) {
    const uint32_t at = ptx::smem_u32(&m.part[rank][h]);
    for (int r = 0; r < C; ++r) st_cluster_f2(ptx::mapa(at, r), make_float2(top, sum));
  }
  ptx::tc_fence_before();
  __syncwarp();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  float inv = 0.0f;
  if (warp < kSoftWarps && h < a.H) {  // this lane's head over all of the query's pages
    top = -CUDART_INF_F;
    for (int r = 0; r < C; ++r) top = fmaxf(top, m.part[r][h].x);
    if (top == -CUDART_INF_F) top = 0.0f;
    sum = 0.0f;
    for (int r = 0; r < C; ++r) sum = fmaf(m.part[r][h].y, exp2_approx(m.part[r][h].x - top), sum);
    if (sum > 0.0f) inv = 1.0f / sum;
  }
  if (warp < kSoftWarps) soft_sync();  // the parts have been read; the weights take their place

  // ---- second sweep: weights and their sum over the heads ----
  if (warp < kSoftWarps) {
    float* out = a.scores + static_cast<size_t>(unit) * a.width;
    const int all = (a.width + kTile - 1) / kTile;
    for (int n = 0; rank + n * C < all; ++n) {
      if (n < mine) {
        const int k = kTwice ? mine + n : n, buf = k % kHeld;
        bool have = true;
        if (kTwice) {
          const uint32_t ok0 = pages_ok(k, 0), ok1 = pages_ok(k, 1);
          if (quad == 0 && lane < 2) m.ok[n & 1][2 * group + lane] = lane == 0 ? ok0 : ok1;
          // (after a wait that ran out the loop goes on without the tiles, so that no warp misses a barrier)
          have = warp_wait(&m.t_full[buf], (k / kHeld) & 1);
          ptx::tc_fence_after();
        }
        if (heads && have) {
          uint32_t held[kTwice ? 1 : 4][16];
          if (!kTwice) {
#pragma unroll
            for (int q = 0; q < 4; ++q) ptx::tmem_ld16(my_cols + buf * kTile + 16 * q, held[kTwice ? 0 : q]);
            ptx::tmem_ld_wait();
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int c = 16 * q;
            float v[16], f;
            if (kTwice) {
              uint32_t r[kAccs][16];
              fetch(buf, c, r);
              ptx::tmem_ld_wait();
              add_up(r, v);
              f = inv;
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = exp2_approx(v[e] - top);
            } else {
              f = exp2_approx((n == 0 ? refs[0][q] : refs[1][q]) - top) * inv;
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(held[kTwice ? 0 : q][e]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = h < a.H ? v[e] * f : 0.0f;
            const float mass = sum_columns(v, lane);
            if (lane < 16) m.mass[n & 1][quad][64 * group + c + lane] = mass;
          }
        }
        if (kTwice) {
          release(&m.t_empty[buf]);
          release(&m.scratch_empty);
        }
        soft_sync();
      }
      const int p = (rank + n * C) * kTile + tid;
      if (tid < kTile && p < a.width) {
        float total = -CUDART_INF_F;
        if (n < mine && ((m.ok[n & 1][warp] >> lane) & 1)) {
          total = m.mass[n & 1][0][tid];
          for (int q = 1; 32 * q < a.H; ++q) total += m.mass[n & 1][q][tid];
        }
        out[p] = total;
      }
    }
  } else if (kTwice && warp < kMmaWarp) {
    produce(mine, 2 * mine);
  } else if (kTwice && lane == 0) {
    issue(mine, 2 * mine);
  }
  if (a.num_pages == 0 && P > 0 && tid == 0) record_error(a.status, MLA_ERR_INVALID_ARG);

  ptx::tc_fence_before();
  __syncthreads();
  if (*abort_flag) ptx::linger();  // every thread: none frees tensor memory or leaves before
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host side

// Rows of `width` bf16 channels, in boxes of 64 channels x `rows`.
bool make_rows_map(CUtensorMap* m, const void* base, int width, int64_t n, int rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(n)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * 2};
  const cuuint32_t box[2] = {kBlockCh, static_cast<cuuint32_t>(rows)};
  return encode_swizzled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 2, dims, strides, box);
}

// Clusters of 1, 2, 4, 8 and 16 CTAs that run at once on the current device (one
// CTA an SM; clusters stay within a GPC, whose SMs they need not fill; there may be
// none of 16). Asked once a device.
constexpr int kMaxDevices = 64, kSizes = 5;
static_assert(1 << (kSizes - 1) == kMaxCluster, "cluster sizes");
std::mutex g_slots_mu;
int g_slots[kMaxDevices][kSizes];

cudaError_t cluster_slots(int (&slots)[kSizes]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_slots_mu);
  int* kept = g_slots[dev];
  if (kept[0] == 0) {
    for (auto kern : {page_scores_kernel<false>, page_scores_kernel<true>}) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
    }
    int got[kSizes];
    for (int i = 0; i < kSizes; ++i) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(1u << i);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kSmemLimit;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim = {1u << i, 1, 1};
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&got[i], page_scores_kernel<false>, &cfg);
      if (e != cudaSuccess && i + 1 == kSizes) {
        cudaGetLastError();  // no GPC takes one
        got[i] = 0;
        e = cudaSuccess;
      }
      if (e != cudaSuccess) return e;
    }
    for (int i = kSizes - 1; i >= 0; --i) kept[i] = std::max(got[i], i == 0 ? 1 : 0);
  }
  for (int i = 0; i < kSizes; ++i) slots[i] = kept[i];
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_page_scores(const PageScoresLaunch& L) {
  int slots[kSizes];
  const cudaError_t e = cluster_slots(slots);
  if (e != cudaSuccess) return e;
  const int q_block = (L.H + 7) / 8 * 1024;
  const int stages = std::min((kSmemLimit - kSmemFixed - kBlocks * q_block) / kStageBytes, kMaxStages);
  const int smem = kBlocks * q_block + stages * kStageBytes + kSmemFixed;
  const ScoreArgs a{static_cast<const __nv_bfloat16*>(L.digests), L.table, L.seq_lens, L.scores, L.status, L.num_pages,
                    L.max_pages, L.max_seq_len, L.s_q, L.H, L.width, q_block, stages, L.scale * kLog2e};
  const int64_t units = static_cast<int64_t>(L.B) * L.s_q;
  Maps maps;
  const int64_t rows = units * L.H;
  if (!make_rows_map(&maps.q_c, L.q_c, kDc, rows, L.H) || !make_rows_map(&maps.q_r, L.q_r, kDr, rows, L.H))
    return cudaErrorInvalidValue;
  // CTAs a query: those that finish soonest, in units of a tile's time; the query
  // operand is loaded once a CTA, and set-up and the statistics' exchange cost about half a tile
  const int tiles = (L.width + kTile - 1) / kTile;
  int best = 1;
  double best_cost = 1e30;
  for (int i = 0; i < kSizes; ++i) {
    if (slots[i] == 0) continue;
    const int c = 1 << i, per = (tiles + c - 1) / c;
    const int64_t waves = (units + slots[i] - 1) / slots[i];
    const double cost = waves * (per * (per > kHeld ? 2.0 : 1.0) + L.H / 128.0 + 0.5);
    if (cost < best_cost * 0.97) {
      best_cost = cost;
      best = c;
    }
  }
  auto kern = (tiles + best - 1) / best > kHeld ? page_scores_kernel<true> : page_scores_kernel<false>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(units * best));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;  // more than half of an SM's: one CTA keeps the 512-column TMEM allocation uncontended
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(best), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

}  // namespace mla
