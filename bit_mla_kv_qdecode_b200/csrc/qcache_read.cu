// Reading the quantized cache back outside the attention: dequantized rows of a
// token range of every request, and the mean key of completed pages.
//
//   rows:    x_hat = bf16(u * s + z)
//   digest:  kbar_p = bf16( (1/64) sum_t (u_t s_t + z_t) ), fp32 sums
//
// Rows are bf16 because the projections that take them are. Digests are bf16 as the
// scores' operand type and half the bytes to read each step; the rounding, at most 2^-8 of a
// channel's mean and independent between channels, is far below what a mean says
// of its 64 keys.
//
// u * s is exact in fp32 (at most 15 significant bits), so u * s + z is one
// rounding. Codes become floats by setting them into the low bits of 2^23, where
// they stand in the word, and subtracting it (both at full rate; the conversion
// instruction runs at a quarter of it); the step takes back the power of two
// that the place is worth. Additions and products are two values an instruction.
#include <algorithm>

#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"
#include "tensor_map.h"

namespace mla {
namespace {

// Two fp32 values in one 64-bit register pair.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 make2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Codes k and k + 1 of 16 bits of packed codes, left where they are: as floats,
// 2^(BITS k) and 2^(BITS (k + 1)) times their value (exact: below 2^16).
template <int BITS>
__device__ __forceinline__ f32x2 fields2(uint32_t w, int k) {
  constexpr uint32_t kMask = (1u << BITS) - 1, kBias = 0x4B000000u;  // 2^23
  const float lo = __uint_as_float((w & (kMask << (BITS * k))) | kBias);
  const float hi = __uint_as_float((w & (kMask << (BITS * (k + 1)))) | kBias);
  return add2(make2(lo, hi), make2(-8388608.0f, -8388608.0f));
}
// Steps for fields2's values: s * 2^(-BITS k), exact.
template <int BITS>
struct Steps {
  f32x2 v[8 / BITS];  // 16 / BITS codes, two an entry
  __device__ __forceinline__ explicit Steps(float s) {
    constexpr float kDown = 1.0f / (1 << BITS);
    f32x2 x = make2(s, s * kDown);
#pragma unroll
    for (int k = 0; k < 8 / BITS; ++k) {
      v[k] = x;
      x = mul2(x, make2(kDown * kDown, kDown * kDown));
    }
  }
};
__device__ __forceinline__ uint32_t bf16x2(f32x2 v) {
  const float2 f = split2(v);
  const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ f32x2 both(float v) { return make2(v, v); }

struct ReadArgs {
  const uint8_t* pool;
  const int32_t* table;
  const int32_t* start;
  const int32_t* cu_rows;
  __nv_bfloat16* out_c;
  __nv_bfloat16* out_kr;
  int64_t c_stride, kr_stride, total_rows;
  int* status;
  int num_pages, max_pages, max_rows;
};

constexpr int kReadThreads = 256;
constexpr int kReadBatch = 4;  // tokens a warp has in flight at once, at most

// A CTA takes 8 * kTokens tokens of one page of one request, those of them that
// are asked for; a warp kTokens. Lane l takes content channels [8l, 8l + 8) and
// [256 + 8l, 264 + 8l), so that code loads and row stores are contiguous over the
// warp, and RoPE channels 2l and 2l + 1. Bound: bytes (228-388 read, 1,152
// written a token).
template <int BC, int GC, int BR, int GR, int kTokens>
__global__ void __launch_bounds__(kReadThreads) qcache_read_kernel(const ReadArgs a) {
  using G = QGeom<BC, GC, BR, GR>;
  constexpr int kParts = kPage / (kReadThreads / 32 * kTokens);  // CTAs a page
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
  const int r0 = __ldg(a.cu_rows + b), r1 = __ldg(a.cu_rows + b + 1);
  const int64_t first = a.start ? __ldg(a.start + b) : 0;
  int64_t count = static_cast<int64_t>(r1) - r0;
  const bool good = r0 >= 0 && count >= 0 && count <= a.max_rows && r1 <= a.total_rows;
  if (!good || (count > 0 && first < 0)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    if (r0 < 0 || first < 0) return;
    count = min(min(count, static_cast<int64_t>(a.max_rows)), a.total_rows - r0);
  }
  const int64_t idx = first / kPage + blockIdx.x / kParts;  // page of the request
  // slots of the page that are asked for, and this warp's first one
  const int lo = static_cast<int>(max(first - idx * kPage, static_cast<int64_t>(0)));
  const int hi = static_cast<int>(max(min(first + count - idx * kPage, static_cast<int64_t>(kPage)), static_cast<int64_t>(0)));
  const int slot0 = (blockIdx.x % kParts * (kReadThreads / 32) + warp) * kTokens;
  if (slot0 >= hi || slot0 + kTokens <= lo) return;
  const int page = idx < a.max_pages ? __ldg(a.table + static_cast<size_t>(b) * a.max_pages + idx) : -1;
  if (!page_valid(page, a.num_pages)) {
    if (lane == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const uint8_t* pg = a.pool + static_cast<size_t>(page) * G::kPageBytes;
  const int64_t row0 = r0 + idx * kPage - first + slot0;
  __nv_bfloat16* out_c = a.out_c ? a.out_c + row0 * a.c_stride + 8 * lane : nullptr;
  __nv_bfloat16* out_kr = a.out_kr ? a.out_kr + row0 * a.kr_stride + 2 * lane : nullptr;
  constexpr int kBatch = kTokens < kReadBatch ? kTokens : kReadBatch;
#pragma unroll
  for (int t0 = 0; t0 < kTokens; t0 += kBatch) {
    uint32_t code[kBatch][2], meta[kBatch][2], rcode[kBatch], rmeta[kBatch];
    const uint8_t* codes = pg + G::kOffCC + (slot0 + t0) * G::kRowC;
    const uint32_t* metas = reinterpret_cast<const uint32_t*>(pg + G::kOffCM) + (slot0 + t0) * G::kGroupsC;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {  // slots outside the range are read too (they are the page's) and not written
      if (out_c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (BC == 4)
            code[e][h] = __ldg(reinterpret_cast<const uint32_t*>(codes + e * G::kRowC) + 32 * h + lane);
          else
            code[e][h] = __ldg(reinterpret_cast<const uint16_t*>(codes + e * G::kRowC) + 32 * h + lane);
          meta[e][h] = __ldg(metas + e * G::kGroupsC + (256 * h + 8 * lane) / GC);
        }
      }
      if (out_kr) {
        const uint8_t* rrow = pg + G::kOffRC + (slot0 + t0 + e) * G::kRowR;
        rcode[e] = BR == 4 ? __ldg(rrow + lane) : __ldg(rrow + (lane >> 1)) >> (4 * (lane & 1));
        rmeta[e] = __ldg(reinterpret_cast<const uint32_t*>(pg + G::kOffRM) + (slot0 + t0 + e) * G::kGroupsR + 2 * lane / GR);
      }
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int slot = slot0 + t0 + e;
      if (slot < lo || slot >= hi) continue;
      if (out_c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Steps<BC> s(half_bits_to_float(meta[e][h]));
          const f32x2 z = both(half_bits_to_float(meta[e][h] >> 16));
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)  // 16 bits of codes at a time
            o[k] = bf16x2(fma2(fields2<BC>(code[e][h] >> (BC == 4 ? 16 * (k / 2) : 0), 2 * k % (16 / BC)),
                               s.v[k % (8 / BC)], z));
          __stcs(reinterpret_cast<uint4*>(out_c + (t0 + e) * a.c_stride + 256 * h), make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
      if (out_kr) {
        const Steps<BR> s(half_bits_to_float(rmeta[e]));
        const f32x2 z = both(half_bits_to_float(rmeta[e] >> 16));
        __stcs(reinterpret_cast<uint32_t*>(out_kr + (t0 + e) * a.kr_stride), bf16x2(fma2(fields2<BR>(rcode[e], 0), s.v[0], z)));
      }
    }
  }
}

struct DigestArgs {
  const uint8_t* pool;
  const int32_t* table;
  const int32_t* lens_before;
  const int32_t* new_lens;
  __nv_bfloat16* digests;
  int* status;
  int num_pages, max_pages, n_new;
};

// The sums on warp-level MMAs: sum_t u_t s_t over a page's 64 tokens is a product
// of the steps (one row for each group of channels) with the codes (tokens x
// channels), accumulated in fp32. A code standing alone in the low ten bits of an
// fp16 value is the subnormal u * 2^(place - 24), exact, and so are its products:
// one mask makes a pair of operands out of two tokens' codes, and the sum takes
// back the power of two. (fp32 multiply-adds on the vector unit were bound by
// their issue, 4.5 instructions a value.) Nine warps, each with 64 channels of
// its own and no exchange.
constexpr int kDigestWarps = 9;  // eight of the content, one of the RoPE part
constexpr int kDigestThreads = 32 * kDigestWarps;

// c[16 x 8] += a[16 x 16] b[16 x 8], rows 8-15 of a zero (and so c[2] and c[3]). A
// row of c that is not read may come of any row of a.
__device__ __forceinline__ void mma_steps(float (&c)[4], uint32_t a0, uint32_t a2, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(0u), "r"(a2), "r"(0u), "r"(b0), "r"(b1));
}

// Where a page part's codes are: in global memory; in shared memory; in shared
// memory in boxes of 64 rows x 128 bytes with the 128-byte swizzle.
enum class At { kGlobal, kShared, kSwizzled };

// Mean over a page's tokens of the 64 channels from 64 * part on, of codes of BITS
// in rows of CHANNELS with groups of G; out: their bf16 values.
template <int BITS, int CHANNELS, int G, At kAt>
__device__ __forceinline__ void mean_of_tokens(const uint8_t* codes, const uint8_t* metas, int part, __nv_bfloat16* out,
                                               int lane) {
  constexpr int kRow = CHANNELS * BITS / 8, kGroups = CHANNELS / G, kMine = 64 / G;  // groups of the warp: 1 or 2
  const int q = lane & 3, r = lane >> 2;
  auto load_meta = [&](int t, int g) -> uint32_t {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(metas) + t * kGroups + kMine * part + g;
    return kAt == At::kGlobal ? __ldg(p) : *p;
  };
  // eight codes of token t, unit r of the warp's channels
  auto load_unit = [&](int t) -> uint32_t {
    const int byte = BITS * (8 * part + r);  // in the token's row
    const uint8_t* p = codes + t * kRow + byte;
    if (kAt == At::kSwizzled) p = codes + byte / 128 * (kPage * 128) + t * 128 + (((byte / 16 ^ t) & 7) << 4) + byte % 16;
    if constexpr (BITS == 4)
      return kAt == At::kGlobal ? __ldg(reinterpret_cast<const uint32_t*>(p)) : *reinterpret_cast<const uint32_t*>(p);
    else
      return kAt == At::kGlobal ? __ldg(reinterpret_cast<const uint16_t*>(p)) : *reinterpret_cast<const uint16_t*>(p);
  };
  uint32_t w[4][4], m[4][4];  // K-step, token 2q + {0, 1, 8, 9} of it
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 16 * k + 2 * q + (e & 1) + 8 * (e >> 1);
      w[k][e] = load_unit(t);
      m[k][e] = load_meta(t, r % kMine);  // rows of the other lanes are not read
    }
  float z[kMine];  // offsets, over the tokens
#pragma unroll
  for (int g = 0; g < kMine; ++g)
    z[g] = half_bits_to_float(load_meta(lane, g) >> 16) + half_bits_to_float(load_meta(lane + 32, g) >> 16);
  float acc[8][4] = {};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a0 = __byte_perm(m[k][0], m[k][1], 0x5410), a2 = __byte_perm(m[k][2], m[k][3], 0x5410);
    // 16 bits of each of two tokens: all of INT2's eight codes, or four of INT4's
#pragma unroll
    for (int half = 0; half < BITS / 2; ++half) {
      const uint32_t sel = half ? 0x7632 : 0x5410;
      const uint32_t p0 = __byte_perm(w[k][0], w[k][1], sel), p1 = __byte_perm(w[k][2], w[k][3], sel);
      constexpr int kCodes = 16 / BITS, kInPlace = BITS == 4 ? 2 : 5;  // codes within the low ten bits
#pragma unroll
      for (int j = 0; j < kCodes; ++j) {
        const int down = j < kInPlace ? 0 : kInPlace * BITS;
        const uint32_t mask = ((1u << BITS) - 1) * 0x00010001u << (j * BITS - down);
        mma_steps(acc[half * kCodes + j], a0, a2, p0 >> down & mask, p1 >> down & mask);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < kMine; ++g)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z[g] += __shfl_xor_sync(0xffffffffu, z[g], o);
  // lane 4g + q holds units 2q and 2q + 1 against the steps of group g
  if (r >= kMine || 2 * q / (8 / kMine) != r) return;
  const float zr = r == 0 ? z[0] : z[kMine - 1];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        constexpr int kCodes = 16 / BITS, kInPlace = BITS == 4 ? 2 : 5;
        const int c = (j + i) % kCodes, place = c < kInPlace ? c : c - kInPlace;
        v[i] = fmaf(acc[j + i][e], static_cast<float>(1 << (24 - BITS * place)), zr) * (1.0f / kPage);
      }
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
      o[j / 2] = *reinterpret_cast<const uint32_t*>(&h);
    }
    reinterpret_cast<uint4*>(out + 64 * part)[2 * q + e] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Page of the x-th completed page of request b, or -1; bad lengths and table
// entries are flagged.
__device__ __forceinline__ int completed_page(const DigestArgs& a, int b, int x) {
  const int before = __ldg(a.lens_before + b);
  const int n = a.new_lens ? __ldg(a.new_lens + b) : a.n_new;
  if (before < 0 || n < 0 || n > a.n_new || static_cast<int64_t>(before) + n > 0x7fffffff) {
    if (x == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return -1;
  }
  const int p = before / kPage + x;
  if (p >= (before + n) / kPage) return -1;
  const int page = lookup_page(a.table, a.max_pages, a.num_pages, b, p * kPage);
  if (page < 0) record_error(a.status, MLA_ERR_INVALID_ARG);
  return page;
}

// One warp's share of a page's digest: content codes at `content`, the rest of the
// page (from its RoPE codes on) at `rest`.
template <int BC, int GC, int BR, int GR, bool kShared>
__device__ __forceinline__ void digest_warp(const uint8_t* content, const uint8_t* rest, __nv_bfloat16* row, int warp,
                                            int lane) {
  using G = QGeom<BC, GC, BR, GR>;
  if (warp < 8)
    mean_of_tokens<BC, kDc, GC, kShared ? At::kSwizzled : At::kGlobal>(content, rest + (G::kOffCM - G::kOffRC), warp, row,
                                                                      lane);
  else
    mean_of_tokens<BR, kDr, GR, kShared ? At::kShared : At::kGlobal>(rest, rest + (G::kOffRM - G::kOffRC), 0, row + kDc,
                                                                    lane);
}

// Few pages (a decode step): one CTA for each that may be complete.
template <int BC, int GC, int BR, int GR>
__global__ void __launch_bounds__(kDigestThreads) page_digest_kernel(const DigestArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int page = completed_page(a, blockIdx.y, blockIdx.x);
  if (page < 0) return;
  using G = QGeom<BC, GC, BR, GR>;
  const uint8_t* pg = a.pool + static_cast<size_t>(page) * G::kPageBytes;
  digest_warp<BC, GC, BR, GR, false>(pg + G::kOffCC, pg + G::kOffRC, a.digests + static_cast<size_t>(page) * kDqk,
                                     threadIdx.x >> 5, threadIdx.x & 31);
}

// Many pages (after a prefill): CTAs walk the pages, one warp looking up 32 of
// them at a time and copying each whole into a ring, nine warps summing from
// there. The content codes come as TMA boxes in the 128-byte swizzle: a warp's
// fragment takes 32 bytes from each of four tokens, whose rows would otherwise
// share their banks (or, read from global memory directly, take four lines a load).
// Bound: latency. 2,048 pages take 14.7 us, 1,810 of them 14.1 (pools in turn, so that
// none stays in L2), where bytes (14,592-24,832 read and 1,152 written a page) would take
// 6.8 and 6.0; with the profiler's counters issue slots are 29 % busy, the tensor pipe
// 31 %, memory at a third of its rate, and warps wait for their operands: each loads its
// page's words, then multiplies, and two CTAs an SM are 27 % of the warps. The copies alone
// take 8.6 us, the sums alone about 12.
constexpr int kRingPages = 4, kRingCtas = 2;
constexpr uint64_t kRingWaitNs = 2000000000ull;

template <int kContent, int kRest>
struct DigestRing {
  struct alignas(1024) Stage {
    uint8_t content[kContent], rest[kRest];
  } stages[kRingPages];
  uint64_t full[kRingPages], empty[kRingPages];
  int page[kRingPages];
  int abort;
};

template <int BC, int GC, int BR, int GR>
using RingOf = DigestRing<QGeom<BC, GC, BR, GR>::kOffRC, QGeom<BC, GC, BR, GR>::kPageBytes - QGeom<BC, GC, BR, GR>::kOffRC>;

template <int BC, int GC, int BR, int GR>
__global__ void __launch_bounds__(kDigestThreads + 32, kRingCtas) page_digest_ring_kernel(const DigestArgs a, const __grid_constant__ CUtensorMap codes, int per_request, int items) {
  using G = QGeom<BC, GC, BR, GR>;
  extern __shared__ uint8_t smem_raw[];
  auto& m = *reinterpret_cast<RingOf<BC, GC, BR, GR>*>(smem_raw + ((1024 - (ptx::smem_u32(smem_raw) & 1023)) & 1023));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kRingPages; ++s) {
      ptx::mbar_init(&m.full[s], 1);
      ptx::mbar_init(&m.empty[s], kDigestWarps);
    }
    m.abort = 0;
    ptx::fence_mbar_init_cluster();
  }
  __syncthreads();
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  volatile int* abort_flag = &m.abort;
  // A whole warp waits; one whose wait runs out flags it, and all warps leave.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, abort_flag, kRingWaitNs));
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) record_error(a.status, MLA_ERR_TIMEOUT);
    }
    return ok;
  };
  if (warp == kDigestWarps) {  // the copying warp
    int it = 0;
    bool ok = true;
    auto next_slot = [&] {  // free once the summing warps have left it
      const int s = it % kRingPages, round = it / kRingPages;
      ++it;
      ok = round == 0 || wait(&m.empty[s], (round - 1) & 1);
      return s;
    };
    for (int64_t i0 = blockIdx.x; ok && i0 < items; i0 += 32ll * gridDim.x) {
      const int64_t i = i0 + static_cast<int64_t>(lane) * gridDim.x;
      const int mine = i < items ? completed_page(a, static_cast<int>(i / per_request), static_cast<int>(i % per_request)) : -1;
      for (uint32_t left = __ballot_sync(0xffffffffu, mine >= 0); ok && left; left &= left - 1) {
        const int page = __shfl_sync(0xffffffffu, mine, __ffs(left) - 1);
        const int s = next_slot();
        if (ok && lane == 0) {
          m.page[s] = page;
          ptx::mbar_arrive_expect_tx(&m.full[s], G::kPageBytes);
#pragma unroll
          for (int x = 0; x < G::kRowC; x += 128)
            ptx::tma_load_3d(m.stages[s].content + x * kPage, &codes, x, 0, page, &m.full[s]);
          ptx::bulk_load(m.stages[s].rest, a.pool + static_cast<size_t>(page) * G::kPageBytes + G::kOffRC,
                         G::kPageBytes - G::kOffRC, &m.full[s]);
        }
      }
    }
    if (ok) {
      const int s = next_slot();
      if (ok && lane == 0) {
        m.page[s] = -1;  // the end
        ptx::mbar_arrive(&m.full[s]);
      }
    }
    if (!ok) ptx::linger();
    return;
  }
  for (int it = 0;; ++it) {
    const int s = it % kRingPages;
    if (!wait(&m.full[s], (it / kRingPages) & 1)) {
      ptx::linger();  // the copying warp may have left with copies in flight
      break;
    }
    const int page = m.page[s];
    if (page < 0) break;
    digest_warp<BC, GC, BR, GR, true>(m.stages[s].content, m.stages[s].rest, a.digests + static_cast<size_t>(page) * kDqk,
                                      warp, lane);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&m.empty[s]);
  }
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_read_t(const ReadLaunch& L, const ReadArgs& a) {
  // Rows a request can have: no more than the outputs, nor than its table row holds
  // and one (the first position behind the table row is flagged), however loose
  // max_rows is. They touch a page more than they fill where they start inside one.
  const int64_t rows = std::min({static_cast<int64_t>(L.max_rows), L.total_rows, static_cast<int64_t>(L.max_pages) * kPage + 1});
  const unsigned pages = static_cast<unsigned>((rows + 62) / kPage + 1);
  // Eight tokens a warp keep four in flight for longer (64 requests of up to 16,384
  // tokens: 97 us, at two a warp 114); with few CTAs the length of each one's chain
  // counts, and two a warp finish sooner (1,021 tokens: 2.0 us instead of 3.4; even
  // at 32,768 tokens).
  if (static_cast<int64_t>(pages) * L.B < 4 * L.sms)
    return launch_dependent(qcache_read_kernel<BC, GC, BR, GR, 2>, dim3(4 * pages, L.B), dim3(kReadThreads), 0, L.stream, a);
  return launch_dependent(qcache_read_kernel<BC, GC, BR, GR, 8>, dim3(pages, L.B), dim3(kReadThreads), 0, L.stream, a);
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_digest_t(const DigestLaunch& L, const DigestArgs& a) {
  // Pages an append can have completed: no more than its table row has and one (the
  // first behind the row is flagged), however loose n_new is.
  const int per_request = std::min(L.n_new / kPage, L.max_pages) + 1;
  const int64_t items = static_cast<int64_t>(per_request) * L.B;
  // A CTA a page is as fast up to about a thousand pages, four to an SM twice over (pools
  // in L2: 16 requests of 64 pages 7.8 us, the ring 8.1; 32: 16.9 and 14.1; two pages
  // of 128 requests: 2.5 and 3.0).
  if (items < 8 * L.sms || items > 0x7fffffff || L.num_pages < 1)
    return launch_dependent(page_digest_kernel<BC, GC, BR, GR>, dim3(per_request, L.B), dim3(kDigestThreads), 0, L.stream, a);
  auto kern = page_digest_ring_kernel<BC, GC, BR, GR>;
  constexpr int kSmem = sizeof(RingOf<BC, GC, BR, GR>) + 1024;
  static_assert(kRingCtas * (kSmem + 1024) <= 233472, "CTAs an SM");
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  using G = QGeom<BC, GC, BR, GR>;
  CUtensorMap codes;
  const cuuint64_t dims[3] = {G::kRowC, kPage, static_cast<cuuint64_t>(L.num_pages)}, strides[2] = {G::kRowC, G::kPageBytes};
  const cuuint32_t box[3] = {128, kPage, 1};
  if (!encode_swizzled(&codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, static_cast<const uint8_t*>(L.pool) + G::kOffCC, 3, dims, strides, box))
    return cudaErrorInvalidValue;
  return launch_dependent(kern, dim3(kRingCtas * L.sms), dim3(kDigestThreads + 32), kSmem, L.stream, a, codes, per_request,
                          static_cast<int>(items));
}

}  // namespace

cudaError_t launch_qcache_read(const ReadLaunch& L) {
  ReadArgs a{static_cast<const uint8_t*>(L.pool), L.table, L.start, L.cu_rows, static_cast<__nv_bfloat16*>(L.out_c),
             static_cast<__nv_bfloat16*>(L.out_kr), L.c_stride, L.kr_stride, L.total_rows, L.status,
             L.num_pages, L.max_pages, L.max_rows};
  MLA_FORMAT_DISPATCH(L, launch_read_t, L, a)
  return cudaErrorInvalidValue;
}

cudaError_t launch_page_digest(const DigestLaunch& L) {
  DigestArgs a{static_cast<const uint8_t*>(L.pool), L.table, L.lens_before, L.new_lens,
               static_cast<__nv_bfloat16*>(L.digests), L.status, L.num_pages, L.max_pages, L.n_new};
  MLA_FORMAT_DISPATCH(L, launch_digest_t, L, a)
  return cudaErrorInvalidValue;
}

}  // namespace mla
