// Reading the quantized cache back outside the attention: dequantized rows of a
// token range of every request, and the mean key of completed pages.
//
//   rows:    x_hat = bf16(u * s + z)
//   digest:  kbar_p = bf16( (1/64) sum_t (u_t s_t + z_t) ), fp32 sums
//
// u * s is exact in fp32 (at most 15 significant bits), so u * s + z is one
// rounding. Codes become floats by setting them into the low bits of 2^23, where
// they stand in the word, and subtracting it (both at full rate; the conversion
// instruction runs at a quarter of it); the step takes back the power of two
// that the place is worth. Additions and products are two values an instruction.
#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

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
  const int hi = static_cast<int>(min(first + count - idx * kPage, static_cast<int64_t>(kPage)));
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

constexpr int kDigestThreads = 256;

// Sums over tokens of one page part (64 rows of ROW bytes of codes, groups of G
// channels): a thread takes one 32-bit word's channels of every kSlices-th token.
template <int BITS, int ROW, int G>
struct TokenSums {
  static constexpr int kWords = ROW / 4, kCh = 32 / BITS, kGroups = kWords * kCh / G;
  static constexpr int kSlices = kDigestThreads / kWords, kTokens = kPage / kSlices;
  static constexpr int kParts = kWords < 32 ? kDigestThreads / 32 : kSlices;  // left after the sum within a warp
  static_assert(kSlices * kTokens == kPage && kTokens >= 1 && kGroups * G == kWords * kCh, "whole tokens and groups");
  uint32_t word[kTokens], meta[kTokens];

  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* metas, int tid) {
    const int c = tid % kWords, slice = tid / kWords;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(codes) + slice * kWords + c;
    const uint32_t* m = reinterpret_cast<const uint32_t*>(metas) + slice * kGroups + c * kCh / G;
#pragma unroll
    for (int e = 0; e < kTokens; ++e) {
      word[e] = __ldg(w + e * kSlices * kWords);
      meta[e] = __ldg(m + e * kSlices * kGroups);
    }
  }
  // out[part][channel]: the sums of kParts sets of tokens
  __device__ __forceinline__ void sum(float* out, int tid) {
    f32x2 acc[kCh / 2];
#pragma unroll
    for (int k = 0; k < kCh / 2; ++k) acc[k] = make2(0.0f, 0.0f);
    float zsum = 0.0f;
#pragma unroll
    for (int e = 0; e < kTokens; ++e) {
      const Steps<BITS> s(half_bits_to_float(meta[e]));
      zsum += half_bits_to_float(meta[e] >> 16);
#pragma unroll
      for (int k = 0; k < kCh / 2; ++k)  // 16 bits of codes at a time
        acc[k] = fma2(fields2<BITS>(word[e] >> (16 * (k / (8 / BITS))), 2 * k % (16 / BITS)), s.v[k % (8 / BITS)], acc[k]);
    }
    const int c = tid % kWords, part = kWords < 32 ? tid / 32 : tid / kWords;
#pragma unroll
    for (int k = 0; k < kCh / 2; ++k) {
      acc[k] = add2(acc[k], both(zsum));
#pragma unroll
      for (int o = kWords; o < 32; o <<= 1) acc[k] = add2(acc[k], __shfl_xor_sync(0xffffffffu, acc[k], o));
      if (kWords >= 32 || tid % 32 < kWords)
        *reinterpret_cast<float2*>(out + part * (kWords * kCh) + c * kCh + 2 * k) = split2(acc[k]);
    }
  }
};

// One CTA a completed page. Bound: bytes (14,592-24,832 read, 1,152 written a page).
template <int BC, int GC, int BR, int GR>
__global__ void __launch_bounds__(kDigestThreads) page_digest_kernel(const DigestArgs a) {
  using G = QGeom<BC, GC, BR, GR>;
  using SumC = TokenSums<BC, G::kRowC, GC>;
  using SumR = TokenSums<BR, G::kRowR, GR>;
  __shared__ __align__(16) float part_c[SumC::kParts * kDc];
  __shared__ __align__(16) float part_r[SumR::kParts * kDr];
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int before = __ldg(a.lens_before + b);
  const int n = a.new_lens ? __ldg(a.new_lens + b) : a.n_new;
  if (before < 0 || n < 0 || n > a.n_new || static_cast<int64_t>(before) + n > 0x7fffffff) {
    if (blockIdx.x == 0 && tid == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const int p = before / kPage + static_cast<int>(blockIdx.x);
  if (p >= (before + n) / kPage) return;
  const int page = lookup_page(a.table, a.max_pages, a.num_pages, b, p * kPage);
  if (page < 0) {
    if (tid == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const uint8_t* pg = a.pool + static_cast<size_t>(page) * G::kPageBytes;
  SumC content;
  SumR rope;
  content.load(pg + G::kOffCC, pg + G::kOffCM, tid);
  rope.load(pg + G::kOffRC, pg + G::kOffRM, tid);
  content.sum(part_c, tid);
  rope.sum(part_r, tid);
  __syncthreads();
  __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(a.digests + static_cast<size_t>(page) * kDqk);
  for (int j = tid; j < kDqk / 2; j += kDigestThreads) {
    const bool in_c = j < kDc / 2;
    const float* part = in_c ? part_c + 2 * j : part_r + 2 * j - kDc;
    const int parts = in_c ? SumC::kParts : SumR::kParts, stride = in_c ? kDc : kDr;
    float x = 0.0f, y = 0.0f;
#pragma unroll 4
    for (int s = 0; s < parts; ++s) {
      const float2 v = *reinterpret_cast<const float2*>(part + s * stride);
      x += v.x;
      y += v.y;
    }
    dst[j] = __floats2bfloat162_rn(x * (1.0f / kPage), y * (1.0f / kPage));
  }
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_read_t(const ReadLaunch& L, const ReadArgs& a) {
  // Eight tokens a warp keep four in flight for longer (ragged read of 64 requests:
  // 118 us, at two a warp 130); with few CTAs the length of each one's chain counts,
  // and two a warp finish sooner (1,021 tokens: 2.5 us instead of 4.1).
  const unsigned pages = (L.max_rows + 62) / kPage + 1;
  if (static_cast<int64_t>(pages) * L.B < 4 * 148)
    return launch_dependent(qcache_read_kernel<BC, GC, BR, GR, 2>, dim3(4 * pages, L.B), dim3(kReadThreads), 0, L.stream, a);
  return launch_dependent(qcache_read_kernel<BC, GC, BR, GR, 8>, dim3(pages, L.B), dim3(kReadThreads), 0, L.stream, a);
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_digest_t(const DigestLaunch& L, const DigestArgs& a) {
  return launch_dependent(page_digest_kernel<BC, GC, BR, GR>, dim3(L.n_new / kPage + 1, L.B),
                          dim3(kDigestThreads), 0, L.stream, a);
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
