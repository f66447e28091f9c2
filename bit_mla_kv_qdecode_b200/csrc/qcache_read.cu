// Reading the quantized cache back outside the attention: dequantized rows of a
// token range of every request, and the mean key of completed pages.
//
//   rows:    x_hat = bf16(u * s + z)
//   digest:  kbar_p = bf16( (1/64) sum_t (u_t s_t + z_t) ), fp32 sums
//
// u * s is exact in fp32 (at most 15 significant bits), so u * s + z is one rounding.
#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

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

template <int BC, int GC, int BR, int GR>
__global__ void __launch_bounds__(256) qcache_read_kernel(const ReadArgs a) {
  using G = QGeom<BC, GC, BR, GR>;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, b = blockIdx.y;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int r0 = __ldg(a.cu_rows + b), r1 = __ldg(a.cu_rows + b + 1);
  const int64_t count = static_cast<int64_t>(r1) - r0;
  if (i == 0 && lane == 0 && (count < 0 || count > a.max_rows || r0 < 0 || r1 > a.total_rows))
    record_error(a.status, MLA_ERR_INVALID_ARG);
  if (i >= count || i >= a.max_rows) return;
  const int64_t row = static_cast<int64_t>(r0) + i;
  if (row < 0 || row >= a.total_rows) return;
  const int64_t t = (a.start ? __ldg(a.start + b) : 0) + static_cast<int64_t>(i);
  const int page = t >= 0 && t <= 0x7fffffff ? lookup_page(a.table, a.max_pages, a.num_pages, b, static_cast<int>(t)) : -1;
  if (page < 0) {
    if (lane == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const uint8_t* pg = a.pool + static_cast<size_t>(page) * G::kPageBytes;
  const int slot = static_cast<int>(t) % kPage;
  if (a.out_c) {
    uint32_t code[2] = {0u, 0u};
    const uint8_t* crow = pg + G::kOffCC + slot * G::kRowC;
    if constexpr (BC == 4) {
      const uint2 v = reinterpret_cast<const uint2*>(crow)[lane];
      code[0] = v.x;
      code[1] = v.y;
    } else {
      code[0] = reinterpret_cast<const uint32_t*>(crow)[lane];
    }
    const uint32_t m = reinterpret_cast<const uint32_t*>(pg + G::kOffCM + slot * G::kGroupsC * 4)[lane * 16 / GC];
    const float s = half_bits_to_float(m), z = half_bits_to_float(m >> 16);
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float v[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int bit = (2 * k + e) * BC;
        v[e] = fmaf(static_cast<float>((code[bit >> 5] >> (bit & 31)) & ((1u << BC) - 1)), s, z);
      }
      o[k] = pack_bf16(v[0], v[1]);
    }
    uint4* d = reinterpret_cast<uint4*>(a.out_c + row * a.c_stride) + 2 * lane;
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  if (a.out_kr) {
    const uint8_t* rrow = pg + G::kOffRC + slot * G::kRowR;
    const uint32_t code = BR == 4 ? rrow[lane] : (rrow[lane >> 1] >> (4 * (lane & 1)));
    const uint32_t m = reinterpret_cast<const uint32_t*>(pg + G::kOffRM + slot * G::kGroupsR * 4)[lane * 2 / GR];
    const float s = half_bits_to_float(m), z = half_bits_to_float(m >> 16);
    constexpr uint32_t kMask = (1u << BR) - 1;
    reinterpret_cast<uint32_t*>(a.out_kr + row * a.kr_stride)[lane] =
        pack_bf16(fmaf(static_cast<float>(code & kMask), s, z), fmaf(static_cast<float>((code >> BR) & kMask), s, z));
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

template <int BC, int GC, int BR, int GR>
__global__ void __launch_bounds__(kDqk) page_digest_kernel(const DigestArgs a) {
  using G = QGeom<BC, GC, BR, GR>;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int b = blockIdx.y, j = threadIdx.x;
  const int before = __ldg(a.lens_before + b);
  int n = a.new_lens ? __ldg(a.new_lens + b) : a.n_new;
  if (before < 0 || n < 0 || n > a.n_new || static_cast<int64_t>(before) + n > 0x7fffffff) {
    if (blockIdx.x == 0 && j == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const int p = before / kPage + static_cast<int>(blockIdx.x);
  if (p >= (before + n) / kPage) return;
  const int page = lookup_page(a.table, a.max_pages, a.num_pages, b, p * kPage);
  if (page < 0) {
    if (j == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const uint8_t* pg = a.pool + static_cast<size_t>(page) * G::kPageBytes;
  const bool content = j < kDc;
  const int ch = content ? j : j - kDc;
  const int bits = content ? BC : BR, row = content ? G::kRowC : G::kRowR;
  const uint8_t* codes = pg + (content ? G::kOffCC : G::kOffRC) + ch * bits / 8;
  const int shift = ch * bits % 8;
  const int groups = content ? G::kGroupsC : G::kGroupsR;
  const uint32_t* meta = reinterpret_cast<const uint32_t*>(pg + (content ? G::kOffCM : G::kOffRM)) + ch / (content ? GC : GR);
  float sum = 0.0f;
  for (int t = 0; t < kPage; ++t) {
    const uint32_t u = (codes[t * row] >> shift) & ((1u << bits) - 1), m = meta[t * groups];
    sum += fmaf(static_cast<float>(u), half_bits_to_float(m), half_bits_to_float(m >> 16));
  }
  a.digests[static_cast<size_t>(page) * kDqk + j] = __float2bfloat16_rn(sum * (1.0f / kPage));
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_read_t(const ReadLaunch& L, const ReadArgs& a) {
  return launch_dependent(qcache_read_kernel<BC, GC, BR, GR>, dim3((L.max_rows + 7) / 8, L.B), dim3(256), 0, L.stream, a);
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_digest_t(const DigestLaunch& L, const DigestArgs& a) {
  return launch_dependent(page_digest_kernel<BC, GC, BR, GR>, dim3(L.n_new / kPage + 1, L.B), dim3(kDqk), 0, L.stream, a);
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
