// Append straight from the projections: RMS norm of the latent, rotation of the
// RoPE key and of every head's RoPE query, quantize + pack + paged write, in
// one launch.
//
//   c  = bf16( x * (1 / sqrt(sum x^2 / 512 + eps)) * w ),   x the latent, 512 wide
//   k  = bf16( rotate(kr, angle(position)) ),  q' = bf16( rotate(q, angle(position)) )
//   rotate: (a, b) -> (a cos - b sin, a sin + b cos) on each rotary pair
// then the cache's quantizer on c and k (append_token.cuh).
//
// The norm and the key's rotation are computed in fp64 and rounded to fp32 and
// then bf16: c and k sit in front of the quantizer, where a last-bit difference
// moves a value across a code's border, and the cache's codes are reproducible
// bit for bit. The squares of bf16 values and the products of a bf16 value with
// an fp32 cosine are exact in fp64, so the order of the sum does not matter in
// practice. The queries meet no border and are rotated in fp32.
//
// Bound: bytes. A token reads 1,152 B and writes its 228-388 B slot (and 1,152 B
// of rows when asked); its queries read and write 128 B a head each. 8,192 tokens
// of 128 heads, 7,381 of them given: 43.2 us, 6.0 TB/s (45.4 with a division a
// code; 50.6 with the tokens' blocks ahead of the queries' instead of among them,
// 52.5 with 16 heads a warp instead of 32). A step of 32 tokens is latency, 3.6 us.
#include "append_token.cuh"
#include "mla_common.cuh"
#include "mla_internal.h"
#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerWarp = 32;  // heads of one token that a warp rotates

struct NormRopeArgs {
  uint8_t* pool;
  const int32_t* table;
  const int32_t* lens_before;
  const int32_t* new_lens;
  const __nv_bfloat16* kv;
  int64_t kv_stride;
  const __nv_bfloat16* weight;
  const __nv_bfloat16* q;
  int64_t q_token_stride, q_head_stride;
  __nv_bfloat16* q_out;
  const float* cos_sin;
  const int32_t* positions;
  __nv_bfloat16* rows_out;
  int* status;
  double eps;
  int num_pages, max_pages, max_positions, n_tokens, n_new, H, head_chunks, token_blocks, period;
};

// Position whose angle token `tok` (token j of request b) is turned by, or -1
// when it is past the table of angles.
__device__ __forceinline__ int angle_position(const NormRopeArgs& a, int tok, int b, int j) {
  const int p = a.positions ? __ldg(a.positions + tok) : __ldg(a.lens_before + b) + j;
  return p >= 0 && p < a.max_positions ? p : -1;
}

// Tokens given of request b, or -1 for a count out of range: such a request is
// skipped, and flagged by the warp of its first token.
__device__ __forceinline__ int tokens_given(const NormRopeArgs& a, int b) {
  const int n = a.new_lens ? __ldg(a.new_lens + b) : a.n_new;
  return n >= 0 && n <= a.n_new ? n : -1;
}

__device__ __forceinline__ float round_bf16(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// One warp: the token's latent and RoPE key into the cache.
template <int BC, int GC, int BR, int GR, bool kHalf>
__device__ __forceinline__ void token_warp(const NormRopeArgs& a, int tok, int lane) {
  using G = QGeom<BC, GC, BR, GR>;
  const int b = tok / a.n_new, j = tok - b * a.n_new;
  // the row and the weights are on their way while the length and the table are looked up
  const __nv_bfloat16* row = a.kv + static_cast<int64_t>(tok) * a.kv_stride;
  const uint4* src = reinterpret_cast<const uint4*>(row) + 2 * lane;
  const uint4 v0 = __ldg(src), v1 = __ldg(src + 1);
  const uint32_t rw = __ldg(reinterpret_cast<const uint32_t*>(row + kDc) + lane);
  const uint4* ws = reinterpret_cast<const uint4*>(a.weight) + 2 * lane;
  const uint4 ones = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  const uint4 g0 = a.weight ? __ldg(ws) : ones, g1 = a.weight ? __ldg(ws + 1) : ones;
  const int given = tokens_given(a, b);
  const int pos = angle_position(a, tok, b, j);
  const int t = __ldg(a.lens_before + b) + j;
  if (j >= given) {
    if (given < 0 && j == 0 && lane == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const int page = lookup_page(a.table, a.max_pages, a.num_pages, b, t);
  if (pos < 0 || page < 0) {
    if (lane == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = bf16_lo(w[k]);
    x[2 * k + 1] = bf16_hi(w[k]);
  }
  double part[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
  for (int k = 0; k < 16; ++k) part[k & 3] = fma(static_cast<double>(x[k]), static_cast<double>(x[k]), part[k & 3]);
  double ss = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double inv = rsqrt(ss / kDc + a.eps);
  const uint32_t g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    x[2 * k] = static_cast<float>(x[2 * k] * inv * static_cast<double>(bf16_lo(g[k])));
    x[2 * k + 1] = static_cast<float>(x[2 * k + 1] * inv * static_cast<double>(bf16_hi(g[k])));
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = round_bf16(x[k]);

  const float* cs = a.cos_sin + static_cast<int64_t>(pos) * kDr;
  const double e0 = bf16_lo(rw), e1 = bf16_hi(rw);
  float r0, r1;
  if constexpr (kHalf) {
    // channels 2l, 2l+1 pair with those of lane l ^ 16
    const uint32_t pw = __shfl_xor_sync(0xffffffffu, rw, 16);
    const double p0 = bf16_lo(pw), p1 = bf16_hi(pw);
    const int i = 2 * (lane & 15);
    const double c0 = __ldg(cs + i), c1 = __ldg(cs + i + 1);
    const double sgn = lane < 16 ? -1.0 : 1.0;
    const double s0 = sgn * __ldg(cs + 32 + i), s1 = sgn * __ldg(cs + 32 + i + 1);
    r0 = static_cast<float>(fma(e0, c0, p0 * s0));
    r1 = static_cast<float>(fma(e1, c1, p1 * s1));
  } else {
    const double c = __ldg(cs + lane), s = __ldg(cs + 32 + lane);
    r0 = static_cast<float>(fma(e0, c, -(e1 * s)));
    r1 = static_cast<float>(fma(e0, s, e1 * c));
  }
  r0 = round_bf16(r0);
  r1 = round_bf16(r1);
  uint8_t* pg = a.pool + static_cast<size_t>(page) * G::kPageBytes;
  if (a.rows_out) {
    quantize_values_warp<BC, GC, BR, GR, true, false>(pg, t % kPage, x, r0, r1, lane);
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = pack_bf16(x[2 * k], x[2 * k + 1]);
    __nv_bfloat16* dst = a.rows_out + static_cast<size_t>(tok) * kDqk;
    uint4* d = reinterpret_cast<uint4*>(dst) + 2 * lane;
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    reinterpret_cast<uint32_t*>(dst + kDc)[lane] = pack_bf16(r0, r1);
  } else {
    quantize_values_warp<BC, GC, BR, GR, false, false>(pg, t % kPage, x, r0, r1, lane);
  }
}

// One warp: up to 32 heads of one token's queries. Four lanes a head; lane i of
// the four turns rotary pairs [8i, 8i + 8), two 16-byte pieces in either order.
template <bool kHalf>
__device__ __forceinline__ void query_warp(const NormRopeArgs& a, int unit, int lane) {
  const int tok = unit / a.head_chunks, chunk = unit - tok * a.head_chunks;
  const int b = tok / a.n_new, j = tok - b * a.n_new;
  const int given = tokens_given(a, b);
  const int pos = angle_position(a, tok, b, j);
  if (j >= given) return;
  if (pos < 0) {
    if (lane == 0) record_error(a.status, MLA_ERR_INVALID_ARG);
    return;
  }
  const int i = lane & 3;
  const int ia = kHalf ? 8 * i : 16 * i, ib = kHalf ? 32 + 8 * i : 16 * i + 8;
  const __nv_bfloat16* src = a.q + static_cast<int64_t>(tok) * a.q_token_stride;
  __nv_bfloat16* dst = a.q_out + static_cast<int64_t>(tok) * a.H * kDr;
  uint4 va[kHeadsPerWarp / 8], vb[kHeadsPerWarp / 8];
#pragma unroll
  for (int r = 0; r < kHeadsPerWarp / 8; ++r) {
    const int h = chunk * kHeadsPerWarp + 8 * r + (lane >> 2);
    if (h < a.H) {
      va[r] = __ldcs(reinterpret_cast<const uint4*>(src + h * a.q_head_stride + ia));
      vb[r] = __ldcs(reinterpret_cast<const uint4*>(src + h * a.q_head_stride + ib));
    }
  }
  const float4* cs = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(pos) * kDr + 8 * i);
  const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1), s0 = __ldg(cs + 8), s1 = __ldg(cs + 9);
  const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
  const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
  for (int r = 0; r < kHeadsPerWarp / 8; ++r) {
    const int h = chunk * kHeadsPerWarp + 8 * r + (lane >> 2);
    if (h >= a.H) continue;
    const uint32_t wa[4] = {va[r].x, va[r].y, va[r].z, va[r].w}, wb[4] = {vb[r].x, vb[r].y, vb[r].z, vb[r].w};
    uint32_t oa[4], ob[4];
    if constexpr (kHalf) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = bf16_lo(wa[k]), x1 = bf16_hi(wa[k]), y0 = bf16_lo(wb[k]), y1 = bf16_hi(wb[k]);
        oa[k] = pack_bf16(fmaf(x0, c[2 * k], -(y0 * s[2 * k])), fmaf(x1, c[2 * k + 1], -(y1 * s[2 * k + 1])));
        ob[k] = pack_bf16(fmaf(x0, s[2 * k], y0 * c[2 * k]), fmaf(x1, s[2 * k + 1], y1 * c[2 * k + 1]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x0 = bf16_lo(wa[k]), y0 = bf16_hi(wa[k]), x1 = bf16_lo(wb[k]), y1 = bf16_hi(wb[k]);
        oa[k] = pack_bf16(fmaf(x0, c[k], -(y0 * s[k])), fmaf(x0, s[k], y0 * c[k]));
        ob[k] = pack_bf16(fmaf(x1, c[4 + k], -(y1 * s[4 + k])), fmaf(x1, s[4 + k], y1 * c[4 + k]));
      }
    }
    __nv_bfloat16* d = dst + static_cast<int64_t>(h) * kDr;
    *reinterpret_cast<uint4*>(d + ia) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    *reinterpret_cast<uint4*>(d + ib) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
  }
}

template <int BC, int GC, int BR, int GR, bool kHalf>
__global__ void __launch_bounds__(kThreads, 4) norm_rope_append_kernel(const NormRopeArgs a) {
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // every period-th block takes eight tokens, the others eight units of queries: the
  // tokens' long chains (look-up, fp64 norm, quantizer) run beside the queries' traffic
  const int t = blockIdx.x / a.period;
  if (blockIdx.x % a.period == 0 && t < a.token_blocks) {
    const int tok = t * kWarps + warp;
    if (tok < a.n_tokens) token_warp<BC, GC, BR, GR, kHalf>(a, tok, lane);
  } else {
    const int64_t unit = static_cast<int64_t>(blockIdx.x - min(t + 1, a.token_blocks)) * kWarps + warp;
    if (unit < static_cast<int64_t>(a.n_tokens) * a.head_chunks) query_warp<kHalf>(a, static_cast<int>(unit), lane);
  }
}

template <int BC, int GC, int BR, int GR>
cudaError_t launch_t(const NormRopeLaunch& L, const NormRopeArgs& a, unsigned blocks) {
  return L.half_pairs ? launch_dependent(norm_rope_append_kernel<BC, GC, BR, GR, true>, dim3(blocks), dim3(kThreads), 0,
                                         L.stream, a)
                      : launch_dependent(norm_rope_append_kernel<BC, GC, BR, GR, false>, dim3(blocks), dim3(kThreads),
                                         0, L.stream, a);
}

}  // namespace

cudaError_t launch_norm_rope_append(const NormRopeLaunch& L) {
  NormRopeArgs a{};
  a.pool = static_cast<uint8_t*>(L.pool);
  a.table = L.table;
  a.lens_before = L.lens_before;
  a.new_lens = L.new_lens;
  a.kv = static_cast<const __nv_bfloat16*>(L.kv);
  a.kv_stride = L.kv_stride;
  a.weight = static_cast<const __nv_bfloat16*>(L.norm_weight);
  a.q = static_cast<const __nv_bfloat16*>(L.q);
  a.q_token_stride = L.q_token_stride;
  a.q_head_stride = L.q_head_stride;
  a.q_out = static_cast<__nv_bfloat16*>(L.q_out);
  a.cos_sin = L.cos_sin;
  a.positions = L.positions;
  a.rows_out = static_cast<__nv_bfloat16*>(L.rows_out);
  a.status = L.status;
  a.eps = L.eps;
  a.num_pages = L.num_pages;
  a.max_pages = L.max_pages;
  a.max_positions = L.max_positions;
  a.n_tokens = L.B * L.n_new;
  a.n_new = L.n_new;
  a.H = L.H;
  a.head_chunks = (L.H + kHeadsPerWarp - 1) / kHeadsPerWarp;
  a.token_blocks = (a.n_tokens + kWarps - 1) / kWarps;
  const int64_t units = static_cast<int64_t>(a.n_tokens) * a.head_chunks;
  const unsigned blocks = static_cast<unsigned>(a.token_blocks + (units + kWarps - 1) / kWarps);
  a.period = static_cast<int>(blocks / a.token_blocks);
  MLA_FORMAT_DISPATCH(L, launch_t, L, a, blocks)
  return cudaErrorInvalidValue;
}

}  // namespace mla
