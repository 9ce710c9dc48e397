// nvfp4_quant.cu -- rows of bf16 to NVFP4, and NVFP4 back to bf16.
//
//   sf = e4m3(gs amax / 6), amax over a block of 16 columns of |x|
//   q  = e2m1(x gs / decode(sf)); +0 where sf is 0
//   back: bf16(e2m1 value * (decode(sf) / gs))
//
// Both directions are elementwise but for a block's maximum, so the tensor is
// one run of chunks of eight columns (16 bytes of bf16, four of codes): a lane
// takes a chunk, two neighbouring lanes a block.  Every code is the one that
// the exact value rounds to, at next to no cost: the fp32 values decide where
// they are far enough from a border, which a second conversion tells, and
// exact remainders where they are not.
#include "common.cuh"
#include "launch.h"
#include "nvfp4.cuh"

namespace vg {

// Status word of this translation unit's kernels (kErrBounds in debug builds).
__device__ uint32_t g_nvfp4_status;

namespace {

constexpr int kThreads = 256, kPer = 4;  // chunks a thread

__device__ __forceinline__ uint64_t codes_extent(const Nvfp4Args &a) { return VG_ROWS(a.T) * (uint64_t)a.nch * 4; }
__device__ __forceinline__ uint64_t scales_extent(const Nvfp4Args &a) { return VG_ROWS(a.T) * (uint64_t)a.nch / 2; }

__device__ __forceinline__ float e2m1_level(uint32_t c) {  // of a code without its sign
  return c < 4 ? 0.5f * (float)c : (c < 6 ? (float)(c - 2) : (float)(2 * c - 8));
}

// The code of y gs / d where the fp32 quotient lies next to a midpoint m of
// two levels: y gs = p + e exactly, m d is exact (three times four bits), and
// so is its difference from a p that near.
__device__ __noinline__ uint32_t e2m1_exact(float y, float gs, float d) {
  const float a = fabsf(y), p = a * gs, e = fmaf(a, gs, -p), v = p * __frcp_rn(d);
  const float two[8] = {v * (1.0f - 0x1p-20f), v * (1.0f + 0x1p-20f)};
  const uint32_t cc = quant_e2m1x8(two), lo = cc & 7u, hi = (cc >> 4) & 7u;
  uint32_t c = lo;
  if (lo != hi) {
    const float diff = p - 0.5f * (e2m1_level(lo) + e2m1_level(hi)) * d;
    const float s = diff != 0.f ? diff : e;  // |e| is at most half an ulp of p
    c = s > 0.f || (s == 0.f && (lo & 1u)) ? hi : lo;
  }
  return c | (__float_as_uint(y) >> 31 << 3);
}
__device__ __noinline__ uint32_t e2m1x8_exact(uint4 x, float gs, float d) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r = 0;
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    r |= e2m1_exact(i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]), gs, d) << (4 * i);
  return r;
}

// FLAT: the rows follow one another without a gap.
template <bool FLAT>
__global__ void __launch_bounds__(kThreads) nvfp4_quantize_kernel(const Nvfp4Args a) {
  const int64_t total = a.T * a.nch, first = (int64_t)blockIdx.x * (kThreads * kPer);
  if (FLAT && threadIdx.x == 0 && blockIdx.x < (unsigned)a.pf_ctas) {
    const int64_t n = total - first < kThreads * kPer ? total - first : kThreads * kPer;
    prefetch_l2(a.x + first * kElemsPerChunk, (uint32_t)n * 16u);
  }
  pdl_wait();
  const float gs = __ldg(a.global_scale);
  uint4 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    int64_t at = i * kElemsPerChunk;
    if (!FLAT) {
      const int64_t row = total < (1ll << 32) ? (int64_t)((uint32_t)i / (uint32_t)a.nch) : i / a.nch;
      at = row * a.stride + (i - row * a.nch) * kElemsPerChunk;
    }
    v[k] = i < total ? ld_stream_ro(a.x + at) : make_uint4(0, 0, 0, 0);
  }
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
    float2 y[4];
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y[j] = bf16x2_to_f2(w[j]);
      m = fmax3(m, fabsf(y[j].x), fabsf(y[j].y));
    }
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const float p = m * gs;
    const uint32_t code = e4m3_code_settled(p * (1.0f / kE2M1Max), [&] {
      const float e = fmaf(m, gs, -p), xh = __fdiv_rn(p, kE2M1Max);
      const float xl = __fdiv_rn(fmaf(-xh, kE2M1Max, p) + e, kE2M1Max);
      const float x = xh + xl;
      return e4m3_code_df(x, xl - (x - xh));
    });
    const float d = e4m3_value(code), r = code ? __frcp_rn(d) : 0.f;
    const float2 g2 = make_float2(gs, gs), r2 = make_float2(r, r);
    const float2 dn = make_float2(1.0f - 0x1p-21f, 1.0f - 0x1p-21f);
    const float2 up = make_float2(1.0f + 0x1p-21f, 1.0f + 0x1p-21f);
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 q = f2_mul(f2_mul(y[j], g2), r2), l = f2_mul(q, dn), h = f2_mul(q, up);
      lo[2 * j] = l.x, lo[2 * j + 1] = l.y, hi[2 * j] = h.x, hi[2 * j + 1] = h.y;
    }
    uint32_t codes = quant_e2m1x8(lo);
    if (codes != quant_e2m1x8(hi)) codes = e2m1x8_exact(v[k], gs, d);
    if (code == 0) codes = 0;
    if (i < total) {
      if (VG_ACCESS_OK(g_nvfp4_status, a.q + i * 4, 4, a.q, codes_extent(a))) st_stream(a.q + i * 4, codes);
      uint8_t *s = a.sf + (i >> 1);
      if (!(i & 1) && VG_ACCESS_OK(g_nvfp4_status, s, 1, a.sf, scales_extent(a))) *s = (uint8_t)code;
    }
  }
}

// Two codes of a byte as two fp32 values.
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte) {
  float2 r;
  asm("{\n\t.reg .b8 b;\n\t.reg .b32 h2;\n\t.reg .b16 lo, hi;\n\t"
      "cvt.u8.u32 b, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 h2, b;\n\t"
      "mov.b32 {lo, hi}, h2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(byte));
  return r;
}

__global__ void __launch_bounds__(kThreads) nvfp4_dequantize_kernel(const Nvfp4Args a) {
  const int64_t total = a.T * a.nch, first = (int64_t)blockIdx.x * (kThreads * kPer);
  pdl_wait();
  const float gs = __ldg(a.global_scale), inv = __frcp_rn(gs);
  const bool far = !(gs > 0x1p-100f && gs < 0x1p100f);
  uint32_t c[kPer], s[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    c[k] = i < total ? __ldg(reinterpret_cast<const uint32_t *>(a.q) + i) : 0u;
    s[k] = i < total ? __ldg(a.sf + (i >> 1)) : 0u;
  }
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    // decode(sf) / gs, correctly rounded: one step from the reciprocal (the
    // division itself takes its slow way for a zero scale)
    const float d = e4m3_value(s[k]), q = d * inv;
    const float r = far ? __fdiv_rn(d, gs) : fmaf(fmaf(-q, gs, d), inv, q);
    const float2 r2 = make_float2(r, r);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = f2_mul(e2m1x2_values((c[k] >> (8 * j)) & 0xFFu), r2);
      o[j] = pack_bf16x2_rn(x.x, x.y);
    }
    uint16_t *p = a.out + i * kElemsPerChunk;
    if (i < total && VG_ACCESS_OK(g_nvfp4_status, p, 16, a.out, VG_ROWS(a.T) * (uint64_t)a.nch * 16))
      st_stream(p, make_uint4(o[0], o[1], o[2], o[3]));
  }
}

}  // namespace

cudaError_t launch_nvfp4_quantize(const Nvfp4Args &a, cudaStream_t s) {
  const dim3 g((unsigned)((a.T * a.nch + kThreads * kPer - 1) / (kThreads * kPer))), b(kThreads);
  return a.stride == a.nch * kElemsPerChunk ? launch_pdl(nvfp4_quantize_kernel<true>, g, b, 0, s, a)
                                            : launch_pdl(nvfp4_quantize_kernel<false>, g, b, 0, s, a);
}

cudaError_t launch_nvfp4_dequantize(const Nvfp4Args &a, cudaStream_t s) {
  const dim3 g((unsigned)((a.T * a.nch + kThreads * kPer - 1) / (kThreads * kPer))), b(kThreads);
  return launch_pdl(nvfp4_dequantize_kernel, g, b, 0, s, a);
}

uint32_t read_nvfp4_status(bool reset) {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_nvfp4_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (reset) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_nvfp4_status, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  }
  return v;
}

}  // namespace vg
