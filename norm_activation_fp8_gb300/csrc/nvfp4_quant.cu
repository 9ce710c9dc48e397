// nvfp4_quant.cu -- rows of bf16 to NVFP4, and NVFP4 back to bf16.
//
//   sf = e4m3(gs amax / 6), amax over a block of 16 columns of |x|
//   q  = e2m1(x gs / decode(sf)); +0 where sf is 0
//   back: bf16(e2m1 value * (decode(sf) / gs))
//
// Both directions are elementwise but for a block's maximum, so a tensor is one
// run of blocks (32 bytes of bf16, eight of codes, a lane each) or, on the way
// back, of half blocks.  Every code is the one that the exact value rounds to:
// the fp32 values decide where they are far enough from a border, which a
// second conversion tells, and exact remainders where they are not.
#include "common.cuh"
#include "launch.h"
#include "nvfp4.cuh"

namespace vg {

// Status word of this translation unit's kernels (kErrBounds in debug builds).
__device__ uint32_t g_nvfp4_status;

namespace {

constexpr int kThreads = 256;
constexpr int kChunks = 4;  // read back: chunks of 8 columns a thread

[[maybe_unused]] __device__ __forceinline__ uint64_t codes_extent(const Nvfp4Args &a) { return VG_ROWS(a.T) * (uint64_t)a.nch * 4; }
[[maybe_unused]] __device__ __forceinline__ uint64_t scales_extent(const Nvfp4Args &a) { return VG_ROWS(a.T) * (uint64_t)a.nch / 2; }

// 32 bytes, read once: one load (32-byte aligned), or two.
template <bool WIDE>
__device__ __forceinline__ void ld_block(const uint16_t *p, uint32_t (&w)[8]) {
  if constexpr (WIDE) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = ld_ro16(p), b = ld_ro16(p + 8);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}

// Which of two neighbouring codes X = gs v rounds to on a grid that is `unit`
// times as wide: gs v = p + e exactly, mid (the codes' midpoint) times unit is
// exact (few bits), and so is its difference from a p that near.
__device__ __forceinline__ bool above_midpoint(float v, float gs, float p, float mid, float unit, uint32_t lo) {
  const float e = fmaf(v, gs, -p), diff = p - mid * unit;  // |e| is at most half an ulp of p
  const float s = diff != 0.f ? diff : e;
  return s > 0.f || (s == 0.f && (lo & 1u));  // a tie: the even code
}

// Settles the codes of eight columns where the two words of codes differ: scaled
// quotients next to a midpoint.  (A call: it keeps the rest's registers free,
// and a tensor's scale of 6 * 448 over its largest magnitude makes quotients
// of bf16 numbers that lie on a midpoint or a rounding beside it common.)
__device__ __noinline__ uint32_t settle(uint32_t lo, uint32_t hi, uint32_t w0, uint32_t w1, uint32_t w2,
                                        uint32_t w3, float gs, float d) {
  uint32_t diff = lo ^ hi;
  while (diff) {
    const int i = (__ffs((int)diff) - 1) >> 2;
    const uint32_t w = i < 4 ? (i < 2 ? w0 : w1) : (i < 6 ? w2 : w3);
    const float v = fabsf(i & 1 ? bf16_hi(w) : bf16_lo(w));
    const uint32_t c = (lo >> (4 * i)) & 7u;  // the lower code: its midpoint with the next
    const float mid = c < 4 ? 0.5f * (float)c + 0.25f : (c < 6 ? (float)c - 1.5f : 5.0f);
    if (above_midpoint(v, gs, v * gs, mid, d, c)) lo += 1u << (4 * i);
    diff &= ~(15u << (4 * i));
  }
  return lo;
}

// A lane a block, kBlocks blocks a thread.  FLAT: the rows follow one another
// without a gap.
template <bool FLAT, bool WIDE, int kBlocks>
__global__ void __launch_bounds__(kThreads) nvfp4_quantize_kernel(const Nvfp4Args a) {
  const int64_t blocks = a.nch / 2, total = a.T * blocks, first = (int64_t)blockIdx.x * (kThreads * kBlocks);
  if (FLAT && threadIdx.x == 0 && blockIdx.x < (unsigned)a.pf_ctas) {
    const int64_t n = total - first < kThreads * kBlocks ? total - first : kThreads * kBlocks;
    prefetch_l2(a.x + first * kNvfp4Block, (uint32_t)n * 32u);
  }
  pdl_wait();
  const float gs = ld_ro_f32(a.global_scale);
  uint32_t w[kBlocks][8];
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    int64_t at = i * kNvfp4Block;
    if (!FLAT) {
      const int64_t row = total < (1ll << 32) ? (int64_t)((uint32_t)i / (uint32_t)blocks) : i / blocks;
      at = row * a.stride + (i - row * blocks) * kNvfp4Block;
    }
    if (i < total) ld_block<WIDE>(a.x + at, w[k]);
    else
      for (int j = 0; j < 8; ++j) w[k][j] = 0;
  }
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < kBlocks; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmax3(m, fabsf(bf16_lo(w[k][j])), fabsf(bf16_hi(w[k][j])));
    // p / 6 to 2^-22: where the two conversions agree, so does the exact value's
    const float p = m * gs, x = p * (1.0f / kE2M1Max);
    const uint32_t cc = cvt_e4m3x2(x * (1.0f - 0x1p-21f), x * (1.0f + 0x1p-21f));
    uint32_t code = cc & 0xFFu;
    if (code != cc >> 8) {
      const float mid = 0.5f * (e4m3_value(code) + e4m3_value(cc >> 8));
      if (above_midpoint(m, gs, p, mid, kE2M1Max, code)) code = cc >> 8;
    }
    const float d = e4m3_value(code), r = code ? __frcp_rn(d) : 0.f;
    const float2 g2 = make_float2(gs, gs);
    const float dn = r * (1.0f - 0x1p-20f), up = r * (1.0f + 0x1p-20f);
    uint32_t q[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // (y gs) / d to 2^-21, the same way
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = f2_mul(bf16x2_to_f2(w[k][4 * h + j]), g2);
        const float2 l = f2_mul(y, make_float2(dn, dn)), u = f2_mul(y, make_float2(up, up));
        lo[2 * j] = l.x, lo[2 * j + 1] = l.y, hi[2 * j] = u.x, hi[2 * j + 1] = u.y;
      }
      const uint32_t cl = quant_e2m1x8(lo), ch = quant_e2m1x8(hi);
      q[h] = cl == ch ? cl
                      : settle(cl, ch, w[k][4 * h], w[k][4 * h + 1], w[k][4 * h + 2], w[k][4 * h + 3], gs, d);
      if (code == 0) q[h] = 0;
    }
    if (i < total) {
      if (VG_ACCESS_OK(g_nvfp4_status, a.q + i * 8, 8, a.q, codes_extent(a)))
        st_stream(a.q + i * 8, make_uint2(q[0], q[1]));
      if (VG_ACCESS_OK(g_nvfp4_status, a.sf + i, 1, a.sf, scales_extent(a))) a.sf[i] = (uint8_t)code;
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
  const int64_t total = a.T * a.nch, first = (int64_t)blockIdx.x * (kThreads * kChunks);
  pdl_wait();
  const float gs = ld_ro_f32(a.global_scale), inv = __frcp_rn(gs);
  const bool far = !(gs > 0x1p-100f && gs < 0x1p100f);
  uint32_t c[kChunks], s[kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    c[k] = i < total ? ld_ro4(a.q + 4 * i) : 0u;
    s[k] = i < total ? ld_ro1(a.sf + (i >> 1)) : 0u;
  }
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int64_t i = first + k * kThreads + threadIdx.x;
    // decode(sf) / gs, correctly rounded: Markstein's correction of the product
    // with the correctly rounded reciprocal, by its exact remainder (nothing
    // under- or overflows unless gs is `far`; checked for every pair of
    // significands).  The division itself takes its slow way for a zero scale.
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

namespace {

template <int kBlocks>
cudaError_t launch_quantize(const Nvfp4Args &a, cudaStream_t s) {
  const dim3 g((unsigned)((a.T * (a.nch / 2) + kThreads * kBlocks - 1) / (kThreads * kBlocks))), b(kThreads);
  const bool flat = a.stride == a.nch * kElemsPerChunk || a.T == 1;
  const bool wide = reinterpret_cast<uintptr_t>(a.x) % 32 == 0 && (flat || a.stride % 16 == 0);
  return flat ? (wide ? launch_pdl(nvfp4_quantize_kernel<true, true, kBlocks>, g, b, 0, s, a)
                      : launch_pdl(nvfp4_quantize_kernel<true, false, kBlocks>, g, b, 0, s, a))
              : (wide ? launch_pdl(nvfp4_quantize_kernel<false, true, kBlocks>, g, b, 0, s, a)
                      : launch_pdl(nvfp4_quantize_kernel<false, false, kBlocks>, g, b, 0, s, a));
}

}  // namespace

// Few blocks: one a thread; many: four, whose loads are on their way together.
// One and four, in a run of calls, in us: 33 x 8192 1.7, 3.1; 1024 x 4096 3.3, 3.9;
// 2048 x 4096 5.8, 6.7; 4096 x 4096 9.3, 9.9; 6000 x 4096 11.9, 11.7 (rows apart
// 13.5, 14.4); 8192 x 4096 16.7, 16.2 (8191 rows, apart 19.3, 20.1); 10000 x 4096
// apart 21.0, 20.8; 16384 x 4096 30.4, 27.4 (apart 36.7, 36.0).
cudaError_t launch_nvfp4_quantize(const Nvfp4Args &a, cudaStream_t s) {
  return a.T * a.nch < 1 << 22 ? launch_quantize<1>(a, s) : launch_quantize<4>(a, s);
}

cudaError_t launch_nvfp4_dequantize(const Nvfp4Args &a, cudaStream_t s) {
  const dim3 g((unsigned)((a.T * a.nch + kThreads * kChunks - 1) / (kThreads * kChunks))), b(kThreads);
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
