// fp8_gemm.cu -- FP8 matrix product with a scale per block of 128 columns, and
// the gated feed-forward projection on top of it.
//
//   c[t, n] = sum_b sa[t, b] sw[n / 128, b] sum_{k in block b} a[t, k] w[n, k]
//   plain:  out = bf16(c)
//   gated:  g = c[t, n], u = c[t, I + n], y = g / (1 + exp(-g)) u (fp32, never
//           rounded to bf16), s = max(amax |y| over 128 columns, 1e-10) / 448
//           (or the power of two above it), q = e4m3(y / s)
//
// A simple form on the fp32 units: a CTA computes 32 tokens by 128 columns
// (gated: of gate and of up), a warp 4 tokens, so that a warp holds a whole
// scale group.  A block's products are summed in fp32 and scaled into the
// running fp32 sum.
#include "common.cuh"
#include "dyn_scale.cuh"
#include "launch.h"

namespace vg {

// Status word of this translation unit's kernels.
__device__ uint32_t g_gemm_status;

namespace {

constexpr int kTok = 32, kCol = 128, kStep = 32;

__device__ __forceinline__ float2 e4m3x2_to_f2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  float2 f;
  asm("{.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// rows x 32 columns of codes from row0 on, as fp32, column by column in
// shared memory; rows beyond `limit` are zero.
template <int ROWS>
__device__ __forceinline__ void stage(float (&dst)[kStep][ROWS + 1], const uint8_t *src, int64_t row0,
                                      int64_t limit, int64_t ld, int k0) {
  for (int i = (int)threadIdx.x; i < ROWS * (kStep / 4); i += (int)blockDim.x) {
    const int r = i / (kStep / 4), c = i % (kStep / 4) * 4;
    uint32_t v = 0;
    if (row0 + r < limit) v = *reinterpret_cast<const uint32_t *>(src + (row0 + r) * ld + k0 + c);
    const float2 lo = e4m3x2_to_f2((uint16_t)v), hi = e4m3x2_to_f2((uint16_t)(v >> 16));
    dst[c][r] = lo.x;
    dst[c + 1][r] = lo.y;
    dst[c + 2][r] = hi.x;
    dst[c + 3][r] = hi.y;
  }
}

template <bool GATED>
__global__ void __launch_bounds__(256) fp8_gemm_simple_kernel(const GemmArgs a) {
  constexpr int H = GATED ? 2 : 1;
  __shared__ float sa[kStep][kTok + 1];
  __shared__ float sw[H][kStep][kCol + 1];
  const int tx = (int)threadIdx.x & 31, ty = (int)threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * kTok, n0 = (int64_t)blockIdx.y * kCol;
  pdl_wait();
  float acc[H][4][4] = {};
  const int kb = a.K / 128;
  for (int b = 0; b < kb; ++b) {
    float part[H][4][4] = {};
    for (int k0 = b * 128; k0 < b * 128 + 128; k0 += kStep) {
      __syncthreads();
      stage<kTok>(sa, a.a, t0, a.T, a.K, k0);
      for (int h = 0; h < H; ++h)
        stage<kCol>(sw[h], a.w, n0 + (int64_t)h * a.N, (int64_t)(h + 1) * a.N, a.K, k0);
      __syncthreads();
#pragma unroll 4
      for (int k = 0; k < kStep; ++k)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              part[h][i][j] = fmaf(sa[k][ty * 4 + i], sw[h][k][tx + 32 * j], part[h][i][j]);
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float ws = a.w_scale[((n0 + (int64_t)h * a.N) / 128) * kb + b];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + ty * 4 + i;
        const float s = t < a.T ? a.a_scale[t * a.a_ts + b * a.a_bs] * ws : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(part[h][i][j], s, acc[h][i][j]);
      }
    }
  }
  pdl_launch_dependents();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = t0 + ty * 4 + i;
    if (t >= a.T) continue;
    if constexpr (!GATED) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + tx + 32 * j;
        if (n < a.N) a.out[t * a.N + n] = (uint16_t)pack_bf16x2_rn(acc[0][i][j], 0.f);
      }
    } else {
      float y[4], m = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[j] = acc[0][i][j] / (1.0f + __expf(-acc[0][i][j])) * acc[1][i][j];
        m = fmaxf(m, fabsf(y[j]));
      }
      m = fmaxf(warp_max(m), kAmaxFloor);
      const float s = a.ue8m0 ? exp2i(pow2_exponent_448(m)) : m * kInv448;
      if (tx == 0) a.scale[t * a.s_ts + (n0 / 128) * a.s_gs] = s;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        a.q[t * a.N + n0 + tx + 32 * j] = (uint8_t)cvt_e4m3x2(y[j] / s, 0.f);
    }
  }
}

}  // namespace

cudaError_t launch_fp8_gemm(const GemmArgs &a, bool gated, int sms, cudaStream_t s) {
  (void)sms;
  const dim3 grid((unsigned)((a.T + kTok - 1) / kTok), (unsigned)((a.N + kCol - 1) / kCol));
  return gated ? launch_pdl(fp8_gemm_simple_kernel<true>, grid, dim3(256), 0, s, a)
               : launch_pdl(fp8_gemm_simple_kernel<false>, grid, dim3(256), 0, s, a);
}

uint32_t read_gemm_status(bool reset) {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_gemm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (reset) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_gemm_status, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  }
  return v;
}

}  // namespace vg
