// nvfp4_gemm.cu -- NVFP4 matrix product, and the gated feed-forward projection
// on top of it.
//
//   c[t, n] = alpha sum_k a[t, k] sa[t, k / 16] w[n, k] sw[n, k / 16]
//   plain:  out = bf16(c)
//   gated:  g = c[t, n], u = c[t, I + n], y = g / (1 + exp(-g)) u (fp32, never
//           rounded to bf16), sf = e4m3(gs amax / 6) per 16 columns, q = e2m1(y
//           gs / sf)
//
// The tensor cores apply the block scales themselves, so a sum over all of K
// stays in tensor memory.  They want the scales of 128 rows and one K of 64 as
// 32 lanes x 4 columns; the tensors hold them row by row, as the quantising
// ops write them.  Warps that have nothing else to do until the epilogue move
// them: a lane loads the 16 bytes (K of 256, a stage) of rows l, l + 32, ...
// and stores, for each K of 64, the four rows' words as one 16-byte row of the
// copy to tensor memory.
#include "dyn_scale.cuh"
#include "gemm_common.cuh"
#include "nvfp4.cuh"

namespace vg {

// Status word of this translation unit's kernels.
__device__ uint32_t g_fp4_gemm_status;

namespace {

constexpr int kStageK = 256;              // codes of K per stage: 128 bytes a row
constexpr int kChunks = kStageK / 64;     // products per stage
constexpr int kRowBytes = kStageK / 2;
constexpr int kRows = 128;                // rows of a stage's larger operand
constexpr int kAtom = 512;                // bytes of the scales of 128 rows and a K of 64

struct Fp4Maps {
  CUtensorMap a, w, out;
};

[[maybe_unused]] __device__ __forceinline__ uint64_t a_sf_extent(const Fp4GemmArgs &a) {
  return VG_ROWS(a.T) * (uint64_t)(a.K / kNvfp4Block);
}
template <bool GATED>
[[maybe_unused]] __device__ __forceinline__ uint64_t w_sf_extent(const Fp4GemmArgs &a) {
  return (GATED ? 2ull : 1ull) * (uint64_t)a.N * (uint64_t)(a.K / kNvfp4Block);
}

// The scales of one row and a stage's K: a word per K of 64, the first `chunks`
// of them; zeros for a row that is not there.  Rows whose length is no multiple
// of 256 are not 16-byte aligned.
__device__ __forceinline__ uint4 load_scales(const uint8_t *p, bool live, bool wide, int chunks,
                                             const uint8_t *base, uint64_t extent) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!live || !VG_ACCESS_OK(g_fp4_gemm_status, p, 4 * chunks, base, extent)) return v;
  if (wide) return __ldg(reinterpret_cast<const uint4 *>(p));
  const uint32_t *q = reinterpret_cast<const uint32_t *>(p);
  v.x = __ldg(q);
  if (chunks > 1) v.y = __ldg(q + 1);
  if (chunks > 2) v.z = __ldg(q + 2);
  if (chunks > 3) v.w = __ldg(q + 3);
  return v;
}

// Four rows' words as the copies to tensor memory read them: chunk c at c
// kAtom, this lane's 16 bytes.
__device__ __forceinline__ void store_scales(uint8_t *dst, int lane, const uint4 (&v)[4]) {
  uint4 *p = reinterpret_cast<uint4 *>(dst + 16 * lane);
  p[0 * kAtom / 16] = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
  p[1 * kAtom / 16] = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
  p[2 * kAtom / 16] = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
  p[3 * kAtom / 16] = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
}

// SiLU(g) u with the accurate exponential and division: an ulp or two, so that
// codes move only where the value is that near a border.
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdiv_rn(g, 1.0f + expf(-g)) * u; }

// A block's scale code, and the factor that y gs is multiplied by.
__device__ __forceinline__ uint32_t block_code(float amax, float gs, float &r) {
  const uint32_t code = e4m3_code(__fdiv_rn(amax * gs, kE2M1Max));
  r = code ? __frcp_rn(e4m3_value(code)) : 0.f;
  return code;
}

// Four columns of a token's output row, from n on (N is a multiple of 8).
__device__ __forceinline__ void store_out4(const Fp4GemmArgs &a, int64_t t, int n, const float4 &c) {
  uint16_t *o = a.out + t * a.N + n;
  if (n < a.N && VG_ACCESS_OK(g_fp4_gemm_status, o, 8, a.out, VG_ROWS(a.T) * 2ull * (uint64_t)a.N))
    *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2_rn(c.x, c.y), pack_bf16x2_rn(c.z, c.w));
}

// Activation and codes of four columns from n on, four lanes a block of 16.
__device__ __forceinline__ void store_gated4(const Fp4GemmArgs &a, int64_t t, bool live, int n, int lane,
                                             float gs, const float4 &g, const float4 &u) {
  const float y0 = silu_mul(g.x, u.x), y1 = silu_mul(g.y, u.y);
  const float y2 = silu_mul(g.z, u.z), y3 = silu_mul(g.w, u.w);
  const float m = lanes_max(fmax3(fmax3(fabsf(y0), fabsf(y1), fabsf(y2)), fabsf(y3), 0.f), 4);
  float r;
  const uint32_t code = block_code(m, gs, r);
  const float v[8] = {y0 * gs * r, y1 * gs * r, y2 * gs * r, y3 * gs * r};
  const uint32_t q = code ? quant_e2m1x8(v) : 0u;
  if (!live) return;
  uint8_t *o = a.q + t * (a.N / 2) + n / 2;
  if (VG_ACCESS_OK(g_fp4_gemm_status, o, 2, a.q, VG_ROWS(a.T) * (uint64_t)(a.N / 2)))
    *reinterpret_cast<uint16_t *>(o) = (uint16_t)q;
  if ((lane & 3) == 0) {
    uint8_t *p = a.sf + t * (a.N / kNvfp4Block) + n / kNvfp4Block;
    if (VG_ACCESS_OK(g_fp4_gemm_status, p, 1, a.sf, VG_ROWS(a.T) * (uint64_t)(a.N / kNvfp4Block)))
      *p = (uint8_t)code;
  }
}

// ----------------------------------------------------------- stream kernel
//
// For few tokens, where the weight's bytes are the cost.  The weight is the
// products' first operand: a CTA's tile is 128 weight rows (gated: 64 gate rows
// and the same 64 up rows) x TN tokens, and K is split over a cluster.  At the
// end each CTA puts its partial sums in shared memory and the cluster adds them
// in a fixed order, every CTA some of the tokens.
//   warp 0: TMA   warp 1: products   warps 2-5: scales, then the sums

constexpr int kMaxSplit = 8;
constexpr int kStreamThreads = 6 * 32;

template <int TN>
struct StreamSmem {
  static constexpr int kStageBytes = (kRows + TN) * kRowBytes;
  static constexpr int kStages = TN == 16 ? 5 : (TN <= 64 ? 4 : 6);
  static constexpr int kSfColumn = TN < 32 ? 32 : TN;                          // of tensor memory
  static constexpr int kColumns = kSfColumn + 64 <= 128 ? 128 : 256;
  union {
    uint8_t stage[kStages][kStageBytes];
    float part[TN][kRows];  // partial sums, once the products are done
  };
  uint8_t w_sf[kStages][kChunks * kAtom], a_sf[kStages][kChunks * kAtom];
  uint64_t full[kStages], sf_full[kStages], empty[kStages], drain;
  uint32_t tmem;
  uint32_t failed;
  VG_GEMM_NEVER
};

template <bool GATED, int TN>
__global__ void __launch_bounds__(kStreamThreads, TN <= 64 ? 2 : 1)
    fp4_gemm_stream_kernel(const Fp4GemmArgs a, const __grid_constant__ Fp4Maps maps, int num_n,
                           int splits, bool w_once) {
  extern __shared__ __align__(1024) uint8_t raw[];
  using Smem = StreamSmem<TN>;
  Smem &sm = *reinterpret_cast<Smem *>(raw);
  constexpr int kStages = Smem::kStages;
  constexpr int kTile = GATED ? kRows / 2 : kRows;  // output columns
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int num_k = (a.K + kStageK - 1) / kStageK;
  const int split = (int)cluster_rank();
  const int tile = (int)blockIdx.x / splits, t_tile = tile / num_n, n0 = (tile - t_tile * num_n) * kTile;
  // first weight rows of the tile's two halves, first token, stages of K
  const int r0 = n0, r1 = GATED ? a.N + n0 : n0 + kRows / 2;
  const int t0 = t_tile * TN;
  const int k0 = num_k * split / splits, k1 = num_k * (split + 1) / splits;

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.a);
    prefetch_tensormap(&maps.w);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.sf_full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.drain, 1);
    VG_GEMM_NEVER_INIT(sm);
    fence_mbar_init();
    sm.failed = 0;
  }
  if (warp == 1) tmem_alloc<false>(&sm.tmem, Smem::kColumns);
  // Launched with programmatic dependent launch: nothing but L2 prefetches of
  // the first weight stages before the previous grid has finished.
  if (warp == 2 && lane < 2 * kStages && t_tile == 0) {
    const int kb = k0 + (lane >> 1);
    if (kb < k1) tma_prefetch_2d(&maps.w, kb * kRowBytes, lane & 1 ? r1 : r0);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  int issued = 0;  // stages filled (warp 0)

  if (warp == 0) {
    int s = 0, lap = 0;
    const uint64_t policy = l2_evict_first();
    for (int kb = k0; kb < k1; ++kb) {
      if (lap > 0 && !warp_wait_phase(&sm.empty[s], (lap - 1) & 1, &sm.failed)) break;
      if (elect_lane()) {
        mbar_arrive_expect_tx(&sm.full[s], Smem::kStageBytes);
        uint8_t *p = sm.stage[s];
        const int x = kb * kRowBytes;
        if (w_once) {
          tma_load_2d_hint(p, &maps.w, x, r0, &sm.full[s], policy);
          tma_load_2d_hint(p + kRows / 2 * kRowBytes, &maps.w, x, r1, &sm.full[s], policy);
        } else {
          tma_load_2d(p, &maps.w, x, r0, &sm.full[s]);
          tma_load_2d(p + kRows / 2 * kRowBytes, &maps.w, x, r1, &sm.full[s]);
        }
        tma_load_2d(p + kRows * kRowBytes, &maps.a, x, t0, &sm.full[s]);
      }
      __syncwarp();
      ++issued;
      if (++s == kStages) s = 0, ++lap;
    }
  } else if (warp == 1) {
    constexpr uint32_t desc = nvfp4_product_desc(kRows, TN);
    int s = 0, lap = 0;
    for (int kb = k0; kb < k1; ++kb) {
      const int it = kb - k0, chunks = min(kChunks, (a.K - kb * kStageK) / 64);
      // half of the lanes wait for either barrier
      if (!warp_wait_phase(lane & 1 ? &sm.sf_full[s] : &sm.full[s], lap & 1, &sm.failed)) break;
      if (VG_GEMM_FORCED_TIMEOUT(sm, it == 0)) {
        sm.failed = 1;
        break;
      }
      tcgen05_fence_after();
      if (elect_lane()) {
        const uint64_t dw = operand_desc(smem_u32(sm.stage[s]));
        const uint64_t da = operand_desc(smem_u32(sm.stage[s] + kRows * kRowBytes));
        const uint64_t sw = scale_desc(smem_u32(sm.w_sf[s])), sa = scale_desc(smem_u32(sm.a_sf[s]));
        // the scales of alternate stages at two places of tensor memory
        const uint32_t tw = tmem + Smem::kSfColumn + (it & 1) * 32, ta = tw + 16;
        for (int c = 0; c < chunks; ++c) {
          tmem_copy_scales<false>(tw + 4 * c, sw + c * (kAtom >> 4));
          tmem_copy_scales<false>(ta + 4 * c, sa + c * (kAtom >> 4));
        }
        for (int c = 0; c < chunks; ++c)
          mma_nvfp4<false>(tmem, dw + 2 * c, da + 2 * c, desc, tw + 4 * c, ta + 4 * c, it + c > 0);
        mma_commit<false>(&sm.empty[s]);
      }
      __syncwarp();
      if (++s == kStages) s = 0, ++lap;
    }
    if (elect_lane()) mma_commit<false>(&sm.drain);
    __syncwarp();
    (void)mbar_wait_bounded(&sm.drain, 0);
  } else {
    // Scales: warp 2 + x has every fourth stage.
    const bool wide = a.K % kStageK == 0;
    const int64_t pitch = a.K / kNvfp4Block;
    const uint8_t *row_w[4], *row_a[4];
    bool live_w[4], live_a[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = lane + 32 * j, r = j < 2 ? r0 + row : r1 + row - kRows / 2;
      live_w[j] = r < (GATED ? 2 : 1) * a.N;
      row_w[j] = a.w_sf + (live_w[j] ? r * pitch : 0);
      live_a[j] = row < TN && t0 + row < a.T;
      row_a[j] = a.a_sf + (live_a[j] ? (t0 + row) * pitch : 0);
    }
    for (int kb = k0 + warp - 2; kb < k1; kb += 4) {
      const int it = kb - k0, s = it % kStages, lap = it / kStages;
      const int chunks = min(kChunks, (a.K - kb * kStageK) / 64), x = kb * (kStageK / kNvfp4Block);
      uint4 vw[4], va[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        vw[j] = load_scales(row_w[j] + x, live_w[j], wide, chunks, a.w_sf, w_sf_extent<GATED>(a));
        va[j] = load_scales(row_a[j] + x, live_a[j], wide, chunks, a.a_sf, a_sf_extent(a));
      }
      if (lap > 0 && !warp_wait_phase(&sm.empty[s], (lap - 1) & 1, &sm.failed)) break;
      store_scales(sm.w_sf[s], lane, vw);
      store_scales(sm.a_sf[s], lane, va);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.sf_full[s]);
    }
    // The products are done: nothing reads the stages any more.
    const int quarter = warp & 3, row = quarter * 32 + lane;
    if (warp_wait_phase(&sm.drain, 0, &sm.failed) && !*(volatile uint32_t *)&sm.failed) {
      tcgen05_fence_after();
#pragma unroll
      for (int c = 0; c < TN / 16; ++c) {
        uint32_t v[16];
        tmem_load(tmem + ((uint32_t)(quarter * 32) << 16) + c * 16, v);
        tmem_load_wait(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) sm.part[c * 16 + j][row] = __uint_as_float(v[j]);
      }
      tcgen05_fence_before();
    }
  }

  __syncthreads();
  pdl_launch_dependents();  // the loads are done
  if (sm.failed && warp == 0 && lane == 0) {  // copies in flight end here
    atomicOr(&g_fp4_gemm_status, kErrWaitTimeout);
    for (int it = issued < kStages ? 0 : issued - kStages; it < issued; ++it)
      (void)mbar_wait_bounded(&sm.full[it % kStages], (it / kStages) & 1);
  }
  cluster_sync();  // every CTA's partial sums are in place
  __syncwarp();
  if (warp == 1) tmem_dealloc<false>(tmem, Smem::kColumns);

  const int tokens = min(TN, a.T - t0);
  const float alpha = __ldg(a.alpha);
  if constexpr (!GATED) {  // a warp a token, a lane four columns
    for (int j = split + warp * splits; j < tokens; j += kStreamThreads / 32 * splits) {
      float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = 0; x < splits; ++x) {
        const float4 p = ld_cluster4(cluster_addr(&sm.part[j][4 * lane], (uint32_t)x));
        c = make_float4(c.x + p.x, c.y + p.y, c.z + p.z, c.w + p.w);
      }
      c = make_float4(alpha * c.x, alpha * c.y, alpha * c.z, alpha * c.w);
      store_out4(a, t0 + j, n0 + 4 * lane, c);
    }
  } else {  // half a warp a token
    const float gs = __ldg(a.global_scale);
    const int col = 4 * (lane & 15);
    for (int j0 = split + 2 * warp * splits; j0 < tokens; j0 += kStreamThreads / 16 * splits) {
      const int j = j0 + (lane >> 4) * splits;
      const bool live = j < tokens;
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
      for (int x = 0; x < splits; ++x) {
        const uint32_t at = cluster_addr(&sm.part[live ? j : 0][col], (uint32_t)x);
        const float4 p = ld_cluster4(at), q = ld_cluster4(at + 4 * kRows / 2);
        g = make_float4(g.x + p.x, g.y + p.y, g.z + p.z, g.w + p.w);
        u = make_float4(u.x + q.x, u.y + q.y, u.z + q.z, u.w + q.w);
      }
      g = make_float4(alpha * g.x, alpha * g.y, alpha * g.z, alpha * g.w);
      u = make_float4(alpha * u.x, alpha * u.y, alpha * u.z, alpha * u.w);
      store_gated4(a, t0 + j, live, n0 + col, lane, gs, g, u);
    }
  }
  cluster_sync();  // nobody reads this CTA's sums any more
}

// -------------------------------------------------------------------- host

template <bool GATED, int TN>
cudaError_t launch_stream(const Fp4GemmArgs &a, int splits, cudaStream_t s) {
  static std::atomic<uint64_t> opted_in{0};
  const cudaError_t e = opt_in_once(opted_in, (const void *)fp4_gemm_stream_kernel<GATED, TN>);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const int64_t rows = (GATED ? 2 : 1) * (int64_t)a.N;
  Fp4Maps maps;
  if (!make_map(&maps.a, u8, 1, a.a, a.T, a.K / 2, TN, kRowBytes, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&maps.w, u8, 1, a.w, rows, a.K / 2, kRows / 2, kRowBytes, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  maps.out = maps.a;  // not used: the sums are stored by threads
  const bool w_once = a.T <= TN && rows * a.K / 2 > 32 << 20;
  const int tile = GATED ? kRows / 2 : kRows, num_n = (a.N + tile - 1) / tile;
  const int64_t ctas = (int64_t)num_n * ((a.T + TN - 1) / TN) * splits;
  return launch_pdl_cluster(fp4_gemm_stream_kernel<GATED, TN>, dim3((unsigned)ctas), splits,
                            dim3(kStreamThreads), sizeof(StreamSmem<TN>), s, a, maps, num_n, splits, w_once);
}

template <bool GATED>
cudaError_t launch_form(const Fp4GemmArgs &a, const GemmPlan &p, cudaStream_t s) {
  switch (p.tn) {
    case 16: return launch_stream<GATED, 16>(a, p.splits, s);
    case 32: return launch_stream<GATED, 32>(a, p.splits, s);
    case 64: return launch_stream<GATED, 64>(a, p.splits, s);
    default: return launch_stream<GATED, 128>(a, p.splits, s);
  }
}

}  // namespace

GemmPlan plan_fp4_gemm(int64_t T, int64_t N, int64_t K, bool gated, int sms) {
  GemmPlan p;
  p.tn = T <= 16 ? 16 : (T <= 32 ? 32 : (T <= 64 ? 64 : 128));
  const int64_t tile = gated ? kRows / 2 : kRows, blocks = (K + kStageK - 1) / kStageK;
  const int64_t tiles = (N + tile - 1) / tile * ((T + p.tn - 1) / p.tn);
  const int64_t slots = (int64_t)sms * (p.tn <= 64 ? 2 : 1);
  p.splits = 1;
  while (p.splits < kMaxSplit && 2 * p.splits <= blocks && tiles * p.splits * 2 <= slots) p.splits *= 2;
  return p;
}

cudaError_t launch_fp4_gemm(const Fp4GemmArgs &a, bool gated, int sms, cudaStream_t s) {
  const GemmPlan p = plan_fp4_gemm(a.T, a.N, a.K, gated, sms);
  return gated ? launch_form<true>(a, p, s) : launch_form<false>(a, p, s);
}

uint32_t read_fp4_gemm_status(bool reset) {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_fp4_gemm_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (reset) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_fp4_gemm_status, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  }
  return v;
}

}  // namespace vg
