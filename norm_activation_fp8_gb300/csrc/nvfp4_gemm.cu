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
// ops write them.  Warps of their own move them: from 16 bytes (K of 256, a
// stage) of rows l, l + 32, ... come, for each K of 64, the four rows' words as
// one 16-byte row of the copy to tensor memory.
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
constexpr int kMaxSplit = 8;              // shares of K, a CTA each (stream kernel), of a cluster

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

// 16 bytes, or zeros (nothing is read) where `live` is false: a predicate, not a
// branch, so that loads follow one another at once.  It stays where it is
// written, ahead of the wait for the place that the data goes to.
__device__ __forceinline__ uint4 ld_live16(const uint8_t *p, bool live) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"((uint32_t)live));
  return v;
}

// The scales of one row and a stage's K: a word per K of 64; zeros for a row
// that is not there.  WIDE: all four, 16-byte aligned; otherwise (rows whose
// length is no multiple of 256) the first `chunks`, 7 to 15 % slower in all.
template <bool WIDE>
__device__ __forceinline__ uint4 load_scales(const uint8_t *p, bool live, int chunks, const uint8_t *base,
                                             uint64_t extent) {
  live = live && VG_ACCESS_OK(g_fp4_gemm_status, p, WIDE ? 16 : 4 * chunks, base, extent);
  if constexpr (WIDE) return ld_live16(p, live);
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!live) return v;
  v.x = ld_ro4(p);
  if (chunks > 1) v.y = ld_ro4(p + 4);
  if (chunks > 2) v.z = ld_ro4(p + 8);
  if (chunks > 3) v.w = ld_ro4(p + 12);
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

// Scales of 128 rows and a group of kGroup stages.  A row's scales of a group are
// 64 bytes: four lanes load them, so that a load of the warp touches eight rows
// (a lane a row and stage: 32 lines a load, of which an SM asks for one in about
// two cycles; 4096 x 8192 x 28672 395 instead of 297 us).  p0: this lane's
// 16 bytes of row lane / 4.  line(x, j): the distance of row 8 x + 32 j from it
// in the tensor (in bytes it fits 32 bits); place(x, j): in the tile, where rows
// from `left` on are not there.
constexpr int kGroup = 4;
template <bool WIDE, class Place, class Line>
__device__ __forceinline__ void load_group(uint4 (&v)[4][4], const uint8_t *p0, int pitch, int left, int chunks,
                                           const uint8_t *base, uint64_t extent, Place place, Line line) {
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[x][j] = load_scales<WIDE>(p0 + line(x, j) * pitch, place(x, j) < left, chunks, base, extent);
}

// Lane 4 r + p's value to lane 8 p + r.
__device__ __forceinline__ uint4 swap_lanes(const uint4 &v, int lane) {
  const int from = (lane & 7) * 4 + (lane >> 3);
  return make_uint4(__shfl_sync(0xFFFFFFFFu, v.x, from), __shfl_sync(0xFFFFFFFFu, v.y, from),
                    __shfl_sync(0xFFFFFFFFu, v.z, from), __shfl_sync(0xFFFFFFFFu, v.w, from));
}

// ... and to shared memory, the lanes having changed places: eight rows of one
// stage side by side.  dst: the place of this lane's stage, lane / 8.
__device__ __forceinline__ void store_group(uint8_t *dst, int lane, uint4 (&v)[4][4]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[x][j] = swap_lanes(v[x][j], lane);
    store_scales(dst, 8 * x + (lane & 7), v[x]);
  }
}

// SiLU(g) u with the accurate exponential and a division of two ulps (the
// correctly rounded one takes its slow way for g = 0: a tile of zeros took 26
// instead of 11 thousand cycles).
__device__ __forceinline__ float silu_mul(float g, float u) { return __fdividef(g, 1.0f + expf(-g)) * u; }

// A block's scale code, and the factor that y gs is multiplied by.
__device__ __forceinline__ uint32_t block_code(float amax, float gs, float &r) {
  const uint32_t code = e4m3_code(amax * gs * (1.0f / kE2M1Max));
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

__device__ __forceinline__ float4 scaled4(const float4 &v, float s) {
  return make_float4(v.x * s, v.y * s, v.z * s, v.w * s);
}

// Adds the cluster's partial sums at `from` (HALVES: and 64 columns behind it) in
// the order of the shares; all loads are on their way before the first is added.
template <int HALVES>
__device__ __forceinline__ void sum_shares(float4 (&c)[HALVES], const float *from, int splits) {
  float4 p[kMaxSplit][HALVES];
#pragma unroll
  for (int x = 0; x < kMaxSplit; ++x)
    if (x < splits)
#pragma unroll
      for (int h = 0; h < HALVES; ++h) p[x][h] = ld_cluster4(cluster_addr(from + h * (kRows / 2), (uint32_t)x));
#pragma unroll
  for (int h = 0; h < HALVES; ++h) c[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int x = 0; x < kMaxSplit; ++x)
    if (x < splits)
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const float4 q = p[x][h];
        c[h] = make_float4(c[h].x + q.x, c[h].y + q.y, c[h].z + q.z, c[h].w + q.w);
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
// A scale warp has every fourth stage, a lane rows l, l + 32, ... (four lanes a
// row and four stages at once, as in the tile kernel: 57 x 28672 x 8192 gated 49
// -> 52 us).  Up to 64 tokens two CTAs share an SM.
//
// Bound by the weight's bytes and 3.5 us for start and end (some 1.2 for the
// first stage, 0.3 for the last products, 0.9 for the sums of a cluster): gated
// 28672 x 8192, one token, 42 us (6.3 TB/s), 14336 x 4096 13.6 us (4.8); 57
// tokens x 28672 x 8192 gated 50 us (5.3; 448 CTAs are a wave and a half); 6144 x
// 4096, one token, 6.1 to 6.7 us (2.2).  A CTA that has no cluster waits for none
// (gated 57 tokens 52.1 -> 49.6 us, 16 tokens x 14336 x 4096 15.1 -> 14.1).

constexpr int kStreamThreads = 6 * 32;

template <int TN>
struct StreamSmem {
  static constexpr int kStageBytes = (kRows + TN) * kRowBytes;
  static constexpr int kStages = TN == 16 ? 5 : (TN <= 64 ? 4 : 6);
  // A scale warp that comes to stage i has seen stage i - 4 - kStages released,
  // so i - 2 kStages too: only then does the parity of its wait for the slot
  // (stage i - kStages) name one phase.
  static_assert(kStages >= 4, "four scale warps take turns");
  static constexpr int kSfColumn = TN < 32 ? 32 : TN;                          // of tensor memory
  static constexpr int kColumns = kSfColumn + 64 <= 128 ? 128 : 256;
  union {
    uint8_t stage[kStages][kStageBytes];
    float part[TN][kRows];  // partial sums, once the products are done
  };
  uint8_t w_sf[kStages][kChunks * kAtom], a_sf[kStages][kChunks * kAtom];
  uint64_t full[kStages], empty[kStages], drain;
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
      mbar_init(&sm.full[i], 2);  // copies, a scale warp
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
    VG_LOOKS;
    constexpr uint32_t desc = nvfp4_product_desc(kRows, TN);
    int s = 0, lap = 0;
    bool seen = false;
    for (int kb = k0; kb < k1; ++kb) {
      const int it = kb - k0;
      if (!warp_wait_phase(seen, &sm.full[s], lap & 1, &sm.failed)) break;
      if (VG_GEMM_FORCED_TIMEOUT(sm, it == 0)) {
        sm.failed = 1;
        break;
      }
      tcgen05_fence_after();
      const int now = s;
      if (++s == kStages) s = 0, ++lap;
      mbar_look<0>(&sm.full[s], lap & 1);  // while this stage's products are issued
      if (elect_lane()) {
        const uint64_t dw = operand_desc(smem_u32(sm.stage[now]));
        const uint64_t da = operand_desc(smem_u32(sm.stage[now] + kRows * kRowBytes));
        const uint64_t sw = scale_desc(smem_u32(sm.w_sf[now])), sa = scale_desc(smem_u32(sm.a_sf[now]));
        // the scales of alternate stages at two places of tensor memory
        const uint32_t tw = tmem + Smem::kSfColumn + (it & 1) * 32, ta = tw + 16;
        // All of a stage's scales, then its products: these are too short to
        // hide a copy each (one token x 8192 x 28672, two shares: 23.2 us).
        if (kb < num_k - 1 || a.K % kStageK == 0) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            tmem_copy_scales<false>(tw + 4 * c, sw + c * (kAtom >> 4));
            tmem_copy_scales<false>(ta + 4 * c, sa + c * (kAtom >> 4));
          }
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            mma_nvfp4<false>(tmem, dw + 2 * c, da + 2 * c, desc, tw + 4 * c, ta + 4 * c, it + c > 0);
        } else {
#pragma unroll 1
          for (int c = 0; c < a.K % kStageK / 64; ++c) {
            tmem_copy_scales<false>(tw + 4 * c, sw + c * (kAtom >> 4));
            tmem_copy_scales<false>(ta + 4 * c, sa + c * (kAtom >> 4));
            mma_nvfp4<false>(tmem, dw + 2 * c, da + 2 * c, desc, tw + 4 * c, ta + 4 * c, it + c > 0);
          }
        }
        mma_commit<false>(&sm.empty[now]);
      }
      __syncwarp();
      seen = mbar_seen<0>();
    }
    if (elect_lane()) mma_commit<false>(&sm.drain);
    __syncwarp();
    (void)mbar_wait_bounded(&sm.drain, 0);
  } else {
    // Scales: warp 2 + x has every fourth stage.
    const bool wide = a.wide != 0;
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
        if (wide) {
          vw[j] = load_scales<true>(row_w[j] + x, live_w[j], chunks, a.w_sf, w_sf_extent<GATED>(a));
          va[j] = load_scales<true>(row_a[j] + x, live_a[j], chunks, a.a_sf, a_sf_extent(a));
        } else {
          vw[j] = load_scales<false>(row_w[j] + x, live_w[j], chunks, a.w_sf, w_sf_extent<GATED>(a));
          va[j] = load_scales<false>(row_a[j] + x, live_a[j], chunks, a.a_sf, a_sf_extent(a));
        }
      }
      if (lap > 0 && !warp_wait_phase(&sm.empty[s], (lap - 1) & 1, &sm.failed)) break;
      store_scales(sm.w_sf[s], lane, vw);
      store_scales(sm.a_sf[s], lane, va);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.full[s]);
    }
    // The products are done: nothing reads the stages any more.
    const int quarter = warp & 3;
    if (warp_wait_phase(&sm.drain, 0, &sm.failed) && !*(volatile uint32_t *)&sm.failed) {
      tcgen05_fence_after();
#pragma unroll
      for (int c = 0; c < TN / 16; ++c) {
        uint32_t v[16];
        tmem_load(tmem + ((uint32_t)(quarter * 32) << 16) + c * 16, v);
        tmem_load_wait(v);
#pragma unroll
        for (int j = 0; j < 16; ++j) sm.part[c * 16 + j][quarter * 32 + lane] = __uint_as_float(v[j]);
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
  if (splits > 1) cluster_sync();  // every CTA's partial sums are in place
  __syncwarp();
  if (warp == 1) tmem_dealloc<false>(tmem, Smem::kColumns);

  const int tokens = min(TN, a.T - t0);
  const float alpha = ld_ro_f32(a.alpha);
  const float gs = GATED ? ld_ro_f32(a.global_scale) : 0.f;
  // Plain: a warp a token, a lane four columns; gated: half a warp.  The loads
  // of kAtOnce tokens are on their way before the first is added.
  constexpr int kPerWarp = GATED ? 2 : 1, kAtOnce = 2;
  const int col = GATED ? 4 * (lane & 15) : 4 * lane, mine = GATED ? lane >> 4 : 0;
  for (int j0 = split + kPerWarp * warp * splits; j0 < tokens;
       j0 += kAtOnce * kPerWarp * (kStreamThreads / 32) * splits) {
    float4 c[kAtOnce][kPerWarp];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = j0 + (i * kPerWarp * (kStreamThreads / 32) + mine) * splits;
      const float *from = &sm.part[j < tokens ? j : 0][col];
      sum_shares<kPerWarp>(c[i], from, splits);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = j0 + (i * kPerWarp * (kStreamThreads / 32) + mine) * splits;
      if constexpr (GATED)
        store_gated4(a, t0 + j, j < tokens, n0 + col, lane, gs, scaled4(c[i][0], alpha), scaled4(c[i][1], alpha));
      else if (j < tokens)
        store_out4(a, t0 + j, n0 + col, scaled4(c[i][0], alpha));
    }
  }
  if (splits > 1) cluster_sync();  // nobody reads this CTA's sums any more
}

// ------------------------------------------------------------- tile kernel
//
// Pairs of CTAs, one CTA per SM, compute tiles of 256 tokens x 256 weight rows
// (gated: 128 gate rows and the same 128 up rows, in turns of 16, so that a
// thread has gate and up of a block side by side).  A CTA of the pair stages
// its 128 tokens and one half of the weight rows; the scales of its tokens and
// of all the weight rows.
//   warp 0: TMA   warp 1: products   warps 2-7: scales   warps 8-15: epilogue
// Two accumulators of 256 columns and the scales do not fit into 512 columns,
// so the accumulators share kOverlap columns, which the epilogue reads first:
// the next tile's products start when these are in registers.
// Many tiles: persistent pairs.  Few tiles and a long K (SPLIT): up to four
// pairs of a cluster share a tile's K and add their sums through distributed
// shared memory in a fixed order.
//
// What bounds it, at 8192 x 8192 x 8192 (164 to 182 us by box, 6030 to 6700
// TFLOP/s in a burst; in a long run the power limit, 4093 x 8192 x 28672 284 us
// and then 324): a product of a pair takes 135 cycles, a stage's four 540. The
// issuing thread takes some 500 a stage (16 copies and products 130, two commits
// 80, the waits' votes 130, a look ahead 50, descriptors 50; the answer to the
// look taken at once was 120 more, 182 -> 193 us).  Between two tiles some 600
// cycles pass until the shared columns are read.  One wave of short tiles is
// bound by its start and end: 1024 x 4096 x 4096 12.4 us, 2.4 of them from the
// wait for the previous grid to the first products, 2.2 for the epilogue.  With
// most SMs at work a stage takes 0.30 to 0.35 us where eight pairs take 0.21
// (gated 0.28); which of the clock, the L2 and the scales' loads does that has not
// been measured apart.
// Narrow TMA boxes for the scales (64 bytes a row) were slower (4096 x 8192 x
// 28672 290 -> 331 us): they hold up the data's.

constexpr int kTileStages = 5;
constexpr int kTileStageBytes = 2 * kRows * kRowBytes;  // of either CTA
constexpr int kScaleWarps = 6, kOutWarps = 8, kTileThreads = 32 * (2 + kScaleWarps + kOutWarps);
constexpr int kAcc = 256;       // columns of an accumulator
constexpr int kOverlap = 64;    // shared by the two: what the epilogue reads first
constexpr int kSfColumn = 2 * kAcc - kOverlap;  // first column of the scales
static_assert(kSfColumn + 12 * kChunks <= 512, "tensor memory");
constexpr int kTileSplit = 4;   // shares of K, a pair each, of a cluster
constexpr int kTileGroup = 16;  // pairs' token tiles that share a sweep over the weight

template <bool GATED>
struct TileSmem {
  union {
    uint8_t stage[kTileStages][kTileStageBytes];
    float4 part[kRows][kAcc / 4];  // split K: partial sums, once the products are done
  };
  uint8_t out[GATED ? 1 : kOutWarps][GATED ? 16 : 32 * 64];  // boxes of 32 rows x 32 columns
  uint8_t sf[2][kGroup][3][kChunks * kAtom];  // of the tokens, of the weight's halves
  uint64_t full[kTileStages], empty[kTileStages], sf_full[2], sf_empty[2];
  uint64_t acc_full[2], acc_free, drain;
  uint32_t tmem;
  uint32_t failed;
  VG_GEMM_NEVER
};

// The i-th tile: token tiles run fastest within groups of kTileGroup, so that
// the tiles in flight share weight rows and the group's activations stay in L2
// while the weight streams by.
struct Tile {
  int t0;  // first token of the pair
  int n0;  // first output column
};
template <bool GATED>
__device__ __forceinline__ Tile tile_at(uint32_t i, uint32_t num_t, uint32_t num_n) {
  const uint32_t per_group = kTileGroup * num_n, g = i / per_group, r = i - g * per_group;
  const uint32_t rows = min((uint32_t)kTileGroup, num_t - g * kTileGroup), n = r / rows;
  return {(int)(g * kTileGroup + r - n * rows) * 2 * kRows, (int)n * (GATED ? kAcc / 2 : kAcc)};
}

// The rows of scales that a scale warp moves for a tile: role 0 the CTA's tokens,
// 1 and 2 either half of the weight's; a lane row lane / 4 and what lies 8 x +
// 32 j behind it in the tile.
template <bool GATED>
struct ScaleRows {
  const uint8_t *p, *base;  // this lane's row (of any stage)
  int left, pitch, up;      // rows from its own that are there; bytes a row; gate to up
  bool wide, turns;         // turns: of 16 gate rows and the same 16 up rows
  __device__ __forceinline__ ScaleRows(const Fp4GemmArgs &a, const Tile &t, int my_t, int role, int lane)
      : pitch(a.K / kNvfp4Block), up(a.N), wide(a.wide != 0), turns(GATED && role > 0) {
    const int row = (role == 0 ? t.t0 + my_t : t.n0 + (role - 1) * (GATED ? kRows / 2 : kRows)) + (lane >> 2);
    base = role == 0 ? a.a_sf : a.w_sf;
    p = base + (int64_t)row * pitch + (lane & 3) * (kStageK / kNvfp4Block);
    left = (role == 0 ? a.T : a.N) - row;
  }
  static __device__ __forceinline__ int plain(int x, int j) { return 32 * j + 8 * x; }
  static __device__ __forceinline__ int col(int x, int j) { return 16 * j + 8 * (x & 1); }

  // The group of stages from kb on, of those before `end`.
  __device__ __forceinline__ void load(uint4 (&v)[4][4], const Fp4GemmArgs &a, int kb, int end) const {
    const int mine = kb + ((int)threadIdx.x & 3), chunks = min(kChunks, (a.K - mine * kStageK) / 64);
    const uint8_t *q = p + kb * (kStageK / kNvfp4Block);
    const int n = mine < end ? left : 0;
    const uint64_t extent = base == a.a_sf ? a_sf_extent(a) : w_sf_extent<GATED>(a);
    const auto turned = [&](int x, int j) { return col(x, j) + (x >= 2 ? up : 0); };
    // (four calls: with the choice inside, at run time, the gated form spilled;
    // 4096 x 28672 x 8192 660 instead of 613 us)
    if (turns && wide)
      load_group<true>(v, q, pitch, n, chunks, base, extent, col, turned);
    else if (turns)
      load_group<false>(v, q, pitch, n, chunks, base, extent, col, turned);
    else if (wide)
      load_group<true>(v, q, pitch, n, chunks, base, extent, plain, plain);
    else
      load_group<false>(v, q, pitch, n, chunks, base, extent, plain, plain);
  }
};

template <bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp4_gemm_tile_kernel(const Fp4GemmArgs a, const __grid_constant__ Fp4Maps maps, int num_t, int num_n,
                         int splits) {
  extern __shared__ __align__(1024) uint8_t raw[];
  TileSmem<GATED> &sm = *reinterpret_cast<TileSmem<GATED> *>(raw);
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int all_k = (a.K + kStageK - 1) / kStageK;
  const uint32_t tiles = (uint32_t)num_t * (uint32_t)num_n;
  // rank in the pair, the pair's first rank in the cluster; the tiles of the
  // pair (SPLIT: one, shared by the cluster's pairs) and its stages of K
  const uint32_t rank = cluster_rank() & 1u, base = SPLIT ? cluster_rank() & ~1u : 0u;
  const uint32_t first = SPLIT ? blockIdx.x / (2u * (uint32_t)splits) : blockIdx.x >> 1;
  const uint32_t pairs = SPLIT ? tiles : gridDim.x >> 1;
  const int k_lo = SPLIT ? all_k * (int)(base >> 1) / splits : 0;
  const int num_k = (SPLIT ? all_k * (int)((base >> 1) + 1) / splits : all_k) - k_lo;
  const int my_t = (int)rank * kRows;  // this CTA's tokens within the pair's

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.a);
    prefetch_tensormap(&maps.w);
    if (!GATED) prefetch_tensormap(&maps.out);
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.sf_full[i], 6);  // three warps of both CTAs (the first CTA's counts)
      mbar_init(&sm.sf_empty[i], 1);
    }
    mbar_init(&sm.acc_free, 2 * kOutWarps);  // of both CTAs (the first CTA's counts)
    mbar_init(&sm.drain, 1);
    VG_GEMM_NEVER_INIT(sm);
    fence_mbar_init();
    sm.failed = 0;
  }
  if (warp == 1) tmem_alloc<true>(&sm.tmem, 512);
  tcgen05_fence_before();
  __syncthreads();
  // The pair's barriers are initialised.  (Relaxed: they are all that the other
  // CTA may see by now, and fence_mbar_init() has ordered them; a release here
  // took 1.3 us.)
  cluster_arrive_relaxed();
  // Launched with programmatic dependent launch: nothing but L2 prefetches of
  // the first stages before the previous grid has finished.
  const Tile t_first = tile_at<GATED>(first, num_t, num_n);
  const ScaleRows<GATED> rows(a, t_first, my_t, (warp + 1) % 3, lane);  // (warps 2-7; of the first tile)
  if (warp == 2 + kScaleWarps && lane < 2 * kTileStages && (lane >> 1) < num_k) {
    const int x = (k_lo + (lane >> 1)) * kRowBytes;
    if (lane & 1)
      tma_prefetch_2d(&maps.a, x, t_first.t0 + my_t);
    else if constexpr (GATED)
      tma_prefetch_4d(&maps.w, x, 0, 0, t_first.n0 / 16 + (int)rank * 4);
    else
      tma_prefetch_2d(&maps.w, x, t_first.n0 + (int)rank * kRows);
  }
  cluster_wait();
  tcgen05_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  pdl_launch_dependents();
  uint32_t issued = 0;  // stages this CTA has filled (warp 0)

  if (warp == 0) {
    uint32_t s = 0, lap = 0;
    bool ok = true;
    for (uint32_t i = first; i < tiles && ok; i += pairs) {
      const Tile t = tile_at<GATED>(i, num_t, num_n);
      for (int kb = 0; kb < num_k; ++kb) {
        if (lap > 0 && !(ok = warp_wait_phase(&sm.empty[s], (lap - 1) & 1, &sm.failed))) break;
        if (elect_lane()) {
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * kTileStageBytes);
          uint8_t *p = sm.stage[s];
          const uint32_t bar = cluster_addr(&sm.full[s], base);
          const int x = (k_lo + kb) * kRowBytes;
          tma_load_2d_pair(p, &maps.a, x, t.t0 + my_t, bar);
          if constexpr (GATED)
            tma_load_4d_pair(p + kRows * kRowBytes, &maps.w, x, 0, 0, t.n0 / 16 + (int)rank * 4, bar);
          else
            tma_load_2d_pair(p + kRows * kRowBytes, &maps.w, x, t.n0 + (int)rank * kRows, bar);
        }
        __syncwarp();
        ++issued;
        if (++s == kTileStages) s = 0, ++lap;
      }
    }
    // The last stages are released in both CTAs by products that the first one
    // issued: neither CTA may end before these arrivals have landed.
    for (uint32_t i = issued < kTileStages ? 0 : issued - kTileStages; i < issued && ok; ++i)
      ok = warp_wait_phase(&sm.empty[i % kTileStages], (i / kTileStages) & 1, &sm.failed);
  } else if (warp == 1 && rank == 0) {
    VG_LOOKS;
    constexpr uint32_t desc = nvfp4_product_desc(2 * kRows, kAcc);
    uint32_t s = 0, lap = 0, j = 0, group = 0;
    bool ok = true, seen = false, seen_sf = false;
    for (uint32_t i = first; i < tiles && ok; i += pairs, ++j) {
      const uint32_t acc = tmem + (j & 1) * (kAcc - kOverlap);
      if (j > 0 && !(ok = warp_wait_phase(&sm.acc_free, (j - 1) & 1, &sm.failed))) break;
      for (int kb = 0; kb < num_k; ++kb) {
        const int part = kb % kGroup;
        if (part == 0 && !(ok = warp_wait_phase<true>(seen_sf, &sm.sf_full[group & 1], (group >> 1) & 1, &sm.failed)))
          break;
        if (!(ok = warp_wait_phase(seen, &sm.full[s], lap & 1, &sm.failed))) break;
        if (VG_GEMM_FORCED_TIMEOUT(sm, j == 0 && kb == 0)) {
          sm.failed = 1;
          ok = false;
          break;
        }
        tcgen05_fence_after();
        const uint32_t now = s;
        if (++s == kTileStages) s = 0, ++lap;
        // A look at the next stage, answered once this one's products are issued
        // (even a wait for nothing takes some 160 cycles).
        mbar_look<0>(&sm.full[s], lap & 1);
        const bool last = part == kGroup - 1 || kb == num_k - 1;
        if (last) mbar_look<1>(&sm.sf_full[(group + 1) & 1], ((group + 1) >> 1) & 1);
        if (elect_lane()) {
          const uint64_t da = operand_desc(smem_u32(sm.stage[now]));
          const uint64_t dw = operand_desc(smem_u32(sm.stage[now] + kRows * kRowBytes));
          const uint64_t sa = scale_desc(smem_u32(sm.sf[group & 1][part][0]));
          const uint64_t sw = sa + (kChunks * kAtom >> 4);
          const uint32_t ta = tmem + kSfColumn, tw = ta + 4 * kChunks;
          // Each product right behind its own scales (all of a stage's scales
          // first: 4390 instead of 5270 TFLOP/s): they are copied while the
          // product before runs.
          const auto issue = [&](int c) {
            tmem_copy_scales<true>(ta + 4 * c, sa + c * (kAtom >> 4));
            tmem_copy_scales<true>(tw + 8 * c, sw + c * (kAtom >> 4));
            tmem_copy_scales<true>(tw + 8 * c + 4, sw + (kChunks + c) * (kAtom >> 4));
            mma_nvfp4<true>(acc, da + 2 * c, dw + 2 * c, desc, ta + 4 * c, tw + 8 * c, kb + c > 0);
          };
          if (k_lo + kb < all_k - 1 || a.K % kStageK == 0) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) issue(c);
          } else {
#pragma unroll 1
            for (int c = 0; c < a.K % kStageK / 64; ++c) issue(c);
          }
          mma_commit_pair(&sm.empty[now], base);
          if (last) mma_commit_pair(&sm.sf_empty[group & 1], base);
          if (kb == num_k - 1) mma_commit_pair(&sm.acc_full[j & 1], base);
        }
        __syncwarp();
        seen = mbar_seen<0>();
        if (last) seen_sf = mbar_seen<1>();
        group += last;
      }
    }
    // Nothing is in flight once this arrives (at once, unless a wait gave up).
    if (elect_lane()) mma_commit<true>(&sm.drain);
    __syncwarp();
    (void)mbar_wait_bounded(&sm.drain, 0);
  } else if (warp >= 2 && warp < 2 + kScaleWarps) {
    // Scales of 128 rows (tokens, either half of the weight's), every other
    // group of stages, counted over all tiles.
    const int role = (warp - 2) % 3, turn = (warp - 2) / 3;
    uint32_t group = 0, lap = 0;  // groups so far, this warp's
    bool ok = true;
    for (uint32_t i = first; i < tiles && ok; i += pairs) {
      const ScaleRows<GATED> r = i == first ? rows : ScaleRows<GATED>(a, tile_at<GATED>(i, num_t, num_n), my_t, role, lane);
      for (int k = 0; k < num_k; k += kGroup, ++group) {
        if ((int)(group & 1) != turn) continue;
        uint4 v[4][4];
        r.load(v, a, k_lo + k, k_lo + num_k);
        if (lap > 0 && !(ok = warp_wait_phase(&sm.sf_empty[turn], (lap - 1) & 1, &sm.failed))) break;
        ++lap;
        store_group(sm.sf[turn][lane >> 3][role], lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_written(cluster_addr(&sm.sf_full[turn], base));
      }
    }
    // (as for the stages: the last release has landed)
    if (lap > 0 && ok) (void)warp_wait_phase(&sm.sf_empty[turn], (lap - 1) & 1, &sm.failed);
  } else if (warp >= 2 + kScaleWarps) {
    const int quarter = warp & 3, half = (warp - 2 - kScaleWarps) >> 2;  // lanes, columns
    const uint32_t free_bar = cluster_addr(&sm.acc_free, base);
    const float alpha = ld_ro_f32(a.alpha), gs = GATED ? ld_ro_f32(a.global_scale) : 0.f;
    uint32_t j = 0;
    for (uint32_t i = first; i < tiles; i += pairs, ++j) {
      const Tile t = tile_at<GATED>(i, num_t, num_n);
      const uint32_t b = j & 1;
      if (!warp_wait_phase(&sm.acc_full[b], (j >> 1) & 1, &sm.failed)) break;
      tcgen05_fence_after();
      const uint32_t base =
          tmem + ((uint32_t)(quarter * 32) << 16) + b * (kAcc - kOverlap) + half * (kAcc / 2);
      const int t0 = t.t0 + my_t + quarter * 32;  // this warp's first token
#pragma unroll 1
      for (int p = 0; p < 2; ++p) {
        // The 64 columns that the other accumulator shares come first: the top
        // ones of the first, the bottom ones of the second.
        const int c0 = (b ? p : 1 - p) * 64;
        uint32_t v[2][32];
        tmem_load(base + c0, v[0]);
        tmem_load(base + c0 + 32, v[1]);
        tmem_load_wait(v[0]);
        tmem_load_wait(v[1]);
        if constexpr (SPLIT) {
          // Partial sums to shared memory (the products are done, so nothing
          // reads the stages), 16-byte chunks swizzled by the row.
          const int c = (half * (kAcc / 2) + c0) / 4;
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const uint32_t *x = &v[q >> 3][4 * (q & 7)];
            sm.part[quarter * 32 + lane][(c + q) ^ (lane & 7)] =
                make_float4(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]), __uint_as_float(x[3]));
          }
          continue;
        }
        if (p == 0) {
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(free_bar);
        }
        if constexpr (!GATED) {
          const int n = t.n0 + half * (kAcc / 2) + c0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // a box of 32 columns, 64 bytes a row
            uint8_t *box = sm.out[warp - 2 - kScaleWarps];
            if (lane == 0) tma_store_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2_rn(alpha * __uint_as_float(v[h][8 * q + 2 * k]),
                                      alpha * __uint_as_float(v[h][8 * q + 2 * k + 1]));
              *reinterpret_cast<uint4 *>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (t0 < a.T && n + 32 * h < a.N) tma_store_2d(&maps.out, box, n + 32 * h, t0);
              tma_store_commit();
            }
          }
        } else {
          const int n = t.n0 + (half * (kAcc / 2) + c0) / 2;
          uint32_t codes[4], sf = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 gate columns, then up
            float y[16], m = 0.f, r;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              y[k] = silu_mul(alpha * __uint_as_float(v[h][k]), alpha * __uint_as_float(v[h][16 + k]));
              m = fmaxf(m, fabsf(y[k]));
            }
            const uint32_t code = block_code(m, gs, r);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float q[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) q[k] = y[8 * x + k] * gs * r;
              codes[2 * h + x] = code ? quant_e2m1x8(q) : 0u;
            }
            sf |= code << (8 * h);
          }
          const int64_t token = t0 + lane;
          if (token < a.T && n < a.N) {  // whole: n and N are multiples of 32 and 64
            uint8_t *o = a.q + token * (a.N / 2) + n / 2;
            if (VG_ACCESS_OK(g_fp4_gemm_status, o, 16, a.q, VG_ROWS(a.T) * (uint64_t)(a.N / 2)))
              *reinterpret_cast<uint4 *>(o) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            uint8_t *f = a.sf + token * (a.N / kNvfp4Block) + n / kNvfp4Block;
            if (VG_ACCESS_OK(g_fp4_gemm_status, f, 2, a.sf, VG_ROWS(a.T) * (uint64_t)(a.N / kNvfp4Block)))
              *reinterpret_cast<uint16_t *>(f) = (uint16_t)sf;
          }
        }
      }
    }
    if (!GATED && lane == 0) tma_store_wait_read<0>();
  }

  __syncthreads();
  if (sm.failed && warp == 0 && lane == 0) {  // the pair's copies in flight end here
    atomicOr(&g_fp4_gemm_status, kErrWaitTimeout);
    if (rank == 0)
      for (uint32_t it = issued < kTileStages ? 0 : issued - kTileStages; it < issued; ++it)
        (void)mbar_wait_bounded(&sm.full[it % kTileStages], (it / kTileStages) & 1);
    // copies that the other CTA issued ahead of this one's count: a millisecond
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
  }
  cluster_sync();  // SPLIT: all partial sums are in place; otherwise the pair is done
  __syncwarp();
  if (warp == 1) tmem_dealloc<true>(tmem, 512);
  if constexpr (SPLIT) {
    // Each pair of the cluster adds some of the tile's rows, in a fixed order:
    // a warp a token row, a lane four columns of either half (gated: gate and
    // up of four columns).
    const Tile t = tile_at<GATED>(first, num_t, num_n);
    const float alpha = ld_ro_f32(a.alpha), gs = GATED ? ld_ro_f32(a.global_scale) : 0.f;
    for (int row = (int)(base >> 1) + warp * splits; row < kRows; row += kTileThreads / 32 * splits) {
      const int64_t token = t.t0 + my_t + row;
      if (token >= a.T) break;
      // gated: turns of 16 gate and 16 up columns, four lanes each
      const int c0 = GATED ? 8 * (lane >> 2) + (lane & 3) : lane, c1 = c0 + (GATED ? 4 : kAcc / 8);
      float4 p[kTileSplit][2], c[2] = {};
#pragma unroll
      for (int x = 0; x < kTileSplit; ++x)
        if (x < splits) {
          const uint32_t from = 2u * (uint32_t)x + rank;
          p[x][0] = ld_cluster4(cluster_addr(&sm.part[row][c0 ^ (row & 7)], from));
          p[x][1] = ld_cluster4(cluster_addr(&sm.part[row][c1 ^ (row & 7)], from));
        }
#pragma unroll
      for (int x = 0; x < kTileSplit; ++x)
        if (x < splits)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            c[h] = make_float4(c[h].x + p[x][h].x, c[h].y + p[x][h].y, c[h].z + p[x][h].z, c[h].w + p[x][h].w);
      const int n = t.n0 + 4 * lane;
      if constexpr (!GATED) {
        store_out4(a, token, n, scaled4(c[0], alpha));
        store_out4(a, token, n + kAcc / 2, scaled4(c[1], alpha));
      } else {
        store_gated4(a, token, n < a.N, n, lane, gs, scaled4(c[0], alpha), scaled4(c[1], alpha));
      }
    }
    cluster_sync();  // nobody reads this CTA's sums any more
  }
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

template <bool GATED, bool SPLIT>
cudaError_t launch_tile(const Fp4GemmArgs &a, int splits, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> opted_in{0};
  const cudaError_t e = opt_in_once(opted_in, (const void *)fp4_gemm_tile_kernel<GATED, SPLIT>);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  Fp4Maps maps;
  if (!make_map(&maps.a, u8, 1, a.a, a.T, a.K / 2, kRows, kRowBytes, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  if constexpr (GATED) {
    // byte of a row, row of a turn of 16, gate or up, turn
    const cuuint64_t row = (cuuint64_t)a.K / 2;
    const cuuint64_t dims[4] = {row, 16, 2, (cuuint64_t)a.N / 16};
    const cuuint64_t strides[3] = {row, row * (cuuint64_t)a.N, row * 16};
    const cuuint32_t box[4] = {kRowBytes, 16, 2, 4};
    if (!make_map(&maps.w, u8, a.w, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    maps.out = maps.a;  // not used: the codes are stored by threads
  } else if (!make_map(&maps.w, u8, 1, a.w, a.N, a.K / 2, kRows, kRowBytes, CU_TENSOR_MAP_SWIZZLE_128B) ||
             !make_map(&maps.out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.out, a.T, a.N, 32, 32,
                       CU_TENSOR_MAP_SWIZZLE_64B)) {
    return cudaErrorInvalidValue;
  }
  const int num_t = (a.T + 2 * kRows - 1) / (2 * kRows);
  const int tile = GATED ? kAcc / 2 : kAcc, num_n = (a.N + tile - 1) / tile;
  const int64_t tiles = (int64_t)num_t * num_n;
  const int64_t pairs = SPLIT ? tiles * splits : (tiles < sms / 2 ? tiles : sms / 2);
  return launch_pdl_cluster(fp4_gemm_tile_kernel<GATED, SPLIT>, dim3((unsigned)(2 * pairs)),
                            SPLIT ? 2 * splits : 2, dim3(kTileThreads), sizeof(TileSmem<GATED>), s, a, maps,
                            num_t, num_n, splits);
}

template <bool GATED>
cudaError_t launch_form(const Fp4GemmArgs &a, const GemmPlan &p, int sms, cudaStream_t s) {
  switch (p.tn) {
    case 16: return launch_stream<GATED, 16>(a, p.splits, s);
    case 32: return launch_stream<GATED, 32>(a, p.splits, s);
    case 64: return launch_stream<GATED, 64>(a, p.splits, s);
    case 128: return launch_stream<GATED, 128>(a, p.splits, s);
    default:
      return p.splits > 1 ? launch_tile<GATED, true>(a, p.splits, sms, s)
                          : launch_tile<GATED, false>(a, 1, sms, s);
  }
}

}  // namespace

// Which kernel, and its split, by a cost of either one, in microseconds (fitted
// on GB300 to T = 1..2048, N = 1024..28672, K = 4096..28672, plain and gated;
// over those 117 sizes the choice was on average 1.5 %, at most 12 % above the
// best one).  It ranks forms and is no forecast: where tiles fill the chip a stage
// takes up to 0.35 us, and it is 15 to 25 % low (8192 x 8192 x 8192 140 us, 164 to
// 182 measured), but there no other form comes near (the stream kernel's 440).
//   tile kernel    8.1 (one share) .. 10 (four) for start and end, 1.2 for each
//                  further wave of pairs, and 0.26 per stage of K or the
//                  weight's bytes at 6 TB/s, whichever is longer
//   stream kernel  a wave of CTAs: 3.5 and 0.11 for each CTA of a cluster, and
//                  0.2 (128 tokens: 0.4) per stage of its share or the weight's
//                  bytes at 6.3 TB/s (0.7 of that again for every further token
//                  tile, which reads the weight from L2), whichever is longer,
//                  with a fifth of the other
// Clusters do not fill every SM, and a second wave costs as much as the first,
// so a wave is taken as the part of the slots that clusters of that size were
// seen to fill.  Splits of the stream kernel are powers of two: others pack
// worse.
GemmPlan plan_fp4_gemm(int64_t T, int64_t N, int64_t K, bool gated, int sms) {
  GemmPlan p;
  const int64_t blocks = (K + kStageK - 1) / kStageK;
  const double bytes = (double)N * (double)K * (gated ? 2 : 1) * 0.5625e-6;  // of the weight, in MB
  const auto waves_of = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
  const auto part = [](int64_t slots, int64_t percent) { return slots < 8 ? slots : slots * percent / 100; };
  const int64_t column = gated ? kAcc / 2 : kAcc;
  const int64_t pairs = (T + 2 * kRows - 1) / (2 * kRows) * ((N + column - 1) / column);
  static const double kFixed[kTileSplit] = {8.1, 8.4, 9.0, 10.0};
  static const int kFill[kTileSplit] = {100, 90, 64, 64};
  double best = 1e30;
  for (int s = 1; s <= kTileSplit && s <= blocks; ++s) {
    const double waves = waves_of(pairs * s, part(sms < 2 ? 1 : sms / 2, kFill[s - 1]));
    if (s > 1 && waves > 1) break;
    const double chain = waves * 0.26 * (double)((blocks + s - 1) / s), traffic = bytes / 6.0;
    const double cost = kFixed[s - 1] + 1.2 * (waves - 1) + (chain > traffic ? chain : traffic);
    if (cost < best) {
      best = cost;
      p.splits = s;
    }
  }
  // one token tile, or for more than 64 tokens tiles of 64 or 128
  const int64_t rows = gated ? N / (kRows / 2) : (N + kRows - 1) / kRows;
  const int smallest = T <= 16 ? 16 : (T <= 32 ? 32 : 64);
  for (int tn = smallest; tn <= (T <= 64 ? smallest : 128); tn *= 2) {
    const int64_t token_tiles = (T + tn - 1) / tn, slots = (int64_t)sms * (tn <= 64 ? 2 : 1);
    if (rows * token_tiles * kMaxSplit > INT32_MAX) continue;
    for (int s = 1; s <= kMaxSplit && s <= blocks; s *= 2) {
      const double waves = waves_of(rows * token_tiles * s, part(slots, s == 8 ? 64 : 86));
      const double chain = (double)((blocks + s - 1) / s) * (tn <= 64 ? 0.2 : 0.4);
      const double traffic = bytes * (1.0 + 0.7 * (double)(token_tiles - 1)) / waves / 6.3;
      const double cost =
          waves * (3.5 + 0.11 * s + (chain > traffic ? chain + 0.2 * traffic : traffic + 0.2 * chain));
      if (cost < best) {
        best = cost;
        p.tn = tn;
        p.splits = s;
      }
    }
  }
  return p;
}

cudaError_t launch_fp4_gemm(const Fp4GemmArgs &a, bool gated, int sms, cudaStream_t s) {
  const GemmPlan p = plan_fp4_gemm(a.T, a.N, a.K, gated, sms);
  return gated ? launch_form<true>(a, p, sms, s) : launch_form<false>(a, p, sms, s);
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
