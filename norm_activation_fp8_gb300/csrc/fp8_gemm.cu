// fp8_gemm.cu -- FP8 matrix product with a scale per block of 128 columns, and
// the gated feed-forward projection on top of it.
//
//   c[t, n] = sum_b sa[t, b] sw[n / 128, b] sum_{k in block b} a[t, k] w[n, k]
//   plain:  out = bf16(c)
//   gated:  g = c[t, n], u = c[t, I + n], y = g / (1 + exp(-g)) u (fp32, never
//           rounded to bf16), s = max(amax |y| over 128 columns, 1e-10) / 448
//           (or the power of two above it), q = e4m3(y / s)
//
// Tile kernel.  Pairs of CTAs, one CTA per SM, compute tiles of 256 tokens x
// 256 weight rows (gated: 128 gate rows and the same 128 up rows), one scale
// block (128 of K) at a time.  A CTA of the pair stages its 128 tokens and one
// half of the weight rows by TMA in five 32 KB stages; one thread of the pair
// issues four M256 N256 K32 products, which read the weight halves of both (a
// CTA alone would stage and read all 256 weight rows: 96 KB of shared memory
// traffic a block for 512 cycles of products, more than the 128 bytes a cycle
// that there are; a pair needs 64 KB).  They go to one of two 256-column
// accumulators, and in either CTA sixteen warps take the block's sum out of
// tensor memory and add it, times its two scales, to an fp32 sum in registers
// (the block scales are arbitrary fp32 numbers, so the tensor cores cannot
// apply them).  The two accumulators let the products of the next block run
// meanwhile.  A thread holds 32 columns of either half of a token's row: for
// the gated form gate and up of the same columns, so that the activation needs
// no exchange and a group's amax one float from each of the three warps beside
// it.
//   warp 0: TMA   warp 1: products   warp 2: scales (global -> shared)
//   warps 4-19: sums and epilogue (warp w: tensor memory lanes 32 (w mod 4))
// Many tiles: persistent pairs.  Few tiles and a long K (SPLIT): up to four
// pairs of a cluster share a tile's scale blocks and add their fp32 sums
// through distributed shared memory in a fixed order.
//
// What bounds it, at 4096 x 8192 x 28672 (684 us, 2810 TFLOP/s; the measured
// bf16 rate is 1946 in a burst, so e4m3 at most about 3890): a block takes 840
// cycles.  Its products are 512; the way round an accumulator (products
// issued, finished, seen by the summing warps, read, given back to the issuing
// warp) costs 940 cycles without any work in it, and with two accumulators half
// of that and of the work shows.  Without the sums it runs at 3230, without
// sums and tensor memory loads at 3470 TFLOP/s.  A block's products take two
// cycles a column (back to back, a pair: 259, 323, 387, 451, 515 cycles for 128,
// 160, 192, 224, 256 columns; 64 columns take 175), so narrower accumulators
// lose nothing there; but four of 128 columns, or one released by halves, have
// twice the waits and arrivals for the same work and were slower (2120).  Three
// of 160 columns have not been built.  A CTA alone reached 1980, eight summing
// warps 1760.  The persistent forms spill 20 bytes.  Long runs meet the power
// limit first.
#include "dyn_scale.cuh"
#include "gemm_common.cuh"

namespace vg {

// Status word of this translation unit's kernels.
__device__ uint32_t g_gemm_status;

namespace {

constexpr int kBlockK = 128;  // codes of K per scale block (and per stage)
constexpr int kHalfW = 128;   // weight rows of a tile's half (tile kernel), of a tile (stream kernel)

__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// The scale of a group (an ulp or two in s moves only codes that near a
// midpoint) and the factor that its codes are multiplied by.
__device__ __forceinline__ float group_scale(float amax, bool ue8m0) {
  const float a = fmaxf(amax, kAmaxFloor);
  return ue8m0 ? exp2i(pow2_exponent_448(a)) : a * kInv448;
}

// Extent in bytes of the scale tensor (debug checks).
[[maybe_unused]] __device__ __forceinline__ uint64_t gemm_scale_extent(const GemmArgs &a) {
  const uint64_t rows = VG_ROWS(a.T);
  return rows == 0 ? 0 : 4 * ((rows - 1) * (uint64_t)a.s_ts + (uint64_t)(a.N / kBlockK - 1) * a.s_gs + 1);
}

// Extents in bytes of the operands' scale tensors (debug checks; the operands
// themselves and the tile kernel's outputs are clipped by their tensor maps).
[[maybe_unused]] __device__ __forceinline__ uint64_t a_scale_extent(const GemmArgs &a) {
  const uint64_t rows = VG_ROWS(a.T);
  return rows == 0 ? 0 : 4 * ((rows - 1) * (uint64_t)a.a_ts + (uint64_t)(a.K / kBlockK - 1) * a.a_bs + 1);
}
template <bool GATED>
[[maybe_unused]] __device__ __forceinline__ uint64_t w_scale_extent(const GemmArgs &a) {
  return 4ull * (((GATED ? 2 : 1) * (uint64_t)a.N + kBlockK - 1) / kBlockK) * (uint64_t)(a.K / kBlockK);
}

// Four columns of a token's output row, from n on (N is a multiple of 8).
__device__ __forceinline__ void store_out4(const GemmArgs &a, int64_t t, int n, const float4 &c) {
  uint16_t *o = a.out + t * a.N + n;
  if (n < a.N && VG_ACCESS_OK(g_gemm_status, o, 8, a.out, VG_ROWS(a.T) * 2ull * (uint64_t)a.N))
    *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2_rn(c.x, c.y), pack_bf16x2_rn(c.z, c.w));
}

// Activation and codes of a token's group of 128 columns, a warp: lane has
// gate and up of columns 4 lane ..
__device__ __forceinline__ void store_gated4(const GemmArgs &a, int64_t t, int group, int lane,
                                             const float4 &g, const float4 &u) {
  const float y0 = silu_mul(g.x, u.x), y1 = silu_mul(g.y, u.y);
  const float y2 = silu_mul(g.z, u.z), y3 = silu_mul(g.w, u.w);
  const float m = warp_max(fmax3(fmax3(fabsf(y0), fabsf(y1), fabsf(y2)), fabsf(y3), 0.f));
  const float s = group_scale(m, a.ue8m0 != 0), r = __frcp_rn(s);
  uint8_t *o = a.q + t * a.N + (int64_t)group * kHalfW + 4 * lane;
  if (VG_ACCESS_OK(g_gemm_status, o, 4, a.q, VG_ROWS(a.T) * (uint64_t)a.N))
    *reinterpret_cast<uint32_t *>(o) = cvt_e4m3x2(y0 * r, y1 * r) | (cvt_e4m3x2(y2 * r, y3 * r) << 16);
  if (lane == 0) {
    float *p = a.scale + t * a.s_ts + (int64_t)group * a.s_gs;
    if (VG_ACCESS_OK(g_gemm_status, p, 4, a.scale, gemm_scale_extent(a))) *p = s;
  }
}

// ------------------------------------------------------------- tile kernel

constexpr int kTileT = 128, kTileW = 256;
constexpr int kTileStages = 5;
constexpr int kScaleSlots = 8;  // scale blocks staged ahead
constexpr int kTileStageBytes = (kTileT + kHalfW) * kBlockK;  // of either CTA
// Four warps of a scheduler hide each other's tensor memory loads (eight warps
// of 128 columns a thread: 1760 instead of 1980 TFLOP/s, before the pairs).
constexpr int kSumWarps = 16, kTileThreads = 128 + 32 * kSumWarps;
constexpr int kPart = kHalfW * 4 / kSumWarps;  // columns of either half that a thread sums
// The launch holds 640 x 96 registers; setmaxnreg hands out 128 x 56 + 512 x
// 104 of them.
constexpr int kServiceRegs = 56, kSumRegs = 104;
static_assert(128 * kServiceRegs + 32 * kSumWarps * kSumRegs <= kTileThreads * 96, "register split");
constexpr int kTileGroup = 16;  // pairs' token tiles that share a sweep over the weight

// Dynamic shared memory (1024-byte aligned).
template <bool GATED>
struct TileSmem {
  union {
    uint8_t stage[kTileStages][kTileStageBytes];
    float4 part[kTileT][kTileW / 4];  // split K: partial sums, once the products are done
  };
  uint8_t out[kSumWarps][32 * kPart * (GATED ? 1 : 2)];  // a box of 32 rows
  float sa[2][kScaleSlots][kTileT];
  float sw[2][kScaleSlots][2];
  float amax[GATED ? 2 : 1][GATED ? kSumWarps / 4 : 1][GATED ? kTileT : 1];
  uint64_t full[kTileStages], empty[kTileStages];
  uint64_t acc_full[2], acc_empty[2], scale_full[2], scale_empty[2], drain;
  uint32_t tmem;
  uint32_t failed;
  VG_GEMM_NEVER
};

// The i-th tile: token tiles run fastest within groups of kTileGroup, so that
// the tiles in flight share weight rows and the group's activations stay in L2
// while the weight streams by (groups of 4 and 8: within 5 %).
struct Tile {
  int t0;  // first token of the pair
  int n;   // weight tile
};
__device__ __forceinline__ Tile tile_at(uint32_t i, uint32_t num_t, uint32_t num_n) {
  const uint32_t per_group = kTileGroup * num_n, g = i / per_group, r = i - g * per_group;
  const uint32_t rows = min((uint32_t)kTileGroup, num_t - g * kTileGroup), n = r / rows;
  return {(int)(g * kTileGroup + r - n * rows) * 2 * kTileT, (int)n};
}

// First weight rows of a tile's two halves.
template <bool GATED>
__device__ __forceinline__ int half_row(const GemmArgs &a, int n, int half) {
  return GATED ? half * a.N + n * kHalfW : n * kTileW + half * kHalfW;
}

struct GemmMaps {
  CUtensorMap a, w, out;
};

template <bool GATED, bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1)
    fp8_gemm_tile_kernel(const GemmArgs a, const __grid_constant__ GemmMaps maps, int num_t, int num_n,
                         int splits) {
  extern __shared__ __align__(1024) uint8_t raw[];
  TileSmem<GATED> &sm = *reinterpret_cast<TileSmem<GATED> *>(raw);
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int all_k = a.K / kBlockK;
  const uint32_t tiles = (uint32_t)num_t * (uint32_t)num_n;  // at most 2^29
  // rank in the pair, the pair's first rank in the cluster; the tiles of the
  // pair (SPLIT: one, shared by the cluster's pairs) and its scale blocks
  const uint32_t rank = cluster_rank() & 1u, base = SPLIT ? cluster_rank() & ~1u : 0u;
  const uint32_t first = SPLIT ? blockIdx.x / (2u * (uint32_t)splits) : blockIdx.x >> 1;
  const uint32_t pairs = SPLIT ? tiles : gridDim.x >> 1;
  const int k_lo = SPLIT ? all_k * (int)(base >> 1) / splits : 0;
  const int num_k = (SPLIT ? all_k * (int)((base >> 1) + 1) / splits : all_k) - k_lo;
  const int my_t = (int)rank * kTileT;  // this CTA's tokens within the pair's

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.a);
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.out);
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], 2 * kSumWarps);  // of both CTAs (the first CTA's counts)
      mbar_init(&sm.scale_full[i], 32);
      mbar_init(&sm.scale_empty[i], kSumWarps);
    }
    mbar_init(&sm.drain, 1);
    VG_GEMM_NEVER_INIT(sm);
    fence_mbar_init();
    sm.failed = 0;
  }
  if (warp == 1) tmem_alloc<true>(&sm.tmem, 512);
  // Launched with programmatic dependent launch: nothing but L2 prefetches of
  // the first weight stages before the previous grid has finished.
  if (warp == 3 && lane < kTileStages && lane < num_k) {
    const Tile t = tile_at(first, num_t, num_n);
    tma_prefetch_2d(&maps.w, (k_lo + lane) * kBlockK, half_row<GATED>(a, t.n, (int)rank));
  }
  tcgen05_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers are initialised
  tcgen05_fence_after();
  const uint32_t tmem = sm.tmem;
  pdl_wait();
  pdl_launch_dependents();
  uint32_t issued = 0;  // stages this CTA has filled (warp 0)

  if (warp < 4) {
    regs_decrease<kServiceRegs>();
    if (warp == 0) {
      uint32_t it = 0, s = 0, lap = 0;
      bool ok = true;
      for (uint32_t i = first; i < tiles && ok; i += pairs) {
        const Tile t = tile_at(i, num_t, num_n);
        const int r0 = half_row<GATED>(a, t.n, (int)rank);
        for (int kb = 0; kb < num_k; ++kb, ++it) {
          if (lap > 0 && !(ok = warp_wait_phase(&sm.empty[s], (lap - 1) & 1, &sm.failed))) break;
          if (elect_lane()) {
            if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * kTileStageBytes);
            uint8_t *p = sm.stage[s];
            const uint32_t bar = cluster_addr(&sm.full[s], base);
            tma_load_2d_pair(p, &maps.a, (k_lo + kb) * kBlockK, t.t0 + my_t, bar);
            tma_load_2d_pair(p + kTileT * kBlockK, &maps.w, (k_lo + kb) * kBlockK, r0, bar);
          }
          __syncwarp();
          ++issued;
          if (++s == kTileStages) s = 0, ++lap;
        }
      }
      // The last stages are released in both CTAs by products that the first
      // one issued: neither CTA may end before these arrivals have landed.
      for (uint32_t i = it < kTileStages ? 0 : it - kTileStages; i < it && ok; ++i)
        ok = warp_wait_phase(&sm.empty[i % kTileStages], (i / kTileStages) & 1, &sm.failed);
    } else if (warp == 1 && rank == 0) {
      constexpr uint32_t desc = product_desc(2 * kTileT, kTileW);
      uint32_t it = 0, s = 0, lap = 0;
      bool ok = true;
      for (uint32_t i = first; i < tiles && ok; i += pairs)
        for (int kb = 0; kb < num_k; ++kb, ++it) {
          const uint32_t b = it & 1;
          // Operands staged and accumulator free: half of the lanes wait for
          // either (one after the other would put both waits' latencies, some
          // 130 cycles each even when nothing is left to wait for, before
          // every block's products).
          const bool odd = lane & 1;
          if (!(ok = __all_sync(0xFFFFFFFFu, (odd && it < 2) ||
                                                 wait_phase(odd ? &sm.acc_empty[b] : &sm.full[s],
                                                            odd ? (it / 2 - 1) & 1 : lap & 1, &sm.failed))))
            break;
          if (VG_GEMM_FORCED_TIMEOUT(sm, it == 0)) {
            sm.failed = 1;
            ok = false;
            break;
          }
          tcgen05_fence_after();
          if (elect_lane()) {
            const uint64_t da = operand_desc(smem_u32(sm.stage[s]));
            const uint64_t dw = operand_desc(smem_u32(sm.stage[s] + kTileT * kBlockK));
#pragma unroll
            for (int k = 0; k < kBlockK / 32; ++k)
              mma_e4m3<true>(tmem + b * kTileW, da + 2 * k, dw + 2 * k, desc, k > 0);
            mma_commit_pair(&sm.acc_full[b], base);
            mma_commit_pair(&sm.empty[s], base);
          }
          __syncwarp();
          if (++s == kTileStages) s = 0, ++lap;
        }
      // Nothing is in flight once this arrives (at once, unless a wait gave up).
      if (elect_lane()) mma_commit<true>(&sm.drain);
      __syncwarp();
      (void)mbar_wait_bounded(&sm.drain, 0);
    } else if (warp == 2) {
      // Scales go straight to shared memory, in groups of eight blocks of a
      // tile (measured with two blocks prefetched in registers: their L2
      // latency, not the products, set the pace, 1980 instead of 2800 TFLOP/s;
      // a group takes one wait and one release of the summing warps, not
      // eight).
      uint32_t g = 0;  // groups so far
      bool ok = true;
      for (uint32_t i = first; i < tiles && ok; i += pairs) {
        const Tile t = tile_at(i, num_t, num_n);
        const int r = half_row<GATED>(a, t.n, lane & 1), row = t.t0 + my_t + lane;
        const bool w_live = r < (GATED ? 2 : 1) * a.N;
        const float *pw = a.w_scale + (w_live ? (int64_t)(r / kBlockK) * all_k + k_lo : 0);
        const float *pa = a.a_scale + k_lo * a.a_bs;
        for (int kb = 0; kb < num_k; kb += kScaleSlots, ++g) {
          if (g >= 2 && !(ok = warp_wait_phase(&sm.scale_empty[g & 1], (g / 2 - 1) & 1, &sm.failed))) break;
          const int n = min(kScaleSlots, num_k - kb);
          for (int x = 0; x < n; ++x) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool live = row + 32 * j < a.T;
              const float *p = pa + (live ? (row + 32 * j) * a.a_ts + (kb + x) * a.a_bs : 0);
              copy_async4(&sm.sa[g & 1][x][lane + 32 * j], p,
                          live && VG_ACCESS_OK(g_gemm_status, p, 4, a.a_scale, a_scale_extent(a)));
            }
            if (lane < 2) {
              const float *p = pw + (w_live ? kb + x : 0);
              copy_async4(&sm.sw[g & 1][x][lane], p,
                          w_live && VG_ACCESS_OK(g_gemm_status, p, 4, a.w_scale, w_scale_extent<GATED>(a)));
            }
          }
          copy_async_arrive(&sm.scale_full[g & 1]);
        }
      }
      copy_async_wait_all();
    }
  } else {
    regs_increase<kSumRegs>();
    const int quarter = warp & 3, part = (warp - 4) >> 2;  // lanes, columns of each half
    const int row = quarter * 32 + lane;
    uint8_t *box = sm.out[warp - 4];
    const uint32_t release = cluster_addr(&sm.acc_empty[0], base);
    uint32_t it = 0, g = 0;
    int turn = 0;
    bool ok = true;
    for (uint32_t i = first; i < tiles; i += pairs, turn ^= 1) {
      float2 acc[2][kPart / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < kPart / 2; ++j) acc[h][j] = make_float2(0.f, 0.f);
      for (int kb = 0; kb < num_k; ++kb, ++it) {
        const uint32_t b = it & 1, x = (uint32_t)kb % kScaleSlots;
        if (x == 0 && !(ok = warp_wait_phase(&sm.scale_full[g & 1], (g >> 1) & 1, &sm.failed))) break;
        const float s = sm.sa[g & 1][x][row];
        const float2 w = *reinterpret_cast<const float2 *>(sm.sw[g & 1][x]);
        if (x == kScaleSlots - 1 || kb == num_k - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.scale_empty[g & 1]);
          ++g;
        }
        if (!(ok = warp_wait_phase(&sm.acc_full[b], (it >> 1) & 1, &sm.failed))) break;
        tcgen05_fence_after();
        const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16) + b * kTileW + part * kPart;
        uint32_t v[kPart];
        tmem_load(base, v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h > 0) tmem_load(base + kHalfW, v);
          const float sh = s * (h ? w.y : w.x);
          const float2 sc = make_float2(sh, sh);
          tmem_load_wait(v);
          if (h > 0) {  // all read: the products of the block after next may start
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(release + 8 * b);
          }
#pragma unroll
          for (int j = 0; j < kPart / 2; ++j)
            acc[h][j] = f2_fma(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])),
                               sc, acc[h][j]);
        }
      }
      if (!(GATED && !SPLIT) && !ok) break;
      if constexpr (SPLIT) {
        // Partial sums to shared memory (the last products are done, so nothing
        // reads the stages), 16-byte chunks swizzled by the row.
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int q = 0; q < kPart / 4; ++q) {
            const float2 x = acc[h][2 * q], y = acc[h][2 * q + 1];
            const int c = h * (kHalfW / 4) + part * (kPart / 4) + q;
            sm.part[row][c ^ (row & 7)] = make_float4(x.x, x.y, y.x, y.y);
          }
        break;
      }

      const Tile t = tile_at(i, num_t, num_n);
      const int t0 = t.t0 + my_t + quarter * 32;  // this warp's first token
      if constexpr (!GATED) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // a box of 32 columns, 64 bytes a row
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 *x = &acc[h][q * 4];
            *reinterpret_cast<uint4 *>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) =
                make_uint4(pack_bf16x2_rn(x[0].x, x[0].y), pack_bf16x2_rn(x[1].x, x[1].y),
                           pack_bf16x2_rn(x[2].x, x[2].y), pack_bf16x2_rn(x[3].x, x[3].y));
          }
          fence_proxy_async_smem();
          __syncwarp();
          const int n = half_row<false>(a, t.n, h) + part * kPart;
          if (lane == 0) {
            if (t0 < a.T && n < a.N) tma_store_2d(&maps.out, box, n, t0);
            tma_store_commit();
          }
        }
      } else {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < kPart / 2; ++j) {
          float2 &g = acc[0][j];
          g = make_float2(silu_mul(g.x, acc[1][j].x), silu_mul(g.y, acc[1][j].y));
          m = fmax3(m, fabsf(g.x), fabsf(g.y));
        }
        sm.amax[turn][part][row] = m;
        // all of the warps leave together where a wait of one gave up
        if (named_sync_or(1, kSumWarps * 32, !ok)) break;
#pragma unroll
        for (int x = 0; x < kSumWarps / 4; ++x) m = fmaxf(m, sm.amax[turn][x][row]);
        const float s = group_scale(m, a.ue8m0 != 0);
        const float2 r = make_float2(__frcp_rn(s), __frcp_rn(s));
        if (lane == 0) tma_store_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // a box of 32 columns, 32 bytes a row
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = f2_mul(acc[0][q * 8 + 2 * k], r), y = f2_mul(acc[0][q * 8 + 2 * k + 1], r);
            w[k] = cvt_e4m3x2(x.x, x.y) | (cvt_e4m3x2(y.x, y.y) << 16);
          }
          *reinterpret_cast<uint4 *>(box + lane * 32 + ((q ^ ((lane >> 2) & 1)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (t0 < a.T) tma_store_2d(&maps.out, box, t.n * kHalfW + part * kPart, t0);
          tma_store_commit();
        }
        if (part == 0 && t0 + lane < a.T) {
          float *p = a.scale + (int64_t)(t0 + lane) * a.s_ts + (int64_t)t.n * a.s_gs;
          if (VG_ACCESS_OK(g_gemm_status, p, 4, a.scale, gemm_scale_extent(a))) *p = s;
        }
      }
    }
    if (lane == 0) tma_store_wait_read<0>();
  }

  __syncthreads();
  if (sm.failed && warp == 0 && lane == 0) {  // the pair's copies in flight end here
    atomicOr(&g_gemm_status, kErrWaitTimeout);
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
    // a warp a token row, a lane four columns of either half.
    const Tile t = tile_at(first, num_t, num_n);
    for (int row = (int)(base >> 1) + warp * splits; row < kTileT; row += kTileThreads / 32 * splits) {
      const int64_t token = t.t0 + my_t + row;
      if (token >= a.T) break;
      float4 c[2] = {};
      for (int x = 0; x < splits; ++x)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 p = ld_cluster4(cluster_addr(&sm.part[row][(h * (kHalfW / 4) + lane) ^ (row & 7)],
                                                    2u * (uint32_t)x + rank));
          c[h] = make_float4(c[h].x + p.x, c[h].y + p.y, c[h].z + p.z, c[h].w + p.w);
        }
      if constexpr (!GATED) {
#pragma unroll
        for (int h = 0; h < 2; ++h) store_out4(a, token, half_row<false>(a, t.n, h) + 4 * lane, c[h]);
      } else {
        store_gated4(a, token, t.n, lane, c[0], c[1]);
      }
    }
    cluster_sync();  // nobody reads this CTA's sums any more
  }
}

// ----------------------------------------------------------- stream kernel
//
// For few tokens, where the weight's bytes are the cost.  Operands change
// places: a CTA's tile is 128 weight rows (gated: 64 gate rows and the same 64
// up rows) x TN tokens, so that sixteen tokens fill a product, and K is split
// over a cluster, as many ways as fill the GPU.  The sums stay in fp32
// registers, a thread a weight row; at the end each CTA puts its partial sums
// in shared memory and the cluster adds them in a fixed order, every CTA some
// of the tokens, a warp a token: for the gated form the two CTAs of a scale
// group (64 columns each) meet there too.
//   warp 0: TMA   warp 1: products   warp 2: scales   warps from 4 on: sums
// Up to 64 tokens two CTAs share an SM (each asks for more than a third of its
// shared memory and for at most half of its tensor memory, so no allocation
// ever waits).
//
// Bound by the weight's bytes: 57344 x 8192, one token, 71 us (0.97 of the copy
// rate); gated 14336 x 4096, one token, 19.3 us (0.90); 57 tokens x 28672 x
// 8192 gated 86 us (0.80: 448 CTAs are a wave and a half).  Small products are
// bound by a call's fixed 3.5 us (6144 x 4096, one token: 6.5 us, 0.57).

constexpr int kMaxSplit = 8;

// Warps that sum: four, or for 128 tokens eight of 64 tokens each, over four
// accumulators (four warps took longer for a block's sums than its products do:
// 100 x 4096 x 14336 18.4 -> 17.5 us, 128 x 8192 x 8192 21.3 -> 20.0).
template <int TN>
constexpr int kStreamSums = TN <= 64 ? 4 : 8;
template <int TN>
constexpr int kStreamThreads = 128 + 32 * kStreamSums<TN>;

template <int TN>
struct StreamSmem {
  static constexpr int kStageBytes = (kHalfW + TN) * kBlockK;
  static constexpr int kStages = TN <= 32 ? 5 : (TN == 64 ? 4 : 6);
  static constexpr int kBufs = 4;              // accumulators
  static constexpr int kColumns = kBufs * TN;  // of tensor memory
  union {
    uint8_t stage[kStages][kStageBytes];
    float part[TN][kHalfW];  // partial sums, once the products are done
  };
  float sa[kScaleSlots][TN];
  float sw[kScaleSlots][2];
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[kBufs], acc_empty[kBufs], scale_full[kScaleSlots], scale_empty[kScaleSlots], drain;
  uint32_t tmem;
  uint32_t failed;
  VG_GEMM_NEVER
};

template <bool GATED, int TN>
__global__ void __launch_bounds__(kStreamThreads<TN>, TN <= 64 ? 2 : 1)
    fp8_gemm_stream_kernel(const GemmArgs a, const __grid_constant__ GemmMaps maps, int splits,
                           bool w_once) {
  extern __shared__ __align__(1024) uint8_t raw[];
  using Smem = StreamSmem<TN>;
  Smem &sm = *reinterpret_cast<Smem *>(raw);
  constexpr int kStages = Smem::kStages, kBufs = Smem::kBufs;
  const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
  const int num_k = a.K / kBlockK;
  const int rank = (int)cluster_rank(), ctas = GATED ? 2 * splits : splits;
  const int tile = (int)blockIdx.x / ctas, split = GATED ? rank >> 1 : rank;
  // first weight rows of the tile's two halves, first token, scale blocks
  const int r0 = tile * kHalfW + (GATED ? (rank & 1) * (kHalfW / 2) : 0);
  const int r1 = GATED ? a.N + r0 : r0 + kHalfW / 2;
  const int t0 = (int)blockIdx.y * TN;
  const int k0 = num_k * split / splits, k1 = num_k * (split + 1) / splits;

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&maps.a);
    prefetch_tensormap(&maps.w);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], kStreamSums<TN>);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(&sm.scale_full[i], 32);
      mbar_init(&sm.scale_empty[i], kStreamSums<TN>);
    }
    mbar_init(&sm.drain, 1);
    VG_GEMM_NEVER_INIT(sm);
    fence_mbar_init();
    sm.failed = 0;
  }
  if (warp == 1) tmem_alloc<false>(&sm.tmem, Smem::kColumns);
  // Launched with programmatic dependent launch: nothing but L2 prefetches of
  // the first weight stages before the previous grid has finished.
  if (warp == 3 && lane < 2 * kStages && blockIdx.y == 0) {
    const int kb = k0 + (lane >> 1);
    if (kb < k1) tma_prefetch_2d(&maps.w, kb * kBlockK, lane & 1 ? r1 : r0);
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
        if (w_once) {
          tma_load_2d_hint(p, &maps.w, kb * kBlockK, r0, &sm.full[s], policy);
          tma_load_2d_hint(p + kHalfW / 2 * kBlockK, &maps.w, kb * kBlockK, r1, &sm.full[s], policy);
        } else {
          tma_load_2d(p, &maps.w, kb * kBlockK, r0, &sm.full[s]);
          tma_load_2d(p + kHalfW / 2 * kBlockK, &maps.w, kb * kBlockK, r1, &sm.full[s]);
        }
        tma_load_2d(p + kHalfW * kBlockK, &maps.a, kb * kBlockK, t0, &sm.full[s]);
      }
      __syncwarp();
      ++issued;
      if (++s == kStages) s = 0, ++lap;
    }
  } else if (warp == 1) {
    constexpr uint32_t desc = product_desc(kHalfW, TN);
    int s = 0, lap = 0;
    for (int kb = k0; kb < k1; ++kb) {
      const int it = kb - k0, b = it % kBufs;
      const bool odd = lane & 1;  // half of the lanes wait for either barrier
      if (!__all_sync(0xFFFFFFFFu, (odd && it < kBufs) ||
                                       wait_phase(odd ? &sm.acc_empty[b] : &sm.full[s],
                                                  odd ? (it / kBufs - 1) & 1 : lap & 1, &sm.failed)))
        break;
      if (VG_GEMM_FORCED_TIMEOUT(sm, it == 0)) {
        sm.failed = 1;
        break;
      }
      tcgen05_fence_after();
      if (elect_lane()) {
        const uint64_t dw = operand_desc(smem_u32(sm.stage[s]));
        const uint64_t da = operand_desc(smem_u32(sm.stage[s] + kHalfW * kBlockK));
#pragma unroll
        for (int k = 0; k < kBlockK / 32; ++k)
          mma_e4m3<false>(tmem + b * TN, dw + 2 * k, da + 2 * k, desc, k > 0);
        mma_commit<false>(&sm.acc_full[b]);
        mma_commit<false>(&sm.empty[s]);
      }
      __syncwarp();
      if (++s == kStages) s = 0, ++lap;
    }
    if (elect_lane()) mma_commit<false>(&sm.drain);
    __syncwarp();
    (void)mbar_wait_bounded(&sm.drain, 0);
  } else if (warp == 2) {
    const int r = lane & 1 ? r1 : r0;
    const bool w_live = r < (GATED ? 2 : 1) * a.N;
    const float *pw = a.w_scale + (w_live ? (int64_t)(r / kBlockK) * num_k : 0);
    int s = 0, lap = 0;
    for (int kb = k0; kb < k1; ++kb) {
      if (lap > 0 && !warp_wait_phase(&sm.scale_empty[s], (lap - 1) & 1, &sm.failed)) break;
#pragma unroll
      for (int j = 0; j < (TN + 31) / 32; ++j) {
        const int t = lane + 32 * j;
        const bool live = t0 + t < a.T && t < TN;
        const float *p = a.a_scale + (live ? (t0 + t) * a.a_ts + kb * a.a_bs : 0);
        if (t < TN)
          copy_async4(&sm.sa[s][t], p,
                      live && VG_ACCESS_OK(g_gemm_status, p, 4, a.a_scale, a_scale_extent(a)));
      }
      if (lane < 2) {
        const float *p = pw + (w_live ? kb : 0);
        copy_async4(&sm.sw[s][lane], p,
                    w_live && VG_ACCESS_OK(g_gemm_status, p, 4, a.w_scale, w_scale_extent<GATED>(a)));
      }
      copy_async_arrive(&sm.scale_full[s]);
      if (++s == kScaleSlots) s = 0, ++lap;
    }
    copy_async_wait_all();
  } else if (warp >= 4) {
    constexpr int kCols = TN * 4 / kStreamSums<TN>;  // tokens a thread sums
    const int quarter = warp & 3, row = quarter * 32 + lane, col0 = (warp - 4) / 4 * kCols;
    float2 acc[kCols / 2];
#pragma unroll
    for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    for (int kb = k0; kb < k1; ++kb) {
      const int it = kb - k0, b = it % kBufs, x = it % kScaleSlots;
      const bool odd = lane & 1;  // half of the lanes wait for either barrier
      if (!warp_wait_phase(odd ? &sm.scale_full[x] : &sm.acc_full[b],
                           (odd ? it / kScaleSlots : it / kBufs) & 1, &sm.failed))
        break;
      tcgen05_fence_after();
      constexpr int kLoad = TN == 128 ? 32 : 16;  // (32 would spill at two CTAs an SM)
#pragma unroll
      for (int c = 0; c < kCols / kLoad; ++c) {
        uint32_t v[kLoad];
        tmem_load(tmem + ((uint32_t)(quarter * 32) << 16) + b * TN + col0 + c * kLoad, v);
        const float w = sm.sw[x][quarter >> 1];  // while the sums are on their way
        const float2 w2 = make_float2(w, w);
        float2 s[kLoad / 2];
#pragma unroll
        for (int j = 0; j < kLoad / 4; ++j) {
          const float4 sa = *reinterpret_cast<const float4 *>(&sm.sa[x][col0 + c * kLoad + 4 * j]);
          s[2 * j] = f2_mul(make_float2(sa.x, sa.y), w2);
          s[2 * j + 1] = f2_mul(make_float2(sa.z, sa.w), w2);
        }
        tmem_load_wait(v);
        if (c == kCols / kLoad - 1) {  // all read
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.acc_empty[b]);
            mbar_arrive(&sm.scale_empty[x]);
          }
        }
#pragma unroll
        for (int j = 0; j < kLoad / 2; ++j) {
          float2 &y = acc[c * kLoad / 2 + j];
          y = f2_fma(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), s[j], y);
        }
      }
    }
    // The last block's products are done, so nothing reads the stages.
    if (!sm.failed) {
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) {
        sm.part[col0 + 2 * j][row] = acc[j].x;
        sm.part[col0 + 2 * j + 1][row] = acc[j].y;
      }
    }
  }

  __syncthreads();
  pdl_launch_dependents();  // the loads are done
  if (sm.failed && warp == 0 && lane == 0) {  // copies in flight end here
    atomicOr(&g_gemm_status, kErrWaitTimeout);
    for (int it = issued < kStages ? 0 : issued - kStages; it < issued; ++it)
      (void)mbar_wait_bounded(&sm.full[it % kStages], (it / kStages) & 1);
  }
  cluster_sync();  // every CTA's partial sums are in place
  __syncwarp();
  if (warp == 1) tmem_dealloc<false>(tmem, Smem::kColumns);

  const int tokens = min(TN, a.T - t0);
  for (int j = rank + warp * ctas; j < tokens; j += kStreamThreads<TN> / 32 * ctas) {
    const int64_t t = t0 + j;
    if constexpr (!GATED) {
      float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = 0; x < splits; ++x) {
        const float4 p = ld_cluster4(cluster_addr(&sm.part[j][4 * lane], (uint32_t)x));
        c = make_float4(c.x + p.x, c.y + p.y, c.z + p.z, c.w + p.w);
      }
      store_out4(a, t, r0 + 4 * lane, c);
    } else {
      // lane: columns 4 lane .. of the group, from the half that has them
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
      const int col = (4 * lane) & (kHalfW / 2 - 1);
      for (int x = 0; x < splits; ++x) {
        const uint32_t from = 2 * (uint32_t)x + (uint32_t)(lane >> 4);
        const float4 p = ld_cluster4(cluster_addr(&sm.part[j][col], from));
        const float4 q = ld_cluster4(cluster_addr(&sm.part[j][kHalfW / 2 + col], from));
        g = make_float4(g.x + p.x, g.y + p.y, g.z + p.z, g.w + p.w);
        u = make_float4(u.x + q.x, u.y + q.y, u.z + q.z, u.w + q.w);
      }
      store_gated4(a, t, tile, lane, g, u);
    }
  }
  cluster_sync();  // nobody reads this CTA's sums any more
}

// ------------------------------------------------------------------- host

template <bool GATED, bool SPLIT>
cudaError_t launch_tile(const GemmArgs &a, int splits, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> opted_in{0};
  const cudaError_t e = opt_in_once(opted_in, (const void *)fp8_gemm_tile_kernel<GATED, SPLIT>);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  GemmMaps maps;
  if (!make_map(&maps.a, u8, 1, a.a, a.T, a.K, kTileT, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&maps.w, u8, 1, a.w, (GATED ? 2 : 1) * (int64_t)a.N, a.K, kHalfW, kBlockK,
                CU_TENSOR_MAP_SWIZZLE_128B) ||
      !(GATED ? make_map(&maps.out, u8, 1, a.q, a.T, a.N, 32, kPart, CU_TENSOR_MAP_SWIZZLE_32B)
              : make_map(&maps.out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.out, a.T, a.N, 32, kPart,
                         CU_TENSOR_MAP_SWIZZLE_64B)))
    return cudaErrorInvalidValue;
  const int num_t = (a.T + 2 * kTileT - 1) / (2 * kTileT);
  const int num_n = GATED ? a.N / kHalfW : (a.N + kTileW - 1) / kTileW;
  const int64_t tiles = (int64_t)num_t * num_n;
  const int64_t pairs = SPLIT ? tiles * splits : (tiles < sms / 2 ? tiles : sms / 2);
  return launch_pdl_cluster(fp8_gemm_tile_kernel<GATED, SPLIT>, dim3((unsigned)(2 * pairs)),
                            SPLIT ? 2 * splits : 2, dim3(kTileThreads), sizeof(TileSmem<GATED>), s, a, maps,
                            num_t, num_n, splits);
}

template <bool GATED, int TN>
cudaError_t launch_stream(const GemmArgs &a, int splits, cudaStream_t s) {
  static std::atomic<uint64_t> opted_in{0};
  const cudaError_t e = opt_in_once(opted_in, (const void *)fp8_gemm_stream_kernel<GATED, TN>);
  if (e != cudaSuccess) return e;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  GemmMaps maps;
  if (!make_map(&maps.a, u8, 1, a.a, a.T, a.K, TN, kBlockK, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map(&maps.w, u8, 1, a.w, (GATED ? 2 : 1) * (int64_t)a.N, a.K, kHalfW / 2, kBlockK,
                CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  maps.out = maps.a;  // not used: the sums are stored by threads
  const int ctas = GATED ? 2 * splits : splits;
  // A weight that one token tile reads once and that would fill more than a
  // quarter of L2 passes it by (117 MB, one token: 21.2 -> 19.7 us; 67 MB: 12.9
  // -> 11.8; 25 MB, which stays in L2 from call to call: 6.4 -> 6.8).
  const bool w_once = a.T <= TN && (GATED ? 2 : 1) * (int64_t)a.N * a.K > 32 << 20;
  const dim3 grid((unsigned)((a.N + kHalfW - 1) / kHalfW * ctas), (unsigned)((a.T + TN - 1) / TN));
  return launch_pdl_cluster(fp8_gemm_stream_kernel<GATED, TN>, grid, ctas, dim3(kStreamThreads<TN>),
                            sizeof(StreamSmem<TN>), s, a, maps, splits, w_once);
}

template <bool GATED>
cudaError_t launch_form(const GemmArgs &a, const GemmPlan &p, int sms, cudaStream_t s) {
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

// Which kernel, and its split, by an estimate of either one's time, in
// microseconds (fitted on GB300 to T = 1..1024, N = 1024..57344, K =
// 4096..28672; over those the choice was within 10 % of the best one at all
// sizes but one: 700 x 1024 x 4096 takes 64-token tiles, 14.0 us, where
// 128-token tiles take 12.4):
//   tile kernel    a wave of pairs: 0.42 per scale block of its share of K, and
//                  4.4 (one share) .. 9.5 (four) for start, end and the sum of
//                  the shares
//   stream kernel  a wave of CTAs: 3.5 and 0.15 for each CTA of a cluster, and
//                  0.27 (16 tokens) .. 0.44 (128) per block of its split or the
//                  weight's bytes at 6.3 TB/s (two thirds of that again for
//                  every further token tile, which reads the weight from L2),
//                  whichever is longer, with a fifth of the other
// Clusters do not fill every SM, and a second wave costs as much as the first
// (6144 x 4096, one token: five ways, 240 CTAs, 6.5 us; six ways, 288 of 304
// slots, 10.3 us; 256 x 4096 x 14336 in tiles: three shares, 96 CTAs, 24.9 us,
// four, 128, 40.7), so a wave is taken as the part of the slots that clusters
// of that size were seen to fill.  Stream splits are powers of two: others
// pack worse (64 x 4096 x 4096: four ways 7.5 us, five 9.4).
GemmPlan plan_gemm(int64_t T, int64_t N, int64_t K, bool gated, int sms) {
  GemmPlan p;
  const int64_t blocks = K / kBlockK, rows = (N + kHalfW - 1) / kHalfW * (gated ? 2 : 1);
  const auto waves_of = [](int64_t n, int64_t slots) { return (double)((n + slots - 1) / slots); };
  const auto part = [](int64_t slots, int64_t percent) { return slots < 8 ? slots : slots * percent / 100; };
  const int64_t pairs =
      (T + 2 * kTileT - 1) / (2 * kTileT) * (gated ? N / kHalfW : (N + kTileW - 1) / kTileW);
  const int64_t pair_slots = sms < 2 ? 1 : sms / 2;
  static const double kFixed[4] = {4.4, 7.0, 9.0, 9.5};
  static const int kFill[4] = {100, 90, 64, 64};
  double best = 1e30;
  for (int s = 1; s <= 4 && s <= blocks; ++s) {
    const double waves = waves_of(pairs * s, part(pair_slots, kFill[s - 1]));
    if (s > 1 && waves > 1) break;
    const double cost = waves * (kFixed[s - 1] + 0.42 * (double)((blocks + s - 1) / s));
    if (cost < best) {
      best = cost;
      p.splits = s;
    }
  }
  // one token tile, or for more than 64 tokens tiles of 64 or 128
  const int smallest = T <= 16 ? 16 : (T <= 32 ? 32 : 64);
  for (int tn = smallest; tn <= (T <= 64 ? smallest : 128); tn *= 2) {
    const int64_t token_tiles = (T + tn - 1) / tn, tiles = rows * token_tiles;
    if (token_tiles > 65535) continue;
    const int64_t slots = (int64_t)sms * (tn <= 64 ? 2 : 1);
    const double per_block = tn <= 32 ? 0.27 : (tn == 64 ? 0.36 : 0.44);
    const double bytes = (double)rows * kHalfW * (double)K * (1.0 + (double)(token_tiles - 1) * 2.0 / 3.0);
    for (int s = 1; s <= (gated ? kMaxSplit / 2 : kMaxSplit) && s <= blocks; s *= 2) {
      const bool big = tn == 128 && s * (gated ? 2 : 1) == 8;  // eight SMs a cluster
      const double waves = waves_of(tiles * s, part(slots, big ? 64 : 85));
      const double chain = (double)((blocks + s - 1) / s) * per_block;
      const double traffic = bytes / waves / 6.3e6;
      const double fixed = 3.5 + 0.15 * (double)(s * (gated ? 2 : 1));
      const double cost = waves * (fixed + (chain > traffic ? chain + 0.2 * traffic : traffic + 0.2 * chain));
      if (cost < best) {
        best = cost;
        p.tn = tn;
        p.splits = s;
      }
    }
  }
  return p;
}

cudaError_t launch_fp8_gemm(const GemmArgs &a, bool gated, int sms, cudaStream_t s) {
  const GemmPlan p = plan_gemm(a.T, a.N, a.K, gated, sms);
  return gated ? launch_form<true>(a, p, sms, s) : launch_form<false>(a, p, sms, s);
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
