// qk_norm_rope.cu -- per-head RMSNorm of Q and K, then the rotary embedding,
// in place, one pass over HBM.
//
// Implements "QK Norm + RoPE (enable_qk_norm_rope_fusion)" of the "Fusion
// torch.compile passes" page: split QKV -> per-head RMSNorm of the Q heads
// (q weight) and K heads (k weight) -> rotary embedding, as one kernel.  A
// qkv row is [Q heads | K heads | V heads], D columns a head; V is not
// touched.  The rotation reads an fp32 cos/sin cache [max_pos, D] (cos in
// the first D/2 columns, sin in the rest) at each token's position and
// turns the pairs (i, i + D/2) (neox) or (2i, 2i + 1) (gptj).
//
// Layout: one token per CTA (blockIdx.y splits very many heads); a head is
// D/8 chunks of 8 bf16 held by G = D/16 consecutive lanes, lane l holding
// chunks l and l + G -- so a neox pair (i, i + D/2) lives in one lane, and a
// gptj pair inside one chunk.  Each lane keeps t = x * w (exact in fp32).
//
// Arithmetic (fp32): the head's sum of squares in fp32 (longest path 11
// roundings of non-negative terms: <= 11u), inv = rsqrt(sum/D + eps)
// (<= 10u with rsqrtf's 2 ulps), o = t_a c -/+ t_b s by Kahan's FMA
// algorithm for a*c - b*s (q = b*s, e = fma(b, s, -q), f = fma(a, c, -q),
// o = f - e: within 2 ulps of the exact value even under cancellation), and
// p = o * inv rounded once to bf16.  So p is within ~15u (2^-20 relative) of
// the exact result, and its bf16 differs from the correctly rounded one only
// where the exact value lies that close to a bf16 midpoint, by one ulp.
//
// Two further forms, in a kernel of their own.  AXES: pair i turns by the position
// on its axis, positions[axis(i), t]; each lane takes its pairs' values from
// the rows of their axes (measured against a row put together in shared
// memory once per CTA: its barrier couples the warps, 16411 tokens of 32 + 8
// heads 84 us).  APPEND: Q in place, K (normed, rotated) and V go
// to their slot of a paged cache instead, as bf16 or as e4m3(value / scale)
// from the fp32 value, so that the qkv row is read once and K and V are
// written once.  A rotation without a norm takes weights of one and y = 1, and
// keeps infinities (NaN only where IEEE arithmetic gives it); FP8 caches
// saturate them.
#include "common.cuh"
#include "launch.h"
#include "row_norm.cuh"

namespace vg {

// Status word of this translation unit's kernels: kErrBadPosition when a
// position lies outside [0, max_pos) (that head is left as it was).
__device__ uint32_t g_rope_status;

namespace {

__device__ __forceinline__ void load8f(const float *p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void load4f(const float *p, float (&v)[8], int at) {
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
  v[at] = a.x; v[at + 1] = a.y; v[at + 2] = a.z; v[at + 3] = a.w;
}

// Two elements of a*c -/+ b*s (Kahan), packed; a zero keeps the plain
// expression's sign, and so does an infinite b, whose error term is NaN (the
// comparison is false for it).  nb = -b for the minus form.
__device__ __forceinline__ float2 kahan2x(float2 a, float2 c, float2 nb, float2 s) {
  const float2 q = f2_mul(nb, s);
  const float2 e = f2_fma(nb, s, make_float2(-q.x, -q.y));
  const float2 f = f2_fma(a, c, q);
  const float2 o = f2_add(f, e);
  return make_float2(fabsf(e.x) > 0.f ? o.x : f.x, fabsf(e.y) > 0.f ? o.y : f.y);
}

// The plain form, in place: one head a lane group, weights and one axis.  A
// kernel of its own: as an instance of the one below its gptj rotation took 3 %
// longer (32768 tokens of 32 + 8 heads 108.2 us against 104.7; 4096 tokens 15.4
// against 14.8; neox alike).
template <int G, bool NEOX>
__global__ void __launch_bounds__(512) qk_norm_rope_kernel(const QkArgs a) {
  constexpr int D = G * 16;
  const int lane = threadIdx.x & 31;
  const int l = lane & (G - 1);
  const int64_t t = blockIdx.x;
  const int h = ((int)blockIdx.y * (int)(blockDim.x >> 5) + (int)(threadIdx.x >> 5)) * (32 / G) + lane / G;
  // Launched with programmatic dependent launch: nothing in global memory
  // before the previous grid has finished, except that the CTA's heads are
  // asked into L2 first; the next grid may be scheduled once the loads are out.
  if (threadIdx.x == 0 && (int)blockIdx.x < a.pf_ctas) {
    const int h0 = (int)blockIdx.y * (int)(blockDim.x >> 5) * (32 / G);
    const int nh = a.nh - h0 < (int)(blockDim.x >> 5) * (32 / G) ? a.nh - h0 : (int)(blockDim.x >> 5) * (32 / G);
    prefetch_l2(a.qkv + t * a.row + (int64_t)h0 * D, 2u * (uint32_t)(nh * D));
  }
  pdl_wait();
  // The head's loads do not depend on the token's position, so they go out
  // together with it (a head with a bad position is loaded but not stored);
  // only the cos/sin row waits for the position.
  const bool in_head = h < a.nh;
  uint16_t *head = a.qkv + t * a.row + (in_head ? (int64_t)h * D : 0);
  const uint16_t *w = h < a.hq ? a.qw : a.kw;
  const int64_t pos = a.pos[t];
  // chunk 0 of the lane: l (first half of the head), chunk 1: l + G
  const uint4 xa = in_head ? ld_stream(head + l * kElemsPerChunk) : make_uint4(0, 0, 0, 0);
  const uint4 xb = in_head ? ld_stream(head + (l + G) * kElemsPerChunk) : make_uint4(0, 0, 0, 0);
  const uint4 wa = in_head ? ld_keep(w + l * kElemsPerChunk) : make_uint4(0, 0, 0, 0);
  const uint4 wb = in_head ? ld_keep(w + (l + G) * kElemsPerChunk) : make_uint4(0, 0, 0, 0);
  const bool live = in_head && pos >= 0 && pos < a.max_pos;  // same for the head's lanes
  if (in_head && !live && l == 0) atomicOr(&g_rope_status, kErrBadPosition);
  pdl_launch_dependents();
  float2 ta[4], tb[4];
  float cmax;
  RowAcc acc;
  pass1_chunk<false, false>(xa, xa, wa, ta, cmax, acc);
  pass1_chunk<false, false>(xb, xb, wb, tb, cmax, acc);
  float ss = acc.ss.x + acc.ss.y;
#pragma unroll
  for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
  const float y = rsqrtf(fmaf(ss, 1.0f / (float)D, a.eps));

  // mine[0..7]: chunk 0, mine[8..15]: chunk 1; other: each element's pair
  // partner; c, s: its pair's cos and sin; submask bit k: minus sign
  float mine[16], other[16], c[16], s[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mine[2 * i] = ta[i].x;
    mine[2 * i + 1] = ta[i].y;
    mine[8 + 2 * i] = tb[i].x;
    mine[8 + 2 * i + 1] = tb[i].y;
  }
  const float *cs = a.cache + (live ? pos * D : 0);
  uint32_t submask;
  if (NEOX) {  // element k of chunk 0 pairs with element k of chunk 1: pair 8l + k
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      other[k] = mine[8 + k];
      other[8 + k] = mine[k];
    }
    float c8[8] = {}, s8[8] = {};
    if (live) {
      load8f(cs + 8 * l, c8);
      load8f(cs + D / 2 + 8 * l, s8);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c[k] = c[8 + k] = c8[k];
      s[k] = s[8 + k] = s8[k];
    }
    submask = 0x00FFu;
  } else {  // pairs (2i, 2i + 1) inside each chunk: pair 4 chunk + k / 2
#pragma unroll
    for (int k = 0; k < 16; ++k) other[k] = mine[k ^ 1];
    float c4[8] = {}, s4[8] = {};
    if (live) {
      load4f(cs + 4 * l, c4, 0);
      load4f(cs + 4 * (l + G), c4, 4);
      load4f(cs + D / 2 + 4 * l, s4, 0);
      load4f(cs + D / 2 + 4 * (l + G), s4, 4);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      c[k] = c4[k >> 1];
      s[k] = s4[k >> 1];
    }
    submask = 0x5555u;
  }

  float p[16];
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    const bool m0 = (submask >> k) & 1u, m1 = (submask >> (k + 1)) & 1u;
    const float2 o = kahan2x(make_float2(mine[k], mine[k + 1]), make_float2(c[k], c[k + 1]),
                             make_float2(m0 ? -other[k] : other[k], m1 ? -other[k + 1] : other[k + 1]),
                             make_float2(s[k], s[k + 1]));
    const float2 pp = f2_mul(o, make_float2(y, y));
    p[k] = pp.x;
    p[k + 1] = pp.y;
  }
  const uint4 oa = make_uint4(pack_bf16x2_rn(p[0], p[1]), pack_bf16x2_rn(p[2], p[3]),
                              pack_bf16x2_rn(p[4], p[5]), pack_bf16x2_rn(p[6], p[7]));
  const uint4 ob = make_uint4(pack_bf16x2_rn(p[8], p[9]), pack_bf16x2_rn(p[10], p[11]),
                              pack_bf16x2_rn(p[12], p[13]), pack_bf16x2_rn(p[14], p[15]));
  [[maybe_unused]] const uint64_t bytes = VG_ROWS(a.T) * 2ull * (uint64_t)a.row;
  if (live && VG_ACCESS_OK(g_rope_status, head + l * kElemsPerChunk, 16, a.qkv, bytes))
    st_stream(head + l * kElemsPerChunk, oa);
  if (live && VG_ACCESS_OK(g_rope_status, head + (l + G) * kElemsPerChunk, 16, a.qkv, bytes))
    st_stream(head + (l + G) * kElemsPerChunk, ob);
}

// Eight fp32 values (in registers: every index is a constant) as bf16, as
// E4M3 codes; a chunk of eight bf16 times m as E4M3 codes.
__device__ __forceinline__ uint4 bf16x8(const float *p) {
  return make_uint4(pack_bf16x2_rn(p[0], p[1]), pack_bf16x2_rn(p[2], p[3]),
                    pack_bf16x2_rn(p[4], p[5]), pack_bf16x2_rn(p[6], p[7]));
}

__device__ __forceinline__ uint2 codes8(const float *p) {
  return make_uint2(cvt_e4m3x2(p[0], p[1]) | (cvt_e4m3x2(p[2], p[3]) << 16),
                    cvt_e4m3x2(p[4], p[5]) | (cvt_e4m3x2(p[6], p[7]) << 16));
}

__device__ __forceinline__ uint2 scaled_codes(const uint4 &x, float m) {
  const float v[8] = {bf16_lo(x.x) * m, bf16_hi(x.x) * m, bf16_lo(x.y) * m, bf16_hi(x.y) * m,
                      bf16_lo(x.z) * m, bf16_hi(x.z) * m, bf16_lo(x.w) * m, bf16_hi(x.w) * m};
  return codes8(v);
}

// The element at which head kv of a token with this slot starts: the slot's
// page, the token in it, the head.  -1: the token is not appended (a padding
// token, or a slot beyond the cache, which `report` makes known).
__device__ __forceinline__ int64_t cache_place(const QkArgs &a, int64_t slot, int kv, bool report) {
  if (slot < 0) return -1;
  if (slot >= a.num_slots) {
    if (report) atomicOr(&g_rope_status, kErrBadSlot);
    return -1;
  }
  const uint32_t page = (uint32_t)slot / (uint32_t)a.page_size;
  const uint32_t in_page = (uint32_t)slot - page * (uint32_t)a.page_size;
  return (int64_t)page * a.page_stride + (int64_t)in_page * a.token_stride +
         (int64_t)kv * a.head_stride;
}

// One head's two chunks of 8 (columns 8l and 8(l + G)) to its slot of a paged
// cache.  MANY: streaming stores (a long prompt's K and V pass L2 by; measured
// 122 -> 119 us, FP8 56 -> 52); few tokens' lines stay in L2 for the attention
// that reads them next.
template <bool MANY, class V>
__device__ __forceinline__ void cache_put(const QkArgs &a, void *cache, void *o, const V &v) {
  if (!VG_ACCESS_OK(g_rope_status, o, sizeof(V), cache, sizeof(V) / 8 * a.cache_elems)) return;
  if constexpr (MANY)
    st_stream(o, v);
  else
    *static_cast<V *>(o) = v;
}

template <bool MANY>
__device__ __forceinline__ void cache_store(const QkArgs &a, void *cache, int64_t at, int l, int g,
                                            const uint4 &ca, const uint4 &cb) {
  uint16_t *o = static_cast<uint16_t *>(cache) + at;
  cache_put<MANY>(a, cache, o + 8 * l, ca);
  cache_put<MANY>(a, cache, o + 8 * (l + g), cb);
}

template <bool MANY>
__device__ __forceinline__ void cache_store(const QkArgs &a, void *cache, int64_t at, int l, int g,
                                            const uint2 &ca, const uint2 &cb) {
  uint8_t *o = static_cast<uint8_t *>(cache) + at;
  cache_put<MANY>(a, cache, o + 8 * l, ca);
  cache_put<MANY>(a, cache, o + 8 * (l + g), cb);
}

// The multi-axis and cache forms.  H: heads that a lane group takes, one after
// the other; their loads go out together and they share the token's position,
// slot and cos/sin values.  One for few tokens (the shortest chain: a token 1.8
// us against 2.5) and three for many (16411 tokens of 32 + 8 heads with three
// axes: 80, 57, 55, 55 us with one to four; 32768 tokens into a bf16 cache: 171,
// 140, 122, 124 us, the copy rate; 8191 tokens of 64 + 8 heads into an FP8
// cache: 66, 59, 56, 54; gptj with one to three: 80, 58, 56; 170, 133, 121; 66,
// 55, 52, although three spill 16 to 20 bytes).
constexpr int kManyHeads = 3;

template <int G, bool NEOX, bool AXES, bool APPEND, int H>
__global__ void __launch_bounds__(512, 2) qk_norm_rope_form_kernel(const QkArgs a) {
  constexpr int D = G * 16, kPerWarp = 32 / G;
  const int lane = threadIdx.x & 31;
  const int l = lane & (G - 1);
  const int64_t t = blockIdx.x;
  // the warp's first head; a lane group's heads: h0 + lane / G + k * kPerWarp
  const int h0 = ((int)blockIdx.y * (int)(blockDim.x >> 5) + (int)(threadIdx.x >> 5)) * kPerWarp * H;
  // Launched with programmatic dependent launch: nothing in global memory
  // before the previous grid has finished, except that the CTA's heads are
  // asked into L2 first; the next grid may be scheduled once the loads are out.
  if (threadIdx.x == 0 && (int)blockIdx.x < a.pf_ctas) {
    const int most = (int)(blockDim.x >> 5) * kPerWarp * H;
    const int nh = a.nh - h0 < most ? a.nh - h0 : most;
    prefetch_l2(a.qkv + t * a.row + (int64_t)h0 * D, 2u * (uint32_t)(nh * D));
  }
  pdl_wait();
  // The heads' loads do not depend on the token's position, so they go out
  // together with it (a head with a bad position is loaded but not stored);
  // only the cos/sin row waits for the position.
  uint16_t *token = a.qkv + t * a.row;
  const int64_t pos = AXES ? 0 : a.pos[t];
  const int64_t slot = APPEND ? a.slots[t] : 0;
  // chunk 0 of the lane: l (first half of the head), chunk 1: l + G
  uint4 xa[H], xb[H];
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const int h = h0 + lane / G + k * kPerWarp;
    const bool in_head = h < a.nh;
    const uint16_t *head = token + (in_head ? (int64_t)h * D : 0);
    xa[k] = in_head ? ld_stream(head + l * kElemsPerChunk) : make_uint4(0, 0, 0, 0);
    xb[k] = in_head ? ld_stream(head + (l + G) * kElemsPerChunk) : make_uint4(0, 0, 0, 0);
  }
  bool pos_ok = true;                       // the same for the whole CTA
  [[maybe_unused]] uint32_t at[4] = {};     // first element of each axis's table row
  if constexpr (AXES) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t p = x < a.axes ? a.pos[x * a.T + t] : 0;
      pos_ok = pos_ok && p >= 0 && p < a.max_pos;
      at[x] = (uint32_t)p * (uint32_t)D;  // max_pos * D fits 32 bits
    }
  } else {
    pos_ok = pos >= 0 && pos < a.max_pos;
  }
  if (!pos_ok && h0 + lane / G < a.nh && l == 0) atomicOr(&g_rope_status, kErrBadPosition);
  pdl_launch_dependents();

  // cos and sin of the lane's pairs: neox 8l .. 8l + 7 (element k of chunk 0
  // with element k of chunk 1), gptj 4l .. 4l + 3 and 4(l + G) .. + 3 (inside
  // either chunk)
  float cv[8] = {}, sv[8] = {};
  if (pos_ok && h0 + lane / G < a.nh) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const int p0 = NEOX ? 8 * l + i : 4 * (i ? l + G : l);
      if constexpr (!AXES) {
        load4f(a.cache + pos * D + p0, cv, i);
        load4f(a.cache + pos * D + D / 2 + p0, sv, i);
      } else {
        // from one row, or from the row of each pair's axis (one wide load
        // where all four share it)
        const auto row = [&](uint32_t x) { return x < 2 ? (x == 0 ? at[0] : at[1]) : (x == 2 ? at[2] : at[3]); };
        const uint32_t m = (a.axis_map[p0 >> 4] >> (2 * (p0 & 15))) & 0xFFu;
        if (m == (m & 3u) * 0x55u) {
          const float *r = a.cache + row(m & 3u) + p0;
          load4f(r, cv, i);
          load4f(r + D / 2, sv, i);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float *r = a.cache + row((m >> (2 * k)) & 3u) + p0 + k;
            cv[i + k] = __ldg(r);
            sv[i + k] = __ldg(r + D / 2);
          }
        }
      }
    }
  }

#pragma unroll
  for (int k = 0; k < H; ++k) {
    const int first = h0 + k * kPerWarp, h = first + lane / G;
    const bool live = h < a.nh && pos_ok;  // same for the head's lanes
    if constexpr (APPEND) {
      // V heads go to the cache as they are, and need no more
      if (live && h >= a.hqk) {
        const int64_t place = cache_place(a, slot, h - a.hqk, l == 0);
        if (place >= 0 && a.v_scale == nullptr) {
          cache_store<(H > 1)>(a, a.v_cache, place, l, G, xa[k], xb[k]);
        } else if (place >= 0) {
          const float m = __frcp_rn(__ldg(a.v_scale));
          cache_store<(H > 1)>(a, a.v_cache, place, l, G, scaled_codes(xa[k], m), scaled_codes(xb[k], m));
        }
      }
    }
    if (first >= (APPEND ? a.hqk : a.nh)) continue;  // the whole warp
    const uint16_t *w = h < a.hq ? a.qw : a.kw;
    const bool norm = w != nullptr && h < a.hqk;
    constexpr uint32_t kOnes = 0x3F803F80u;  // two bf16 ones: a rotation without a norm
    const uint4 ones = make_uint4(kOnes, kOnes, kOnes, kOnes);
    const uint4 wa = norm ? ld_keep(w + l * kElemsPerChunk) : ones;
    const uint4 wb = norm ? ld_keep(w + (l + G) * kElemsPerChunk) : ones;
    float2 ta[4], tb[4];
    float cmax;
    RowAcc acc;
    pass1_chunk<false, false>(xa[k], xa[k], wa, ta, cmax, acc);
    pass1_chunk<false, false>(xb[k], xb[k], wb, tb, cmax, acc);
    float ss = acc.ss.x + acc.ss.y;
#pragma unroll
    for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    const float y = norm ? rsqrtf(fmaf(ss, 1.0f / (float)D, a.eps)) : 1.0f;

    // mine[0..7]: chunk 0, mine[8..15]: chunk 1; other: each element's pair
    // partner; c, s: its pair's cos and sin; submask bit i: minus sign
    float mine[16], other[16], c[16], s[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mine[2 * i] = ta[i].x;
      mine[2 * i + 1] = ta[i].y;
      mine[8 + 2 * i] = tb[i].x;
      mine[8 + 2 * i + 1] = tb[i].y;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      other[i] = mine[NEOX ? i ^ 8 : i ^ 1];
      c[i] = cv[NEOX ? i & 7 : i >> 1];
      s[i] = sv[NEOX ? i & 7 : i >> 1];
    }
    constexpr uint32_t submask = NEOX ? 0x00FFu : 0x5555u;

    float p[16];
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const bool m0 = (submask >> i) & 1u, m1 = (submask >> (i + 1)) & 1u;
      const float2 o = kahan2x(make_float2(mine[i], mine[i + 1]), make_float2(c[i], c[i + 1]),
                               make_float2(m0 ? -other[i] : other[i], m1 ? -other[i + 1] : other[i + 1]),
                               make_float2(s[i], s[i + 1]));
      const float2 pp = f2_mul(o, make_float2(y, y));
      p[i] = pp.x;
      p[i + 1] = pp.y;
    }
    if (!live) continue;
    if constexpr (APPEND) {
      if (h >= a.hq) {  // a K head goes to its slot (a V head is already there)
        const int64_t place = h < a.hqk ? cache_place(a, slot, h - a.hq, l == 0) : -1;
        if (place < 0) continue;
        if (a.k_scale != nullptr) {
          const float m = __frcp_rn(__ldg(a.k_scale));
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] *= m;
          cache_store<(H > 1)>(a, a.k_cache, place, l, G, codes8(p), codes8(p + 8));
        } else {
          cache_store<(H > 1)>(a, a.k_cache, place, l, G, bf16x8(p), bf16x8(p + 8));
        }
        continue;
      }
    }
    uint16_t *head = token + (int64_t)h * D;
    [[maybe_unused]] const uint64_t bytes = VG_ROWS(a.T) * 2ull * (uint64_t)a.row;
    if (VG_ACCESS_OK(g_rope_status, head + l * kElemsPerChunk, 16, a.qkv, bytes))
      st_stream(head + l * kElemsPerChunk, bf16x8(p));
    if (VG_ACCESS_OK(g_rope_status, head + (l + G) * kElemsPerChunk, 16, a.qkv, bytes))
      st_stream(head + (l + G) * kElemsPerChunk, bf16x8(p + 8));
  }
}

// One token per CTA: up to 16 warps of heads, more of them dealt out evenly over
// blockIdx.y.  H: heads a lane group takes.
template <int G, int H>
cudaError_t launch_heads(void (*kern)(QkArgs), const QkArgs &a, cudaStream_t s) {
  constexpr int heads_per_warp = 32 / G * H;
  const int all = (a.nh + heads_per_warp - 1) / heads_per_warp;
  const int parts = (all + 15) / 16;
  const int warps = (all + parts - 1) / parts;
  const dim3 grid((unsigned)a.T, (unsigned)((a.nh + warps * heads_per_warp - 1) / (warps * heads_per_warp)));
  return launch_pdl(kern, grid, dim3(warps * 32), 0, s, a);
}

// Many tokens: from four per SM on (pf_ctas is two per SM).
template <int G, bool AXES, bool APPEND>
cudaError_t launch_form(const QkArgs &a, bool neox, cudaStream_t s) {
  constexpr int H = kManyHeads;
  if (a.T >= 2LL * a.pf_ctas)
    return launch_heads<G, H>(neox ? qk_norm_rope_form_kernel<G, true, AXES, APPEND, H>
                                   : qk_norm_rope_form_kernel<G, false, AXES, APPEND, H>, a, s);
  return launch_heads<G, 1>(neox ? qk_norm_rope_form_kernel<G, true, AXES, APPEND, 1>
                                 : qk_norm_rope_form_kernel<G, false, AXES, APPEND, 1>, a, s);
}

template <int G>
cudaError_t launch_g(const QkArgs &a, bool neox, cudaStream_t s) {
  if (a.slots)
    return a.axes > 1 ? launch_form<G, true, true>(a, neox, s) : launch_form<G, false, true>(a, neox, s);
  // the plain form has weights and one axis; without weights the multi-axis
  // form turns by its one axis
  const bool weights = (a.hq == 0 || a.qw) && (a.hqk == a.hq || a.kw);
  if (a.axes > 1 || !weights) return launch_form<G, true, false>(a, neox, s);
  return launch_heads<G, 1>(neox ? qk_norm_rope_kernel<G, true> : qk_norm_rope_kernel<G, false>, a, s);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkArgs &a, int head_dim, bool neox, cudaStream_t s) {
  switch (head_dim) {
    case 64: return launch_g<4>(a, neox, s);
    case 128: return launch_g<8>(a, neox, s);
    default: return launch_g<16>(a, neox, s);
  }
}

uint32_t read_rope_status(bool reset) {
  uint32_t v = 0;
  if (cudaMemcpyFromSymbol(&v, g_rope_status, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (reset) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbol(g_rope_status, &zero, sizeof(zero)) != cudaSuccess) return 0xFFFFFFFFu;
  }
  return v;
}

}  // namespace vg
