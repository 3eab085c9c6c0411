// Attention of a few query rows per key/value head (decoding steps, short chunks), the parts that its
// kernels share: the way the work is cut, the products' wrappers, the end of an item and the kernel
// that puts cut items together.
//
// An item is a tile of 8 RT query rows (the Nq queries of all G heads of a KV head) of one sequence
// against all keys that they see.  The items' key tiles stand in one line that is cut into equal shares,
// one per CTA; a CTA's four warps sum up O, the exponent reference and the sum of P for their own keys
// and merge them at the item's end.  An item inside one CTA is written out there; one that is cut leaves a
// partial result per CTA, at place (CTA + item) - no two pairs that meet share a place - and the
// combining kernel weighs them.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace sparge {

constexpr int CA_WARPS = 4;
constexpr int CA_SMS = 152;
constexpr float CA_RESCALE = 8.f;  // the exponent reference moves when a score passes it by more (log2)

struct SplitArgs {
  __nv_bfloat16 *o;
  int64_t o_sb, o_sh, o_sn;
  int B, Hkv, G, Nq, rows, ntile;  // rows = G Nq, ntile row tiles
  float *part_o, *part_ml;         // [CTA + item][8 RT][D], [CTA + item][8 RT] (reference, sum)
  int2 *ends;                      // per item: its first and last CTA
};

// Row tiles of 8 rows for up to 8 query rows per KV head, else of 16.
inline int row_tile(int64_t rows) { return rows <= 8 ? 1 : 2; }
struct SplitWs {
  size_t o, ml, ends, total;  // offsets of the three arrays
};
inline SplitWs split_ws(int64_t items, int ctas, int rt, int64_t d) {
  const auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const int64_t slots = items + ctas;
  SplitWs w;
  w.o = 0;
  w.ml = up(static_cast<size_t>(slots) * 8 * rt * d * 4);
  w.ends = w.ml + up(static_cast<size_t>(slots) * 8 * rt * 2 * 4);
  w.total = w.ends + up(static_cast<size_t>(items) * 8);
  return w;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The exponent reference of a row (its negative m) follows the maximum x over the warp's tokens when it
// passes t = reference + CA_RESCALE (-inf: nothing seen yet); returns the factor on what has been
// summed.  Lanes 4 g + c hold the same two rows for every g.
__device__ __forceinline__ float follow(float &t, float &m, float x) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if (!(x > t)) return 1.f;
  const float f = t == -INFINITY ? 0.f : exp2f(-m - x);
  m = -x;
  t = x + CA_RESCALE;
  return f;
}

// The weight of a share of reference m and sum l against the largest reference M (without a visible
// token: -inf and 0; NaN inputs: NaN).
__device__ __forceinline__ float share_weight(float m, float l, float M) {
  return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : exp2f(m - M);
}
__device__ __forceinline__ void add_share(float4 &o, float f, float4 v) {
  if (f != 0.f) {
    o.x = fmaf(f, v.x, o.x);
    o.y = fmaf(f, v.y, o.y);
    o.z = fmaf(f, v.z, o.z);
    o.w = fmaf(f, v.w, o.w);
  }
}
__device__ __forceinline__ void put_row(__nv_bfloat16 *to, float4 o, float inv) {
  uint2 w;
  w.x = pack_bf16x2(o.x * inv, o.y * inv);
  w.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2 *>(to) = w;
}
__device__ __forceinline__ __nv_bfloat16 *out_row(const SplitArgs &a, int b, int kvh, int r) {
  return a.o + b * a.o_sb + (kvh * a.G + r / a.Nq) * a.o_sh + static_cast<int64_t>(r % a.Nq) * a.o_sn;
}

// The end of an item in a CTA, called by all its threads.  sums + w * wstride: warp w's O rows, orow
// floats apart; ml: (reference, sum) of warp w's row at w * 8 RT + row.  first / last: this CTA holds the
// item's first / last tile.
template <int D, int RT>
__device__ __forceinline__ void end_item(const SplitArgs &a, const uint8_t *sums, int wstride, int orow, const float2 *ml,
                                         int item, int b, int kvh, int row0, bool first, bool last) {
  __syncthreads();
  if (threadIdx.x == 0) {
    if (first) a.ends[item].x = blockIdx.x;
    if (last) a.ends[item].y = blockIdx.x;
  }
  const int nrow = min(8 * RT, a.rows - row0);
  const int64_t slot = static_cast<int64_t>(blockIdx.x) + item;
  for (int e = threadIdx.x; e < nrow * (D / 4); e += CA_WARPS * 32) {
    const int row = e / (D / 4), d4 = e % (D / 4);
    float2 w[CA_WARPS];
    float M = -INFINITY;
#pragma unroll
    for (int u = 0; u < CA_WARPS; ++u) {
      w[u] = ml[u * 8 * RT + row];
      M = fmaxf(M, w[u].x);
    }
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < CA_WARPS; ++u) {
      const float f = share_weight(w[u].x, w[u].y, M);
      if (f != 0.f) L = fmaf(f, w[u].y, L);
      add_share(o, f, *reinterpret_cast<const float4 *>(sums + u * wstride + (row * orow + 4 * d4) * 4));
    }
    if (first && last) {
      put_row(out_row(a, b, kvh, row0 + row) + 4 * d4, o, L == 0.f ? 0.f : 1.f / L);
    } else {
      *reinterpret_cast<float4 *>(a.part_o + (slot * 8 * RT + row) * D + 4 * d4) = o;
      if (d4 == 0) *reinterpret_cast<float2 *>(a.part_ml + (slot * 8 * RT + row) * 2) = make_float2(M, L);
    }
  }
  fence_proxy_async_smem();  // these reads (and the sums' writes) before the next item's copies into the same places
  __syncthreads();
}

// Items cut between CTAs: the CTAs' partial rows (at CTA + item, a place of its own for every pair
// that meets) weighted by 2^(m - M) and divided by the weighted sum, in an order that the lengths alone
// set.  Items without a token get zero rows.  A CTA takes `nrow` rows of an item: one row per warp
// where the item has few shares (many items, each cut once or twice), the whole CTA on one row after
// another where it has many (one long sequence: 76 shares), so either way a few memory latencies.
// Launched so that it may start while the attention ends (programmatic dependent launch); nothing is
// read before the wait.
constexpr int CC_THREADS = 128, CC_FEW = 8;
template <int D, int RT, typename Args>
__global__ void __launch_bounds__(CC_THREADS) split_combine_kernel(const Args a, int nrow) {
  constexpr int NL = D / 4, NGRP = CC_THREADS / NL;
  __shared__ float wgt[CA_SMS * 4];
  __shared__ float red[2][CC_THREADS / 32];
  __shared__ float4 sums[NGRP][NL];
  const int item = blockIdx.x, per = a.Hkv * a.ntile;
  const int b = item / per, kvh = item % per / a.ntile, row0 = (item % a.ntile) * 8 * RT;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, d4 = t % NL, grp = t / NL;
  const int last = min(8 * RT, a.rows - row0), first = blockIdx.y * nrow;
  auto out = [&](int row) { return out_row(a, b, kvh, row0 + row); };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.empty(b)) {
    for (int row = first + warp; row < min(last, first + nrow); row += CC_THREADS / 32)
      if (lane < NL) put_row(out(row) + 4 * lane, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
    return;
  }
  const int2 ends = a.ends[item];
  const int n = ends.y - ends.x + 1;
  if (n <= 1) return;  // written by its only CTA
  const int64_t at0 = (static_cast<int64_t>(ends.x) + item) * 8 * RT;
  if (n <= CC_FEW) {
    for (int row = first + warp; row < min(last, first + nrow); row += CC_THREADS / 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < n) ml = *reinterpret_cast<const float2 *>(a.part_ml + (at0 + static_cast<int64_t>(lane) * 8 * RT + row) * 2);
      float4 v[CC_FEW];
      if (lane < NL) {
#pragma unroll
        for (int w = 0; w < CC_FEW; ++w)
          if (w < n) v[w] = *reinterpret_cast<const float4 *>(a.part_o + (at0 + static_cast<int64_t>(w) * 8 * RT + row) * D + 4 * lane);
      }
      float M = ml.x;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      M = __shfl_sync(0xffffffffu, M, 0);
      const float f = share_weight(ml.x, ml.y, M);
      float L = f != 0.f ? f * ml.y : 0.f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      L = __shfl_sync(0xffffffffu, L, 0);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < CC_FEW; ++w) {
        const float fw = __shfl_sync(0xffffffffu, f, w);
        if (w < n && lane < NL) add_share(o, fw, v[w]);
      }
      if (lane < NL) put_row(out(row) + 4 * lane, o, L == 0.f ? 0.f : 1.f / L);
    }
    return;
  }
  for (int row = first; row < min(last, first + nrow); ++row) {
    float M = -INFINITY;
    for (int w = t; w < n; w += CC_THREADS) M = fmaxf(M, a.part_ml[(at0 + static_cast<int64_t>(w) * 8 * RT + row) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < CC_THREADS / 32; ++u) M = fmaxf(M, red[0][u]);
    float L = 0.f;
    for (int w = t; w < n; w += CC_THREADS) {
      const float2 ml = *reinterpret_cast<const float2 *>(a.part_ml + (at0 + static_cast<int64_t>(w) * 8 * RT + row) * 2);
      const float f = share_weight(ml.x, ml.y, M);
      wgt[w] = f;
      if (f != 0.f) L = fmaf(f, ml.y, L);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) red[1][warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int u = 0; u < CC_THREADS / 32; ++u) L += red[1][u];
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int w = grp; w < n; w += NGRP)
      add_share(o, wgt[w], *reinterpret_cast<const float4 *>(a.part_o + (at0 + static_cast<int64_t>(w) * 8 * RT + row) * D + 4 * d4));
    sums[grp][d4] = o;
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int u = 1; u < NGRP; ++u) add_share(o, 1.f, sums[u][d4]);
      put_row(out(row) + 4 * d4, o, L == 0.f ? 0.f : 1.f / L);
    }
    __syncthreads();
  }
}


// shares: the attention kernel's CTAs, at most
template <int D, int RT, typename Args>
cudaError_t launch_split_combine(const Args &a, int64_t shares, cudaStream_t st) {
  // rows of a combining CTA: one per warp where items outnumber half the shares (an item then has few), else one
  const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * a.ntile;
  const int nrow = 2 * items > shares ? CC_THREADS / 32 : 1, rows = a.rows < 8 * RT ? a.rows : 8 * RT;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items), static_cast<unsigned>((rows + nrow - 1) / nrow));
  cfg.blockDim = dim3(CC_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, split_combine_kernel<D, RT, Args>, a, nrow);
}

}  // namespace sparge
