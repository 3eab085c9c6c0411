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
#include "dependent.cuh"

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
// where the item has few shares (many items, each cut once or twice), its four warps on one row after
// another where it has many (one long sequence: 76 shares).  A warp loads eight shares' references, sums and rows
// together, so the eight cost one memory latency.  Launched so that it is set up while the attention ends.
constexpr int CC_THREADS = 128, CC_FEW = 8;
template <int D, int RT, typename Args>
__global__ void __launch_bounds__(CC_THREADS) split_combine_kernel(const Args a, int nrow) {
  constexpr int NL = D / 4, NW = CC_THREADS / 32;
  __shared__ float2 wml[NW];
  __shared__ float4 sums[NW][NL];
  const int item = blockIdx.x, per = a.Hkv * a.ntile;
  const int b = item / per, kvh = item % per / a.ntile, row0 = (item % a.ntile) * 8 * RT;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = blockIdx.y * nrow, last = min(min(8 * RT, a.rows - row0), first + nrow);
  auto out = [&](int row) { return out_row(a, b, kvh, row0 + row) + 4 * lane; };
  wait_for_earlier();
  const int2 ends = a.ends[item];
  if (a.empty(b)) {
    for (int row = first + warp; row < last; row += NW)
      if (lane < NL) put_row(out(row), make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
    return;
  }
  const int n = ends.y - ends.x + 1;
  if (n <= 1) return;  // written by its only CTA
  const int64_t at0 = (static_cast<int64_t>(ends.x) + item) * 8 * RT;
  // shares w0, w0 + step, ... of a row: their reference M, sum L and, in lanes below NL, four channels of O
  auto gather = [&](int row, int w0, int step, float &M, float &L, float4 &o) {
    M = -INFINITY;
    L = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = w0; w < n; w += CC_FEW * step) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (lane < CC_FEW && w + lane * step < n)
        ml = *reinterpret_cast<const float2 *>(a.part_ml + (at0 + static_cast<int64_t>(w + lane * step) * 8 * RT + row) * 2);
      float4 v[CC_FEW];
#pragma unroll
      for (int i = 0; i < CC_FEW; ++i)
        if (w + i * step < n && lane < NL)
          v[i] = *reinterpret_cast<const float4 *>(a.part_o + (at0 + static_cast<int64_t>(w + i * step) * 8 * RT + row) * D + 4 * lane);
      float m = ml.x;
#pragma unroll
      for (int k = 4; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
      m = fmaxf(M, __shfl_sync(0xffffffffu, m, 0));
      const float f0 = share_weight(M, L, m), f = share_weight(ml.x, ml.y, m);
      M = m;
      float l = f != 0.f ? f * ml.y : 0.f;
#pragma unroll
      for (int k = 4; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
      L = (f0 != 0.f ? f0 * L : 0.f) + __shfl_sync(0xffffffffu, l, 0);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      add_share(s, f0, o);
#pragma unroll
      for (int i = 0; i < CC_FEW; ++i) {
        const float fi = __shfl_sync(0xffffffffu, f, i);
        if (w + i * step < n && lane < NL) add_share(s, fi, v[i]);
      }
      o = s;
    }
  };
  float M, L;
  float4 o;
  if (n <= CC_FEW) {
    for (int row = first + warp; row < last; row += NW) {
      gather(row, 0, 1, M, L, o);
      if (lane < NL) put_row(out(row), o, L == 0.f ? 0.f : 1.f / L);
    }
    return;
  }
  for (int row = first; row < last; ++row) {
    gather(row, warp, NW, M, L, o);
    if (lane == 0) wml[warp] = make_float2(M, L);
    if (lane < NL) sums[warp][lane] = o;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int u = 0; u < NW; ++u) M = fmaxf(M, wml[u].x);
      L = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int u = 0; u < NW; ++u) {
        const float f = share_weight(wml[u].x, wml[u].y, M);
        if (f != 0.f) L = fmaf(f, wml[u].y, L);
        if (lane < NL) add_share(o, f, sums[u][lane]);
      }
      if (lane < NL) put_row(out(row), o, L == 0.f ? 0.f : 1.f / L);
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
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>((rows + nrow - 1) / nrow));
  return launch_dependent(split_combine_kernel<D, RT, Args>, grid, CC_THREADS, 0, st, a, nrow);
}

}  // namespace sparge
