// The f16 copy of V that the chunk kernels of the window attention multiply with.
//
// bf16 holds 8 bits of values over 2^-126 .. 2^128, f16 the same bits over 2^-17 .. 2^16 alone.  So the copy of a KV head
// whose largest finite value lies outside of 2^-6 .. 65504 is multiplied by a power of two that takes it to 2^14 .. 2^15, and the
// attention divides by it (unit): a copied value is off by at most 2^-25 of the copy, which is 2^-19 of the
// head's largest value or less.  Infinities and NaN stay what they are.
//
// Copying without the factor and noting the largest value of each CTA's rows is one pass over V; a second kernel takes the
// largest of a head and writes its unit.  Only where the factor is not 1 it goes through the head's rows again, so
// values of the usual sizes cost its launch and the few words (4096 queries of 8 + 2 heads, d = 64, window 256: 12.9 us, 12.4
// without).  A pass for the largest values in front of the copy would read V twice every time.
#include <cuda_fp16.h>

#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace sparge {
namespace {

constexpr int WV_THREADS = 256, WV_VECS = 2;  // 16-byte pieces of a thread, both in flight

struct WindowVArgs {
  const __nv_bfloat16 *x;
  int64_t sb, sh, sn;
  __half *y;             // contiguous (B, H, N, D)
  uint32_t *largest;     // [B H][chunks] bf16 magnitudes
  float *unit;           // [B H]
  int H, N, front, lo;   // copied rows: 0 .. front - 1 and lo .. N - 1
  int zero_from, zero_to;  // rows that no query sees: zero, whatever V holds there
  int chunks, front_chunks;
};

template <int D>
struct WvRows {
  static constexpr int VPR = D / 8;                            // pieces of a row
  static constexpr int ROWS = WV_VECS * WV_THREADS / VPR;      // rows of a chunk
};

// Row of piece e of a chunk, or -1 behind the copied rows.
template <int D>
__device__ __forceinline__ int row_of(const WindowVArgs &a, int chunk, int e) {
  using R = WvRows<D>;
  const bool in_front = chunk < a.front_chunks;
  const int t = (in_front ? chunk * R::ROWS : a.lo + (chunk - a.front_chunks) * R::ROWS) + e / R::VPR;
  return t < (in_front ? a.front : a.N) ? t : -1;
}
template <int D>
__device__ __forceinline__ uint4 load_piece(const WindowVArgs &a, int b, int h, int t, int e) {
  if (t < 0 || (t >= a.zero_from && t < a.zero_to)) return make_uint4(0, 0, 0, 0);
  return ld_once_v4(a.x + b * a.sb + h * a.sh + static_cast<int64_t>(t) * a.sn + (e % WvRows<D>::VPR) * 8);
}
// two bf16 times f as two f16 (f = 1: exact in f16's range; past it an infinity, which the factor then makes finite)
__device__ __forceinline__ uint32_t to_f16(uint32_t w, float f) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(bf16hi(w) * f), "f"(bf16lo(w) * f));
  return r;
}
template <int D>
__device__ __forceinline__ void store_piece(const WindowVArgs &a, int64_t bh, int t, int e, uint4 v, float f) {
  *reinterpret_cast<uint4 *>(a.y + (bh * a.N + t) * D + (e % WvRows<D>::VPR) * 8) =
      make_uint4(to_f16(v.x, f), to_f16(v.y, f), to_f16(v.z, f), to_f16(v.w, f));
}
// the larger of m and the finite ones of two bf16 magnitudes, as bits
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
  const uint32_t lo = w & 0x7FFFu, hi = (w >> 16) & 0x7FFFu;
  return max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
}
// The largest of the CTA's values, to all its threads.
__device__ __forceinline__ uint32_t largest_of_cta(uint32_t m, uint32_t *share) {
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) share[threadIdx.x >> 5] = m;
  __syncthreads();
  m = share[threadIdx.x & (WV_THREADS / 32 - 1)];
  return __reduce_max_sync(0xffffffffu, m);
}

// grid (chunks, H, B)
template <int D>
__global__ void __launch_bounds__(WV_THREADS) copy_v_kernel(const WindowVArgs a) {
  __shared__ uint32_t share[WV_THREADS / 32];
  const int chunk = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  let_dependents_start();
  wait_for_earlier();
  uint4 v[WV_VECS];
  int t[WV_VECS];
#pragma unroll
  for (int u = 0; u < WV_VECS; ++u) {
    const int e = threadIdx.x + u * WV_THREADS;
    t[u] = row_of<D>(a, chunk, e);
    v[u] = load_piece<D>(a, b, h, t[u], e);
  }
  uint32_t m = 0u;
#pragma unroll
  for (int u = 0; u < WV_VECS; ++u) {
    m = larger(larger(larger(larger(m, v[u].x), v[u].y), v[u].z), v[u].w);
    if (t[u] >= 0) store_piece<D>(a, bh, t[u], threadIdx.x + u * WV_THREADS, v[u], 1.f);
  }
  m = largest_of_cta(m, share);
  if (threadIdx.x == 0) a.largest[bh * a.chunks + chunk] = m;
}

// grid (CTAs of a head, H, B)
template <int D>
__global__ void __launch_bounds__(WV_THREADS) scale_v_kernel(const WindowVArgs a) {
  __shared__ uint32_t share[WV_THREADS / 32];
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  let_dependents_start();
  wait_for_earlier();
  uint32_t m = 0u;
  for (int c = threadIdx.x; c < a.chunks; c += WV_THREADS) m = max(m, a.largest[bh * a.chunks + c]);
  m = largest_of_cta(m, share);
  const float top = __uint_as_float(m << 16);
  const bool scale = top > 65504.f || (top > 0.f && top < 0.015625f);
  // 2^(14 - exponent); a head of nothing but values below 2^-86 goes less far, so that its unit over a row's sum stays normal
  const int k = scale ? min(14 - (static_cast<int>(m >> 7) - 127), 100) : 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) a.unit[bh] = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
  if (!scale) return;
  const float f = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  for (int c = blockIdx.x; c < a.chunks; c += gridDim.x)
#pragma unroll
    for (int u = 0; u < WV_VECS; ++u) {
      const int e = threadIdx.x + u * WV_THREADS, t = row_of<D>(a, c, e);
      if (t >= 0) store_piece<D>(a, bh, t, e, load_piece<D>(a, b, h, t, e), f);
    }
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t most_chunks(int64_t N, int64_t d) {
  const int64_t rows = WV_VECS * WV_THREADS / (d / 8);
  return (N + rows - 1) / rows + 1;  // the rows in front may end in a chunk of their own
}

template <int D>
cudaError_t launch_t(const WindowVArgs &a, const View &v, cudaStream_t st) {
  const unsigned H = static_cast<unsigned>(v.H), B = static_cast<unsigned>(v.B);
  if (cudaError_t e = launch_dependent(copy_v_kernel<D>, dim3(static_cast<unsigned>(a.chunks), H, B), WV_THREADS, 0, st, a);
      e != cudaSuccess)
    return e;
  // CTAs of a head: two per SM in all, where there are heads few enough
  int64_t per = 304 / (v.H * v.B);
  per = per < 1 ? 1 : per > a.chunks ? a.chunks : per;
  return launch_dependent(scale_v_kernel<D>, dim3(static_cast<unsigned>(per), H, B), WV_THREADS, 0, st, a);
}

}  // namespace

size_t window_v_ws_bytes(int64_t B, int64_t H, int64_t N, int64_t d) {
  return up256(static_cast<size_t>(B) * H * N * d * 2) + up256(static_cast<size_t>(B) * H * most_chunks(N, d) * 4) +
         up256(static_cast<size_t>(B) * H * 4);
}

cudaError_t launch_window_v(const View &v, void *ws, int64_t front, int64_t lo, int64_t zero_from, int64_t zero_to,
                            const float **unit, cudaStream_t st) {
  WindowVArgs a;
  uint8_t *w = static_cast<uint8_t *>(ws);
  const size_t copy = up256(static_cast<size_t>(v.B) * v.H * v.N * v.d * 2);
  a.x = static_cast<const __nv_bfloat16 *>(v.data);
  a.sb = v.sb; a.sh = v.sh; a.sn = v.sn;
  a.y = reinterpret_cast<__half *>(w);
  a.largest = reinterpret_cast<uint32_t *>(w + copy);
  a.unit = reinterpret_cast<float *>(w + copy + up256(static_cast<size_t>(v.B) * v.H * most_chunks(v.N, v.d) * 4));
  a.H = static_cast<int>(v.H);
  a.N = static_cast<int>(v.N);
  a.front = static_cast<int>(front < lo ? front : lo);
  a.lo = static_cast<int>(lo);
  a.zero_from = static_cast<int>(zero_from);
  a.zero_to = static_cast<int>(zero_to);
  const int rows = WV_VECS * WV_THREADS / static_cast<int>(v.d / 8);
  a.front_chunks = (a.front + rows - 1) / rows;
  a.chunks = a.front_chunks + (a.N - a.lo + rows - 1) / rows;
  *unit = a.unit;
  return v.d == 128 ? launch_t<128>(a, v, st) : launch_t<64>(a, v, st);
}

}  // namespace sparge
