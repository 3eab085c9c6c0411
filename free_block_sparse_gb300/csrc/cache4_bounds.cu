// Pages of the 4-bit cache that matter to a query: bounds of each page's keys, and the selection by them.
//
// Bounds.  For every page and KV head the largest and smallest key of each channel, hi_c and lo_c, over the page's
// tokens as the cache reads them back, in int8 codes of one power of two s per page and head, rounded
// outwards: hi = s ceil(hi_c / s), lo = s floor(lo_c / s), s the least power of two with every |code| <= 127 (at least
// 2^-126).  A page that holds an infinity or a NaN has s = infinity.
// Score of a page for a query row: r_c = round-to-even(q_c / t), t a power of two in the same way, and
//   t s sum_c max(r_c hi_c, r_c lo_c) = t s (sum r+ hi + sum r- lo),   r+ = max(r, 0), r- = min(r, 0),
// which no token of the page exceeds in t r . k.  The sums are whole numbers below 2^21 and the factors powers of two, so a
// score is exact and the selection does not depend on the order of any sum.  A KV head's score is the largest of its
// heads'.  d + d bytes of codes per page and head in place of 9 d / 16 for every token.
//
// Layout of a page's bounds: codes [H][hi, lo][d], scales [H] (fp32), padded to 32 bytes.
#include <climits>
#include <cmath>

#include "../../include/sparge.h"
#include "cache4.cuh"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace sparge {
int check_cache4(const ::sparge_cache4 *c, Cache4 *out);
namespace {

constexpr int64_t bounds_row(int64_t H, int64_t d) { return (H * (2 * d + 4) + 31) / 32 * 32; }

// The least power of two s >= 2^-126 with a <= 127 s, for a >= 0; infinity where a is not finite.
__device__ __forceinline__ float code_unit(float a) {
  if (!(a < INFINITY)) return INFINITY;
  const uint32_t b = __float_as_uint(a);
  // a = 1.m 2^x: 127 = 1.984375 * 2^6
  int x = static_cast<int>(b >> 23) - 127 - 6 + ((b & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  x = max(x, -126);
  return __uint_as_float(static_cast<uint32_t>(x + 127) << 23);
}
// 1 / s for a power of two s in 2^-126 .. 2^126
__device__ __forceinline__ float over_unit(float s) { return __uint_as_float((254u << 23) - __float_as_uint(s)); }

struct BoundsArgs {
  const uint8_t *pool;
  uint8_t *bounds;
  const int32_t *table, *lens, *pages;
  int64_t table_stride, n_pages, row, N, count;
  int width, page_shift, H, most;  // most: pages of a sequence that its last N tokens can lie on
  __nv_bfloat16 *hi, *lo;
  int *status;
};

__device__ __forceinline__ int length_of(const int32_t *lens, int b, int width, int page_shift) {
  const int len = lens[b];
  const int64_t cap = static_cast<int64_t>(width) << page_shift;
  return max(len > cap ? static_cast<int>(cap) : len, 0);
}

// One warp per page and head, over the pages on which the last N tokens of each sequence lie.  Lane 4 t + c holds
// the channels 32 w + 8 c + j of every eighth token (the order of the codes in memory: 16-byte loads without gaps) and keeps their
// maxima and minima in registers; at the page's end the eight lanes of a channel exchange halves (28 + 28 values
// instead of 96 + 96) until each holds four channels in a row.
template <int D>
__global__ void __launch_bounds__(128) bounds_update_kernel(const BoundsArgs a) {
  using R = Rec4<D>;
  constexpr int NW = D / 32, NV = 8 * NW;  // words of a lane, values
  start_after_earlier();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tt = lane >> 2, c = lane & 3;
  const int b = static_cast<int>(blockIdx.x / a.most), nth = static_cast<int>(blockIdx.x % a.most);
  const int h = blockIdx.y * 4 + warp;
  const int len = length_of(a.lens, b, a.width, a.page_shift);
  const int first = static_cast<int>((len - a.N > 0 ? len - a.N : 0) >> a.page_shift), col = first + nth;
  const int64_t from = static_cast<int64_t>(col) << a.page_shift;
  if (h >= a.H || from >= len) return;
  const int page = a.table[static_cast<int64_t>(b) * a.table_stride + col];
  if (page < 0 || page >= a.n_pages) {
    if (lane == 0) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
    return;
  }
  const int P = 1 << a.page_shift, n = static_cast<int>(len - from < P ? len - from : P);
  const uint8_t *src = a.pool + (static_cast<int64_t>(page) * a.H + h) * (static_cast<int64_t>(P / C4_TOKENS) * R::BYTES);
  float hi[NV], lo[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    hi[i] = -INFINITY;
    lo[i] = INFINITY;
  }
  bool bad = false;
#pragma unroll 2
  for (int t0 = 0; t0 < n; t0 += 8) {
    const int t = t0 + tt;
    const uint8_t *rec = src + (t0 >> 4) * R::BYTES;
    uint32_t k[NW], word[R::NG];
    if (t < n) {
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4 *>(rec + R::K + (t & 15) * (D / 2) + c * (D / 8));
        const uint2 w = *reinterpret_cast<const uint2 *>(rec + R::KW + (t & 15) * 8);
        k[0] = u.x; k[1] = u.y; k[2] = u.z; k[3] = u.w;
        word[0] = w.x; word[1] = w.y;
      } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(rec + R::K + (t & 15) * (D / 2) + c * (D / 8));
        k[0] = u.x; k[1] = u.y;
        word[0] = *reinterpret_cast<const uint32_t *>(rec + R::KW + (t & 15) * 4);
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float s = bf16lo(word[w / 2]), m = bf16hi(word[w / 2]);
        bad = bad || !(fabsf(s) < INFINITY) || !(fabsf(m) < INFINITY);
        const uint32_t even = k[w] & 0x0F0F0F0Fu, odd = (k[w] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          // a code's byte becomes the low byte of 2^23 (code + 2^23, exactly)
          const float2 f = fadd2(make_float2(__uint_as_float(__byte_perm(even, 0x4B000000u, 0x7650 + j / 2)),
                                             __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7650 + j / 2))),
                                 make_float2(-8388608.f, -8388608.f));
          const float2 x = ffma2(f, make_float2(s, s), make_float2(m, m));
          hi[8 * w + j] = fmaxf(hi[8 * w + j], x.x);
          lo[8 * w + j] = fminf(lo[8 * w + j], x.x);
          hi[8 * w + j + 1] = fmaxf(hi[8 * w + j + 1], x.y);
          lo[8 * w + j + 1] = fminf(lo[8 * w + j + 1], x.y);
        }
      }
    }
  }
  // halves of the values to the lanes of either side of each bit of tt
#pragma unroll
  for (int s = 0, m = NV / 2; s < 3; ++s, m /= 2) {
    const int bit = 16 >> s;
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) {
      if (i >= m) break;
      const float gh = up ? hi[i] : hi[i + m], gl = up ? lo[i] : lo[i + m];
      const float mh = up ? hi[i + m] : hi[i], ml = up ? lo[i + m] : lo[i];
      hi[i] = fmaxf(mh, __shfl_xor_sync(0xffffffffu, gh, bit));
      lo[i] = fminf(ml, __shfl_xor_sync(0xffffffffu, gl, bit));
    }
  }
  constexpr int OWN = NV / 8;  // channels of a lane, in a row: number (lane's bits of tt as the halves went) * OWN of its 8 NW
  const int at = ((lane & 16) ? 4 * OWN : 0) + ((lane & 8) ? 2 * OWN : 0) + ((lane & 4) ? OWN : 0);
  float big = 0.f;
#pragma unroll
  for (int i = 0; i < OWN; ++i) big = fmaxf(big, fmaxf(fabsf(hi[i]), fabsf(lo[i])));
  if (bad) big = INFINITY;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
  const float unit = code_unit(big);
  uint32_t ch = 0u, cl = 0u;
  if (unit < INFINITY) {
    const float inv = over_unit(unit);
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      ch |= (static_cast<uint32_t>(__float2int_ru(hi[i] * inv)) & 0xFFu) << (8 * i);
      cl |= (static_cast<uint32_t>(__float2int_rd(lo[i] * inv)) & 0xFFu) << (8 * i);
    }
  }
  uint8_t *dst = a.bounds + static_cast<int64_t>(page) * a.row;
  const int channel = 32 * (at / 8) + 8 * c + at % 8;
  if constexpr (OWN == 4) {
    *reinterpret_cast<uint32_t *>(dst + h * 2 * D + channel) = ch;
    *reinterpret_cast<uint32_t *>(dst + h * 2 * D + D + channel) = cl;
  } else {
    *reinterpret_cast<uint16_t *>(dst + h * 2 * D + channel) = static_cast<uint16_t>(ch);
    *reinterpret_cast<uint16_t *>(dst + h * 2 * D + D + channel) = static_cast<uint16_t>(cl);
  }
  if (lane == 0) *reinterpret_cast<float *>(dst + a.H * 2 * D + 4 * h) = unit;
}

// The bounds as values (exact in bf16): 8 channels of one page and head a thread.
template <int D>
__global__ void __launch_bounds__(256) bounds_load_kernel(const BoundsArgs a) {
  start_after_earlier();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t n = i / (a.H * (D / 8));
  if (n >= a.count) return;
  const int r = static_cast<int>(i % (a.H * (D / 8))), h = r / (D / 8), c8 = r % (D / 8);
  const int page = a.pages[n];
  uint4 out[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
  if (page >= a.n_pages) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
  if (page >= 0 && page < a.n_pages) {
    const uint8_t *src = a.bounds + static_cast<int64_t>(page) * a.row;
    const float unit = *reinterpret_cast<const float *>(src + a.H * 2 * D + 4 * h);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const uint2 code = *reinterpret_cast<const uint2 *>(src + h * 2 * D + s * D + 8 * c8);
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = j < 2 ? code.x : code.y;
        const int at = (j & 1) * 16;
        const float x = static_cast<float>(static_cast<int8_t>(u >> at)), y = static_cast<float>(static_cast<int8_t>(u >> (at + 8)));
        w[j] = unit < INFINITY ? pack_bf16x2(x * unit, y * unit) : (s ? 0xFF80FF80u : 0x7F807F80u);
      }
      out[s] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  *reinterpret_cast<uint4 *>(a.hi + 8 * i) = out[0];
  *reinterpret_cast<uint4 *>(a.lo + 8 * i) = out[1];
}

// --------------------------------------------------------------------------------------------
// Selection: a cluster of 1 to 8 CTAs per list (sequence, query, KV head).  Each scores its part of the pages and writes their
// keys (scores as unsigned numbers of the same order) into the first CTA's shared memory; that one finds the
// smallest key to keep digit by digit and writes the list in the pages' order.
// --------------------------------------------------------------------------------------------
struct SelectArgs {
  const __nv_bfloat16 *q;
  int64_t q_sb, q_sh, q_sn;
  const uint8_t *bounds;
  const int32_t *table, *lens;
  int64_t table_stride, n_pages, row;
  int width, page_shift, Hkv, G, Nq, keep, first, last;
  int32_t *pages, *out_lens;
  int *status;
};

constexpr int SEL_THREADS = 256, SEL_WARPS = SEL_THREADS / 32, SEL_HEADS = 64;
constexpr int SEL_PAGES = 40960;  // keys that shared memory holds beside the queries

// Scores as numbers of the same order (a score is never a NaN; both zeros are one).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ void cluster_arrive_wait() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a 32-bit store into shared memory of the cluster's first CTA
__device__ __forceinline__ void store_first(uint32_t *p, uint32_t v) {
  uint32_t to;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(to) : "r"(smem_u32(p)));
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
}

template <int D>
__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const SelectArgs a) {
  constexpr int LPP = D / 16;  // lanes that share a page, 16 channels each; pages of such a group of lanes at a time
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float unit[SEL_HEADS];
  __shared__ uint32_t hist[256], found[2], ends[2], count[SEL_WARPS][2];
  start_after_earlier();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t clusters, rank;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(clusters));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t list = blockIdx.x / clusters;
  const int h = static_cast<int>(list % a.Hkv), i = static_cast<int>(list / a.Hkv % a.Nq), b = static_cast<int>(list / a.Hkv / a.Nq);
  const int64_t behind = static_cast<int64_t>(length_of(a.lens, b, a.width, a.page_shift)) - a.Nq + 1 + i;
  const int seen = static_cast<int>(behind > 0 ? behind : 0), P = 1 << a.page_shift;
  const int np = static_cast<int>((static_cast<int64_t>(seen) + P - 1) >> a.page_shift), n = min(np, a.keep);
  const int32_t *table = a.table + static_cast<int64_t>(b) * a.table_stride;
  int32_t *out = a.pages + list * a.keep;
  if (rank == 0) {
    if (h == 0 && threadIdx.x == 0)
      a.out_lens[static_cast<int64_t>(b) * a.Nq + i] = n > 0 ? static_cast<int>(static_cast<int64_t>(n - 1) * P) + (seen - 1) % P + 1 : 0;
    // every page, or those that are kept whatever their scores; then the places without one
    for (int k = threadIdx.x; k < a.keep; k += SEL_THREADS) {
      const bool middle = np > a.keep && k >= a.first && k < a.keep - a.last;
      if (!middle) out[k] = k >= n ? -1 : table[np > a.keep && k >= a.first ? np - (a.keep - k) : k];
    }
  }
  const int m = np - a.first - a.last, want = a.keep - a.first - a.last;  // pages to choose from, to choose
  if (np <= a.keep || want == 0) return;  // the same for the whole cluster
  // ---- the queries' codes: bytes r+ and r- of each head ----
  uint32_t *keys = reinterpret_cast<uint32_t *>(smem);
  uint8_t *codes = smem + (static_cast<int64_t>(a.width) * 4 + 15) / 16 * 16;  // [G][r+, r-][D]
  for (int g = warp; g < a.G; g += SEL_WARPS) {
    const __nv_bfloat16 *q = a.q + b * a.q_sb + (static_cast<int64_t>(h) * a.G + g) * a.q_sh + static_cast<int64_t>(i) * a.q_sn;
    constexpr int C = D / 32;
    float x[C], big = 0.f;
    bool fine = true;
    if constexpr (C == 4) {
      const uint2 u = *reinterpret_cast<const uint2 *>(q + 4 * lane);
      x[0] = bf16lo(u.x); x[1] = bf16hi(u.x); x[2] = bf16lo(u.y); x[3] = bf16hi(u.y);
    } else {
      const uint32_t u = *reinterpret_cast<const uint32_t *>(q + 2 * lane);
      x[0] = bf16lo(u); x[1] = bf16hi(u);
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
      fine = fine && fabsf(x[k]) < INFINITY;
      big = fmaxf(big, fabsf(x[k]));
    }
    fine = __all_sync(0xffffffffu, fine);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    const float t = fine ? code_unit(big) : 0.f, inv = fine ? over_unit(t) : 0.f;  // a query of NaN scores every page 0
    uint32_t plus = 0u, minus = 0u;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int r = fine ? __float2int_rn(x[k] * inv) : 0;
      plus |= (static_cast<uint32_t>(max(r, 0)) & 0xFFu) << (8 * k);
      minus |= (static_cast<uint32_t>(min(r, 0)) & 0xFFu) << (8 * k);
    }
    uint8_t *to = codes + g * 2 * D;
    if constexpr (C == 4) {
      *reinterpret_cast<uint32_t *>(to + 4 * lane) = plus;
      *reinterpret_cast<uint32_t *>(to + D + 4 * lane) = minus;
    } else {
      *reinterpret_cast<uint16_t *>(to + 2 * lane) = static_cast<uint16_t>(plus);
      *reinterpret_cast<uint16_t *>(to + D + 2 * lane) = static_cast<uint16_t>(minus);
    }
    if (lane == 0) unit[g] = t;
  }
  if (clusters > 1)
    cluster_arrive_wait();  // and the first CTA is there
  else
    __syncthreads();
  // ---- scores: 32 pages a warp and step; a group of LPP lanes takes LPP of them, and after the sums are exchanged each lane holds one ----
  const int e = lane % LPP;
  const uint8_t *base = a.bounds + h * 2 * D;
  for (int p0 = (static_cast<int>(rank) * SEL_WARPS + warp) * 32; p0 < m; p0 += static_cast<int>(clusters) * SEL_THREADS) {
    const int p = p0 + lane;
    int page = p < m ? table[a.first + p] : -1;
    if (p < m && (page < 0 || page >= a.n_pages)) {
      record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
      page = -1;
    }
    uint4 hi[LPP], lo[LPP];
#pragma unroll
    for (int u = 0; u < LPP; ++u) {
      const int id = __shfl_sync(0xffffffffu, page, (lane & ~(LPP - 1)) + u);
      hi[u] = lo[u] = make_uint4(0u, 0u, 0u, 0u);
      if (id >= 0) {
        const uint8_t *src = base + static_cast<int64_t>(id) * a.row + 16 * e;
        hi[u] = *reinterpret_cast<const uint4 *>(src);
        lo[u] = *reinterpret_cast<const uint4 *>(src + D);
      }
    }
    const float s = page >= 0 ? *reinterpret_cast<const float *>(a.bounds + static_cast<int64_t>(page) * a.row + a.Hkv * 2 * D + 4 * h) : 0.f;
    float best = -INFINITY;
    for (int g = 0; g < a.G; ++g) {
      const uint4 rp = *reinterpret_cast<const uint4 *>(codes + g * 2 * D + 16 * e), rn = *reinterpret_cast<const uint4 *>(codes + g * 2 * D + D + 16 * e);
      int x[LPP];
#pragma unroll
      for (int u = 0; u < LPP; ++u) {
        int v = __dp4a(static_cast<int>(hi[u].x), static_cast<int>(rp.x), 0);
        v = __dp4a(static_cast<int>(hi[u].y), static_cast<int>(rp.y), v);
        v = __dp4a(static_cast<int>(hi[u].z), static_cast<int>(rp.z), v);
        v = __dp4a(static_cast<int>(hi[u].w), static_cast<int>(rp.w), v);
        v = __dp4a(static_cast<int>(lo[u].x), static_cast<int>(rn.x), v);
        v = __dp4a(static_cast<int>(lo[u].y), static_cast<int>(rn.y), v);
        v = __dp4a(static_cast<int>(lo[u].z), static_cast<int>(rn.z), v);
        x[u] = __dp4a(static_cast<int>(lo[u].w), static_cast<int>(rn.w), v);
      }
      // lane e of the group ends with the sum of its page e
#pragma unroll
      for (int half = LPP / 2; half > 0; half /= 2) {
        const bool up = (e & half) != 0;
#pragma unroll
        for (int u = 0; u < LPP / 2; ++u) {
          if (u >= half) break;
          const int give = up ? x[u] : x[u + half], mine = up ? x[u + half] : x[u];
          x[u] = mine + __shfl_xor_sync(0xffffffffu, give, half);
        }
      }
      best = fmaxf(best, static_cast<float>(x[0]) * unit[g]);
    }
    if (p < m) {
      const uint32_t key = key_of(page < 0 ? -INFINITY : s < INFINITY ? best * s : INFINITY);
      if (clusters > 1)
        store_first(keys + p, key);
      else
        keys[p] = key;
    }
  }
  if (clusters > 1) {
    cluster_arrive_wait();
    if (rank != 0) return;
  } else {
    __syncthreads();
  }
  // ---- the smallest key to keep: digits of 8 bits from the highest bit in which keys differ ----
  uint32_t low = 0xFFFFFFFFu, high = 0u;
  for (int k = threadIdx.x; k < m; k += SEL_THREADS) {
    low = min(low, keys[k]);
    high = max(high, keys[k]);
  }
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (threadIdx.x == 0) {
    ends[0] = 0xFFFFFFFFu;
    ends[1] = 0u;
  }
  __syncthreads();
  if (lane == 0) {
    atomicMin(&ends[0], low);
    atomicMax(&ends[1], high);
  }
  __syncthreads();
  low = ends[0];
  high = ends[1];
  int top = 32 - __clz(low ^ high);  // bits below `top` differ
  uint32_t bound = top < 32 ? (high >> top) << top : 0u;  // keys to keep are at least this, as far as it is known
  int left = want;  // how many of those that agree with bound above bit `top`
  while (top > 0) {
    const int shift = max(top - 8, 0);
    hist[threadIdx.x] = 0u;
    __syncthreads();
    for (int k = threadIdx.x; k < m; k += SEL_THREADS) {
      const uint32_t key = keys[k];
      if (top == 32 || (key >> top) == (bound >> top)) atomicAdd(&hist[(key >> shift) & ((1u << (top - shift)) - 1u)], 1u);
    }
    __syncthreads();
    if (warp == 0) {  // lane l: digits 8 (31 - l) + 7 .. 8 (31 - l), from the largest down
      uint32_t own = 0u, v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) own += v[k] = hist[8 * (31 - lane) + 7 - k];
      uint32_t before = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += o;
      }
      before -= own;
      const uint32_t need = static_cast<uint32_t>(left);
      if (before < need && before + own >= need) {
        int k = 0;
        while (before + v[k] < need) before += v[k++];
        found[0] = static_cast<uint32_t>(8 * (31 - lane) + 7 - k);
        found[1] = need - before;
      }
    }
    __syncthreads();
    bound |= found[0] << shift;
    left = static_cast<int>(found[1]);
    top = shift;
  }
  // ---- the list: keys above the bound, and the first `left` that equal it; every warp a stretch of the pages ----
  const int per = (m + SEL_THREADS - 1) / SEL_THREADS * 32, k0 = min(warp * per, m), k1 = min(k0 + per, m);
  uint32_t above = 0u, equal = 0u;
  for (int k = k0; k < k1; k += 32) {
    const uint32_t key = k + lane < k1 ? keys[k + lane] : 0u;
    above += __popc(__ballot_sync(0xffffffffu, k + lane < k1 && key > bound));
    equal += __popc(__ballot_sync(0xffffffffu, k + lane < k1 && key == bound));
  }
  if (lane == 0) {
    count[warp][0] = above;
    count[warp][1] = equal;
  }
  __syncthreads();
  uint32_t at = a.first, ties = 0u;  // where this warp's pages go, ties in front of its own
  for (int w = 0; w < warp; ++w) {
    const uint32_t room = static_cast<uint32_t>(left) - min(ties, static_cast<uint32_t>(left));
    at += count[w][0] + min(count[w][1], room);
    ties += count[w][1];
  }
  for (int k = k0; k < k1; k += 32) {
    const bool in = k + lane < k1;
    const uint32_t key = in ? keys[k + lane] : 0u, mask = (1u << lane) - 1u;
    const uint32_t eq = __ballot_sync(0xffffffffu, in && key == bound);
    const bool take = in && (key > bound || (key == bound && ties + __popc(eq & mask) < static_cast<uint32_t>(left)));
    const uint32_t taken = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(taken & mask)] = table[a.first + k + lane];
    at += __popc(taken);
    ties += __popc(eq);
  }
}

// A bounds array for the pool: its bytes fit and it is aligned.
int check_bounds(const void *bounds, size_t bytes, const Cache4 &c) {
  if (c.n_pages && !bounds) return fail(SPARGE_ERR_INVALID_ARG, "bounds is NULL");
  if (reinterpret_cast<uintptr_t>(bounds) & 15u) return fail(SPARGE_ERR_INVALID_ARG, "bounds not 16-byte aligned");
  const size_t need = static_cast<size_t>(c.n_pages) * static_cast<size_t>(bounds_row(c.H, c.d));
  if (bytes < need) return fail(SPARGE_ERR_INVALID_ARG, "bounds: %zu bytes, the pool needs %zu", bytes, need);
  return SPARGE_OK;
}
int check_table(const Cache4 &c, int64_t B, const void *table, int64_t width, int64_t stride, const void *lens) {
  if (B < 0 || B > 65535) return fail(SPARGE_ERR_UNSUPPORTED, "B=%lld not in 0..65535", (long long)B);
  if (width < 0 || stride < width || width > INT_MAX / c.page_size)
    return fail(SPARGE_ERR_INVALID_ARG, "table width %lld and stride %lld: the stride must reach the width, the width 2^31 tokens at most",
                (long long)width, (long long)stride);
  if (B && (!lens || (width && !table))) return fail(SPARGE_ERR_INVALID_ARG, "table or kv_lens is NULL");
  return SPARGE_OK;
}

}  // namespace
}  // namespace sparge

using namespace sparge;

extern "C" {

size_t sparge_cache4_bounds_bytes(int64_t n_pages, int H, int d) {
  if (n_pages < 0 || n_pages > INT32_MAX || H <= 0 || H > 65535 || (d != 64 && d != 128)) return 0;
  return static_cast<size_t>(n_pages) * static_cast<size_t>(bounds_row(H, d));
}

int sparge_cache4_bounds_update(const sparge_cache4 *cache, const int32_t *table, int64_t B, int64_t width, int64_t table_stride,
                                const int32_t *kv_lens, int64_t N, void *bounds, size_t bounds_bytes, sparge_stream_t stream) {
  clear_error();
  Cache4 c;
  int rc;
  if ((rc = check_cache4(cache, &c)) || (rc = check_bounds(bounds, bounds_bytes, c)) ||
      (rc = check_table(c, B, table, width, table_stride, kv_lens)))
    return rc;
  if (N < 0) return fail(SPARGE_ERR_INVALID_ARG, "N=%lld is negative", (long long)N);
  if (B == 0 || N == 0 || width == 0) return SPARGE_OK;
  BoundsArgs a = {};
  a.pool = c.data;
  a.bounds = static_cast<uint8_t *>(bounds);
  a.table = table;
  a.lens = kv_lens;
  a.table_stride = table_stride;
  a.n_pages = c.n_pages;
  a.row = bounds_row(c.H, c.d);
  a.N = N < INT_MAX ? N : INT_MAX;
  a.width = static_cast<int>(width);
  a.page_shift = c.page_shift;
  a.H = c.H;
  const int64_t most = (a.N + c.page_size - 2) / c.page_size + 1;
  a.most = static_cast<int>(most < width ? most : width);
  a.status = status_ptr();
  if (B * a.most > INT_MAX) return fail(SPARGE_ERR_UNSUPPORTED, "too many pages");
  const dim3 grid(static_cast<unsigned>(B * a.most), static_cast<unsigned>((c.H + 3) / 4));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c.d == 128 ? launch_dependent(bounds_update_kernel<128>, grid, 128, 0, s, a)
                                   : launch_dependent(bounds_update_kernel<64>, grid, 128, 0, s, a);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "page bounds launch");
}

int sparge_cache4_bounds_load(const sparge_cache4 *cache, const void *bounds, size_t bounds_bytes, const int32_t *pages, int64_t n,
                              void *hi, void *lo, sparge_stream_t stream) {
  clear_error();
  Cache4 c;
  int rc;
  if ((rc = check_cache4(cache, &c)) || (rc = check_bounds(bounds, bounds_bytes, c))) return rc;
  if (n < 0) return fail(SPARGE_ERR_INVALID_ARG, "n=%lld is negative", (long long)n);
  if (n == 0) return SPARGE_OK;
  if (!pages || !hi || !lo) return fail(SPARGE_ERR_INVALID_ARG, "pages, hi or lo is NULL");
  if ((reinterpret_cast<uintptr_t>(hi) | reinterpret_cast<uintptr_t>(lo)) & 15u)
    return fail(SPARGE_ERR_INVALID_ARG, "hi and lo must be 16-byte aligned");
  const int64_t per = c.H * (c.d / 8);
  if (n > (int64_t(INT_MAX) * 256 - 255) / per) return fail(SPARGE_ERR_UNSUPPORTED, "too many pages");
  BoundsArgs a = {};
  a.bounds = const_cast<uint8_t *>(static_cast<const uint8_t *>(bounds));
  a.pages = pages;
  a.n_pages = c.n_pages;
  a.row = bounds_row(c.H, c.d);
  a.count = n;
  a.H = c.H;
  a.hi = static_cast<__nv_bfloat16 *>(hi);
  a.lo = static_cast<__nv_bfloat16 *>(lo);
  a.status = status_ptr();
  const dim3 grid(static_cast<unsigned>((n * per + 255) / 256));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c.d == 128 ? launch_dependent(bounds_load_kernel<128>, grid, 256, 0, s, a)
                                   : launch_dependent(bounds_load_kernel<64>, grid, 256, 0, s, a);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "page bounds load launch");
}

int sparge_cache4_select(const sparge_tensor *q, const sparge_cache4 *cache, const void *bounds, size_t bounds_bytes,
                         const int32_t *table, int64_t width, int64_t table_stride, const int32_t *kv_lens, int64_t keep,
                         int64_t first, int64_t last, int32_t *pages, int32_t *lens, sparge_stream_t stream) {
  clear_error();
  View qv;
  Cache4 c;
  int rc;
  if ((rc = check_tensor(q, "q", &qv)) || (rc = check_cache4(cache, &c)) || (rc = check_bounds(bounds, bounds_bytes, c)) ||
      (rc = check_table(c, qv.B, table, width, table_stride, kv_lens)))
    return rc;
  if (qv.d != c.d) return fail(SPARGE_ERR_INVALID_ARG, "q and the cache disagree in d");
  if (qv.H % c.H) return fail(SPARGE_ERR_UNSUPPORTED, "Hq=%lld not a multiple of the cache's %d heads", (long long)qv.H, c.H);
  if (qv.H / c.H > SEL_HEADS)
    return fail(SPARGE_ERR_UNSUPPORTED, "%lld query heads per key/value head: at most %d", (long long)(qv.H / c.H), SEL_HEADS);
  if (width > SEL_PAGES) return fail(SPARGE_ERR_UNSUPPORTED, "table width %lld: at most %d pages", (long long)width, SEL_PAGES);
  if (first < 0 || last < 1 || keep > INT_MAX / c.page_size || first > keep || last > keep - first)
    return fail(SPARGE_ERR_INVALID_ARG, "first=%lld >= 0, last=%lld >= 1 and their sum at most keep=%lld, keep 2^31 tokens at most",
                (long long)first, (long long)last, (long long)keep);
  if (qv.B * qv.N == 0) return SPARGE_OK;
  if (!pages || !lens) return fail(SPARGE_ERR_INVALID_ARG, "pages or lens is NULL");
  if (lens == kv_lens) return fail(SPARGE_ERR_INVALID_ARG, "lens must not be kv_lens: every list reads those");
  const int64_t lists = qv.B * qv.N * c.H;
  if (lists > INT_MAX / 8) return fail(SPARGE_ERR_UNSUPPORTED, "too many queries");
  SelectArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(qv.data);
  a.q_sb = qv.sb; a.q_sh = qv.sh; a.q_sn = qv.sn;
  a.bounds = static_cast<const uint8_t *>(bounds);
  a.table = table;
  a.lens = kv_lens;
  a.table_stride = table_stride;
  a.n_pages = c.n_pages;
  a.row = bounds_row(c.H, c.d);
  a.width = static_cast<int>(width);
  a.page_shift = c.page_shift;
  a.Hkv = c.H;
  a.G = static_cast<int>(qv.H / c.H);
  a.Nq = static_cast<int>(qv.N);
  a.keep = static_cast<int>(keep);
  a.first = static_cast<int>(first);
  a.last = static_cast<int>(last);
  a.pages = pages;
  a.out_lens = lens;
  a.status = status_ptr();
  // CTAs of a list: two for every SM in all, each with at least one round of its warps
  unsigned cluster = 1;
  while (cluster < 8 && lists * cluster < 152 && static_cast<int64_t>(cluster) * SEL_THREADS < width) cluster *= 2;
  const size_t smem = static_cast<size_t>((width * 4 + 15) / 16 * 16) + static_cast<size_t>(a.G) * 2 * c.d;
  static std::atomic<unsigned long long> set64{0}, set128{0};
  constexpr int MOST = SEL_PAGES * 4 + SEL_HEADS * 2 * 128;
  cudaError_t e = c.d == 128 ? set_smem_limit_once(select_kernel<128>, MOST, set128) : set_smem_limit_once(select_kernel<64>, MOST, set64);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(lists * cluster));
  if (e == cudaSuccess)
    e = c.d == 128 ? launch_dependent_clusters(select_kernel<128>, grid, SEL_THREADS, smem, cluster, s, a)
                   : launch_dependent_clusters(select_kernel<64>, grid, SEL_THREADS, smem, cluster, s, a);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "page selection launch");
}

}  // extern "C"
