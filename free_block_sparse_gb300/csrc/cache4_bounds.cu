// Pages of the 4-bit cache that matter to a query: bounds of each page's keys, and the selection by them.
//
// Bounds.  For every page and KV head the largest and smallest key of each channel, hi_c and lo_c, over the page's
// tokens as the cache reads them back, in int8 codes of one power of two s per page and head, rounded
// outwards: hi = s ceil(hi_c / s), lo = s floor(lo_c / s), s the least power of two with every |code| <= 127 (at least
// 2^-126).  A page that holds an infinity or a NaN has s = infinity.
// Score of a page for a query row: r_c = round-to-even(q_c / t), t a power of two in the same way, and
//   t s sum_c max(r_c hi_c, r_c lo_c) = t s (sum r+ hi + sum r- lo),   r+ = max(r, 0), r- = min(r, 0),
// which no token of the page exceeds in t r . k.  A KV head's score is the largest of its heads'.  The sums are whole numbers below 2^21
// and the factors powers of two, so the selection does not depend on the order of any sum.  Scores are held in units of 2^15 times the
// largest t of the group's heads, which changes no list: so none leaves fp32's range (they stay below 2^128), and each is exact where its head's t / that
// largest * s is 2^-134 or more.  d + d bytes of codes per page and head in place of 9 d / 16 for every token.
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

// 2^-15 / t for t = 2^-126 .. 2^121 (0 for 0: rows that have no say)
__device__ __forceinline__ float score_unit(float t) { return t > 0.f ? over_unit(t) * 0x1p-15f : 0.f; }

__device__ __forceinline__ float fmin3(float a, float b, float c) {  // as fmax3: a NaN among them counts for nothing
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

struct BoundsArgs {
  const uint8_t *pool;
  uint8_t *bounds;
  const int32_t *table, *lens, *pages;
  int64_t table_stride, n_pages, row, N, count;
  int B, width, page_shift, H, most;  // most: pages of a sequence that its last N tokens can lie on
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
// Dependent latencies bound it: length, page, then one record after another (a record's loads wait until the one before is reduced: four in a
// page of 64 tokens, sixteen in one of 256), write.  An update for 256 sequences of one new token and the reading back of their pages
// take 9.5 us, for 4 of 8192 16.2 (23 MB), of which the reading back is 2 and 3.5.  Two warps for a page's 128 channels, twice the warps
// resident, took 0.8 and 2.7 us more; the search for a longer sequence on the page two rows at a time, in 96 registers for 127, 10.4 and 15.7.
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
  if (from >= len) return;
  const int page = a.table[static_cast<int64_t>(b) * a.table_stride + col];
  const int P = 1 << a.page_shift, n = static_cast<int>(len - from < P ? len - from : P);
  // sequences that hold the page in common (a fork) may count different numbers of its tokens: the most of them, by that one's warps
  if (n < P) {
    bool more = false;
    for (int o = threadIdx.x; o < a.B; o += 128) {
      const int theirs = length_of(a.lens, o, a.width, a.page_shift), p = a.table[static_cast<int64_t>(o) * a.table_stride + col];
      more = more || (p == page && theirs > len);
    }
    if (__syncthreads_or(more)) return;
  }
  if (h >= a.H) return;
  if (page < 0 || page >= a.n_pages) {
    if (lane == 0) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
    return;
  }
  const uint8_t *src = a.pool + (static_cast<int64_t>(page) * a.H + h) * (static_cast<int64_t>(P / C4_TOKENS) * R::BYTES);
  float hi[NV], lo[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    hi[i] = -INFINITY;
    lo[i] = INFINITY;
  }
  bool bad = false;
  // two tokens at a time, one of every record's halves: a value then costs half a three-way maximum and minimum
#pragma unroll 1
  for (int t0 = 0; t0 < n; t0 += C4_TOKENS) {
    const uint8_t *rec = src + (t0 >> 4) * R::BYTES;
    uint32_t k[2][NW], word[2][R::NG];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int t = 8 * y + tt;
#pragma unroll
      for (int w = 0; w < NW; ++w) k[y][w] = 0u;
#pragma unroll
      for (int g = 0; g < R::NG; ++g) word[y][g] = 0x7FC07FC0u;  // a token that is not there: NaN, which no maximum takes
      if (t0 + t < n) {
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4 *>(rec + R::K + t * (D / 2) + c * (D / 8));
          const uint2 w = *reinterpret_cast<const uint2 *>(rec + R::KW + t * 8);
          k[y][0] = u.x; k[y][1] = u.y; k[y][2] = u.z; k[y][3] = u.w;
          word[y][0] = w.x; word[y][1] = w.y;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(rec + R::K + t * (D / 2) + c * (D / 8));
          k[y][0] = u.x; k[y][1] = u.y;
          word[y][0] = *reinterpret_cast<const uint32_t *>(rec + R::KW + t * 4);
        }
#pragma unroll
        for (int g = 0; g < R::NG; ++g)
          bad = bad || !(fabsf(bf16lo(word[y][g])) < INFINITY) || !(fabsf(bf16hi(word[y][g])) < INFINITY);
      }
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float2 x[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t even = k[y][w] & 0x0F0F0F0Fu, odd = (k[y][w] >> 4) & 0x0F0F0F0Fu;
          const float s = bf16lo(word[y][w / 2]), m = bf16hi(word[y][w / 2]);
          // a code's byte becomes the low byte of 2^23 (code + 2^23, exactly)
          const float2 f = fadd2(make_float2(__uint_as_float(__byte_perm(even, 0x4B000000u, 0x7650 + j / 2)),
                                             __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7650 + j / 2))),
                                 make_float2(-8388608.f, -8388608.f));
          x[y] = ffma2(f, make_float2(s, s), make_float2(m, m));
        }
        hi[8 * w + j] = fmax3(hi[8 * w + j], x[0].x, x[1].x);
        lo[8 * w + j] = fmin3(lo[8 * w + j], x[0].x, x[1].x);
        hi[8 * w + j + 1] = fmax3(hi[8 * w + j + 1], x[0].y, x[1].y);
        lo[8 * w + j + 1] = fmin3(lo[8 * w + j + 1], x[0].y, x[1].y);
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
// Selection, in two kernels.  The first scores pages: all sequences' and heads' pages stand in one line of stretches that is
// cut into equal shares, one per CTA, so ragged lengths fill the part evenly; a warp takes 16 pages at a time against the
// rows of up to SEL_ROWS query heads, on mma.sync with the codes as f16 (whole numbers up to 127; sums below 2^21 are exact in fp32 in any
// order).  It is bound by the latency of its chain - page number, bounds, product - so both are loaded a step ahead, 4 KB a warp, and
// 16 warps share an SM: 384 lists of up to 8K pages, d = 64, 24 us for 54 MB of bounds (2.2 TB/s).
// The second has a CTA for each list: it takes the list's scores into shared memory, finds the smallest to keep, and writes the
// pages in order.  That score comes from one histogram of 256 equal steps between the smallest
// and the largest score, then the scores of the step that holds it are ranked among themselves; more than 256 of them, or infinities
// at the ends, go digit by digit from the highest bit that differs.  14 us for those lists: barriers and latencies of its six passes.
// --------------------------------------------------------------------------------------------
struct SelectArgs {
  const __nv_bfloat16 *q;
  int64_t q_sb, q_sh, q_sn;
  const uint8_t *bounds;
  const int32_t *table, *lens;
  int64_t table_stride, n_pages, row;
  int B, width, page_shift, Hkv, G, Nq, keep, first, last;
  int rows_log;  // rows of a query in the product: 1, 2 or 4 (three heads: the first again), or tiles of 8
  int tiles;     // of a query; 0: a tile holds 8 >> rows_log queries
  int at_once;   // queries of a round (blockIdx.y)
  float *keys;     // scores [B][Nq][Hkv][pitch]; -inf: a page that is not there
  int pitch;       // the table's width in whole fours
  int32_t *pages, *out_lens;
  int *status;

  __device__ __forceinline__ int tokens(int len, int i) const {  // that query i sees
    const int64_t n = static_cast<int64_t>(len) - Nq + 1 + i;
    return static_cast<int>(n > 0 ? n : 0);
  }
  __device__ __forceinline__ int pages_of(int len, int i) const {
    return static_cast<int>((static_cast<int64_t>(tokens(len, i)) + (1 << page_shift) - 1) >> page_shift);
  }
  // pages to choose from (0: all of them are kept, or none is left to choose)
  __device__ __forceinline__ int choices(int len, int i) const {
    const int n = pages_of(len, i);
    return n > keep && keep > first + last ? n - first - last : 0;
  }
};

constexpr int SEL_THREADS = 128, SEL_WARPS = SEL_THREADS / 32;
// of an SM; d = 128: four (128 registers, spills) took 23.0 us a call for 8 lists of 512 pages and 88.5 for 512, three 21.8 and 85.7
__host__ __device__ constexpr int sel_ctas(int D) { return D == 128 ? 3 : 4; }
constexpr int SEL_STRETCH = SEL_WARPS * 16;   // pages of a CTA and step
constexpr int SEL_HEADS = 64, SEL_ROWS = 64;  // query heads of a KV head at most; rows of a round
constexpr int SEL_PAGES = 32768;              // scores that shared memory holds

// Codes as f16, two channels a register.
__device__ __forceinline__ uint32_t half2_of(int lo, int hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(static_cast<float>(hi)), "f"(static_cast<float>(lo)));
  return r;
}
// Four int8 codes: b + 128 in the low bits of 1024 + .., less 1152.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &a, uint32_t &b) {
  const uint32_t u = w ^ 0x80808080u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}
__device__ __forceinline__ void mma_codes(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint2 b) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// Codes of query row r by a warp, as B operands: step k of the product holds, for lane 4 n + c of row n of the tile, channels
// 64 j + 16 c + 4 w .. + 3 with k = 4 j + w - the bytes that a lane reads of a page - first of r+ (beside hi), then of r- (beside lo).
// Returns t (0 for a row with an infinity or a NaN: it scores every page 0).
template <int D>
__device__ __forceinline__ float code_row(const uint32_t (&u)[D / 64], uint8_t *codes, int r, int lane) {
  constexpr int C = D / 32, S = D / 8;
  float x[C], big = 0.f;
  bool fine = true;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    x[k] = (k & 1) ? bf16hi(u[k / 2]) : bf16lo(u[k / 2]);
    fine = fine && fabsf(x[k]) < INFINITY;
    big = fmaxf(big, fabsf(x[k]));
  }
  fine = __all_sync(0xffffffffu, fine);
  big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
  const float t = fine ? code_unit(big) : 0.f, inv = fine ? over_unit(t) : 0.f;
  int v[C];
#pragma unroll
  for (int k = 0; k < C; ++k) v[k] = fine ? __float2int_rn(x[k] * inv) : 0;
  uint8_t *tile = codes + (r / 8) * (S * 256);
  if constexpr (C == 4) {
    const int k = 4 * (lane >> 4) + (lane & 3), at = 4 * (r % 8) + ((lane >> 2) & 3);
    *reinterpret_cast<uint2 *>(tile + (k * 32 + at) * 8) = make_uint2(half2_of(max(v[0], 0), max(v[1], 0)), half2_of(max(v[2], 0), max(v[3], 0)));
    *reinterpret_cast<uint2 *>(tile + ((k + S / 2) * 32 + at) * 8) =
        make_uint2(half2_of(min(v[0], 0), min(v[1], 0)), half2_of(min(v[2], 0), min(v[3], 0)));
  } else {
    const int k = (lane >> 1) & 3, at = 4 * (r % 8) + (lane >> 3);
    *reinterpret_cast<uint32_t *>(tile + (k * 32 + at) * 8 + 4 * (lane & 1)) = half2_of(max(v[0], 0), max(v[1], 0));
    *reinterpret_cast<uint32_t *>(tile + ((k + S / 2) * 32 + at) * 8 + 4 * (lane & 1)) = half2_of(min(v[0], 0), min(v[1], 0));
  }
  return t;
}

template <int D>
__global__ void __launch_bounds__(SEL_THREADS, sel_ctas(D)) select_score_kernel(const SelectArgs a) {
  constexpr int S = D / 8, NP = D / 32;  // steps of a product, 16 codes each, hi's then lo's; 16-byte pieces of a page and lane
  __shared__ __align__(16) uint8_t codes[SEL_ROWS * 4 * D];
  __shared__ float2 unit[SEL_ROWS / 2];  // t of the rows, in the unit of their query where it has no more than four
  __shared__ float top[SEL_ROWS / 4];    // the largest t of four rows
  __shared__ int limit[SEL_ROWS];        // pages to choose from of each query of the round
  start_after_earlier();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int i0 = blockIdx.y * a.at_once, ni = min(a.at_once, a.Nq - i0);
  // ---- this CTA's share of the line: every warp for itself; the last query of the round sees the most pages ----
  auto stretches = [&](int b) {
    return static_cast<int64_t>((a.choices(length_of(a.lens, b, a.width, a.page_shift), i0 + ni - 1) + SEL_STRETCH - 1) / SEL_STRETCH) * a.Hkv;
  };
  const int per = (a.B + 31) / 32, bt = min(a.B, lane * per), bu = min(a.B, bt + per);
  int64_t own = 0;
#pragma unroll 4
  for (int b = bt; b < bu; ++b) own += stretches(b);
  int64_t inc = own;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  const int64_t total = __shfl_sync(0xffffffffu, inc, 31);
  const int64_t begin = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
  if (begin >= end) return;
  int b = bt;
  int64_t off = begin - (inc - own), left = end - begin;
  const uint32_t here = __ballot_sync(0xffffffffu, off >= 0 && off < own);  // the lane whose sequences hold the start
  if (off >= 0 && off < own)
    for (int64_t n; off >= (n = stretches(b)); ++b) off -= n;
  b = __shfl_sync(0xffffffffu, b, __ffs(here) - 1);
  off = __shfl_sync(0xffffffffu, off, __ffs(here) - 1);
  while (left > 0) {
    const int len = length_of(a.lens, b, a.width, a.page_shift), most = a.choices(len, i0 + ni - 1), nst = (most + SEL_STRETCH - 1) / SEL_STRETCH;
    if (off >= static_cast<int64_t>(nst) * a.Hkv) {
      off -= static_cast<int64_t>(nst) * a.Hkv;
      ++b;
      continue;
    }
    const int h = static_cast<int>(off) / nst, s0 = static_cast<int>(off) - h * nst;
    const int s1 = static_cast<int>(left < nst - s0 ? s0 + left : nst);  // stretches s0 .. s1 - 1 of the head
    off += s1 - s0;
    left -= s1 - s0;
    const int32_t *table = a.table + static_cast<int64_t>(b) * a.table_stride + a.first;
    const uint8_t *base = a.bounds + h * 2 * D + 16 * c, *scales = a.bounds + a.Hkv * 2 * D + 4 * h;
    // ---- the pages' numbers of the first step, and the queries' codes meanwhile ----
    const int p_end = min(most, s1 * SEL_STRETCH);
    int p0 = s0 * SEL_STRETCH + warp * 16;
    int id[2];  // of the step after this one: pages g and g + 8 of each tile
    auto look_up = [&](int p) {
#pragma unroll
      for (int y = 0; y < 2; ++y) id[y] = p + g + 8 * y < p_end ? table[p + g + 8 * y] : -1;
    };
    look_up(p0);
    const int rows = a.tiles ? ni * a.tiles * 8 : ni << a.rows_log, nt = (rows + 7) / 8;
    __syncthreads();  // the codes of the head before have been read
    for (int r0 = warp * 4; r0 < rows; r0 += SEL_WARPS * 4) {  // (the last tile's rows past them hold anything: no sum of another row's)
      uint32_t u[4][D / 64];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + k, i = a.tiles ? r / (8 * a.tiles) : r >> a.rows_log, hd = a.tiles ? r % (8 * a.tiles) : r & ((1 << a.rows_log) - 1);
        const __nv_bfloat16 *q = a.q + b * a.q_sb + (static_cast<int64_t>(h) * a.G + (hd < a.G ? hd : 0)) * a.q_sh +
                                 static_cast<int64_t>(i0 + min(i, ni - 1)) * a.q_sn;
        if constexpr (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2 *>(q + 4 * lane);
          u[k][0] = x.x;
          u[k][1] = x.y;
        } else {
          u[k][0] = *reinterpret_cast<const uint32_t *>(q + 2 * lane);
        }
      }
      float t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = code_row<D>(u[k], codes, r0 + k, lane);
      const float t01 = fmaxf(t[0], t[1]), t23 = fmaxf(t[2], t[3]), all = fmaxf(t01, t23);
      if (lane < 4) {
        const float own = lane == 0 ? t[0] : lane == 1 ? t[1] : lane == 2 ? t[2] : t[3];
        const float most = a.rows_log == 0 ? own : a.rows_log == 1 ? (lane < 2 ? t01 : t23) : all;
        reinterpret_cast<float *>(unit)[r0 + lane] = a.tiles ? own : own * score_unit(most);
      }
      if (lane == 0) top[r0 / 4] = all;
    }
    for (int i = threadIdx.x; i < ni; i += SEL_THREADS) limit[i] = a.choices(len, i0 + i);
    float *keys = a.keys + ((static_cast<int64_t>(b) * a.Nq + i0) * a.Hkv + h) * a.pitch + g;
    const int64_t query = static_cast<int64_t>(a.Hkv) * a.pitch;
    __syncthreads();
    // ---- 16 pages a step: lane 4 g + c reads of pages g and g + 8 of a tile the 16 codes from 64 j + 16 c on, and holds the sums of
    // rows 2c and 2c + 1 with them ----
    uint4 code[2][NP] = {};  // (of a page that is not there: those of one before)
    float next[2];  // the pages' scales; NaN: there is no such page
    auto fetch = [&](int p) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const bool there = static_cast<uint32_t>(id[y]) < static_cast<uint32_t>(a.n_pages);
        const int64_t at = static_cast<int64_t>(id[y]) * a.row;
        if (!there && p + g + 8 * y < p_end) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
        next[y] = __uint_as_float(0x7FFFFFFFu);
        if (there) {
#pragma unroll
          for (int k = 0; k < NP; ++k) code[y][k] = *reinterpret_cast<const uint4 *>(base + at + 64 * k);
          next[y] = *reinterpret_cast<const float *>(scales + at);
        }
      }
    };
    fetch(p0);
    look_up(p0 + SEL_STRETCH);
    for (; p0 < p_end; p0 += SEL_STRETCH) {
      uint32_t w[S][4];  // the pages' codes as A operands
      float s[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        s[y] = next[y];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          const uint4 v = code[y][k];
          widen4(v.x, w[4 * k][y], w[4 * k][2 + y]);
          widen4(v.y, w[4 * k + 1][y], w[4 * k + 1][2 + y]);
          widen4(v.z, w[4 * k + 2][y], w[4 * k + 2][2 + y]);
          widen4(v.w, w[4 * k + 3][y], w[4 * k + 3][2 + y]);
        }
      }
      fetch(p0 + SEL_STRETCH);
      look_up(p0 + 2 * SEL_STRETCH);
      float best[2];  // of a query of several tiles of rows
      best[0] = best[1] = -INFINITY;
      int i = 0, nth = 0;  // of a query of whole tiles: the query, its tile
      float of_query = 1.f;
      const uint8_t *tile = codes + lane * 8;
#pragma unroll 1
      for (int t = 0; t < nt; ++t, tile += S * 256) {
        float acc[4];
        acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
        for (int k = 0; k < S; ++k) {
          const uint2 q = *reinterpret_cast<const uint2 *>(tile + k * 256);
          mma_codes(acc, w[k][0], w[k][1], w[k][2], w[k][3], q);
        }
        if (a.tiles && nth == 0) {
          float most = 0.f;
          for (int x = 0; x < 2 * a.tiles; ++x) most = fmaxf(most, top[2 * t + x]);
          of_query = score_unit(most);
        }
        const float2 un = make_float2(unit[t * 4 + c].x * of_query, unit[t * 4 + c].y * of_query);
        // which lanes write: each its first row's value, the largest of a query's rows; with one row a query its second's too
        const bool several = a.rows_log > 0 || a.tiles > 0;
        const bool put = !several || (a.tiles ? c == 0 && nth == a.tiles - 1 : a.rows_log == 1 || (c & 1) == 0);
        const int at = a.tiles ? i : (t * 8 + 2 * c) >> a.rows_log;
        const int lim0 = (put && at < ni ? limit[at] : 0) - p0 - g, lim1 = (!several && at + 1 < ni ? limit[at + 1] : 0) - p0 - g;
        float *to = keys + at * query + p0;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float v = acc[2 * y] * un.x;
          const float v1 = acc[2 * y + 1] * un.y;
          if (several) {
            v = fmaxf(v, v1);
            if (a.rows_log > 1 || a.tiles) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
            if (a.tiles) {
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
              best[y] = v = fmaxf(best[y], v);
            }
          }
          const float sc = s[y];
          auto score = [&](float x) { return sc < INFINITY ? x * sc : sc == INFINITY ? INFINITY : -INFINITY; };
          const int p = 8 * y;
          if (p < lim0) to[p] = score(v);
          if (p < lim1) to[query + p] = score(v1);
        }
        if (a.tiles && ++nth == a.tiles) {
          nth = 0;
          ++i;
          best[0] = best[1] = -INFINITY;
        }
      }
    }
  }
}

template <int T>  // threads of a list's CTA
struct ListShared {
  uint32_t hist[256];
  float cand[T], red[2][T / 32];
  uint32_t count[T / 32][2], found[3], n_cand;
  float bound;
};

__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fminf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}
__device__ __forceinline__ float warp_max(float x) { return -warp_min(-x); }

// minimum and maximum over the CTA
template <int T>
__device__ __forceinline__ void min_max(ListShared<T> &sh, float &low, float &high) {
  low = warp_min(low);
  high = warp_max(high);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.red[0][threadIdx.x >> 5] = low;
    sh.red[1][threadIdx.x >> 5] = high;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) {
    low = fminf(low, sh.red[0][w]);
    high = fmaxf(high, sh.red[1][w]);
  }
}
// The histogram's place (found[0]) that holds the want-th largest, its rank there (found[1]) and the place's count (found[2]).
template <int T>
__device__ __forceinline__ void find_place(ListShared<T> &sh, uint32_t want) {
  __syncthreads();
  if (threadIdx.x < 32) {  // lane l: places 8 (31 - l) + 7 .. 8 (31 - l), from the largest down
    const int lane = threadIdx.x;
    uint32_t own = 0u, v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) own += v[k] = sh.hist[8 * (31 - lane) + 7 - k];
    uint32_t before = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += o;
    }
    before -= own;
    if (before < want && before + own >= want) {
      bool open = true;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (open && before + v[k] >= want) {
          sh.found[0] = static_cast<uint32_t>(8 * (31 - lane) + 7 - k);
          sh.found[1] = want - before;
          sh.found[2] = v[k];
          open = false;
        }
        if (open) before += v[k];
      }
    }
  }
  __syncthreads();
}

// f(score) for every score, four at a time of a thread.  The array is filled up to whole fours with -inf: below or equal to every score,
// and behind all of them.
template <int T, typename F>
__device__ __forceinline__ void each_score(const float *scores, int m, F f) {
  const float4 *at = reinterpret_cast<const float4 *>(scores);
  const int n = (m + 3) / 4;
#pragma unroll 4
  for (int k = threadIdx.x; k < n; k += T) {
    const float4 v = at[k];
    f(v.x);
    f(v.y);
    f(v.z);
    f(v.w);
  }
}

// The want-th largest of m scores, and how many of its equals are among the want largest.  Called by the whole CTA; low and high:
// the smallest and the largest score that the thread has seen.
template <int T>
__device__ __forceinline__ void want_th(ListShared<T> &sh, const float *scores, int m, int want, float low, float high, float &bound, int &left) {
  if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0u;
  if (threadIdx.x == 0) sh.n_cand = 0u;
  min_max(sh, low, high);
  const float range = high - low;
  left = want;
  if (range > 1e-30f && range < 1e30f) {
    const float step = 255.f / range, zero = low;
    auto place = [&](float x) { return min(static_cast<uint32_t>((x - zero) * step), 255u); };  // (-inf: 0)
    each_score<T>(scores, m, [&](float x) { atomicAdd(&sh.hist[place(x)], 1u); });
    find_place(sh, static_cast<uint32_t>(want));
    const uint32_t at = sh.found[0], n = sh.found[2];
    left = static_cast<int>(sh.found[1]);
    if (n <= T) {
      each_score<T>(scores, m, [&](float x) {
        if (place(x) == at) sh.cand[atomicAdd(&sh.n_cand, 1u)] = x;
      });
      __syncthreads();
      if (threadIdx.x < n) {
        const float mine = sh.cand[threadIdx.x];
        uint32_t above = 0u, equal = 0u;
        for (uint32_t k = 0; k < n; ++k) {
          above += sh.cand[k] > mine;
          equal += sh.cand[k] == mine;
        }
        if (above < static_cast<uint32_t>(left) && above + equal >= static_cast<uint32_t>(left)) {
          sh.bound = mine;
          sh.found[1] = static_cast<uint32_t>(left) - above;
        }
      }
      __syncthreads();
      bound = sh.bound;
      left = static_cast<int>(sh.found[1]);
      return;
    }
    low = INFINITY;
    high = -INFINITY;
    each_score<T>(scores, m, [&](float x) {
      if (place(x) == at) {
        low = fminf(low, x);
        high = fmaxf(high, x);
      }
    });
    min_max(sh, low, high);
  }
  // digits of 8 bits among the scores from low to high, as unsigned numbers of the same order (both zeros are one)
  auto key_of = [](float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
  };
  const uint32_t first = key_of(low), last = key_of(high);
  int top = 32 - __clz(first ^ last);  // bits below `top` differ
  uint32_t key = top < 32 ? (last >> top) << top : 0u;
  while (top > 0) {
    const int shift = max(top - 8, 0);
    __syncthreads();
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0u;
    __syncthreads();
    each_score<T>(scores, m, [&](float x) {
      const uint32_t k = key_of(x);
      if (k >= first && k <= last && (top == 32 || (k >> top) == (key >> top)))
        atomicAdd(&sh.hist[(k >> shift) & ((1u << (top - shift)) - 1u)], 1u);
    });
    find_place(sh, static_cast<uint32_t>(left));
    key |= sh.found[0] << shift;
    left = static_cast<int>(sh.found[1]);
    top = shift;
  }
  bound = __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
}

template <int T>
__global__ void __launch_bounds__(T) select_list_kernel(const SelectArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ ListShared<T> sh;
  start_after_earlier();
  float4 *scores = reinterpret_cast<float4 *>(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, P = 1 << a.page_shift;
  const int64_t list = blockIdx.x;
  const int h = static_cast<int>(list % a.Hkv), i = static_cast<int>(list / a.Hkv % a.Nq), b = static_cast<int>(list / a.Hkv / a.Nq);
  const int32_t *table = a.table + static_cast<int64_t>(b) * a.table_stride;
  const int len = length_of(a.lens, b, a.width, a.page_shift), seen = a.tokens(len, i), np = a.pages_of(len, i), n = min(np, a.keep);
  int32_t *out = a.pages + list * a.keep;
  if (h == 0 && threadIdx.x == 0)
    a.out_lens[static_cast<int64_t>(b) * a.Nq + i] = n > 0 ? static_cast<int>(static_cast<int64_t>(n - 1) * P) + (seen - 1) % P + 1 : 0;
  const int m = a.choices(len, i), m4 = (m + 3) / 4;
  float low = INFINITY, high = -INFINITY;
  const float4 *from = reinterpret_cast<const float4 *>(a.keys + list * a.pitch);
#pragma unroll 4
  for (int k = threadIdx.x; k < m4; k += T) {
    float4 v = from[k];
    if (4 * k + 3 >= m) {
      if (4 * k + 1 >= m) v.y = -INFINITY;
      if (4 * k + 2 >= m) v.z = -INFINITY;
      if (4 * k + 3 >= m) v.w = -INFINITY;
    }
    low = fminf(fminf(low, v.x), fminf(4 * k + 1 < m ? v.y : v.x, fminf(4 * k + 2 < m ? v.z : v.x, 4 * k + 3 < m ? v.w : v.x)));
    high = fmaxf(fmaxf(high, v.x), fmax3(v.y, v.z, v.w));
    scores[k] = v;
  }
  // every page, or those that are kept whatever their scores; then the places without one
  for (int k = threadIdx.x; k < a.keep; k += T) {
    const bool middle = np > a.keep && k >= a.first && k < a.keep - a.last;
    if (!middle) out[k] = k >= n ? -1 : table[np > a.keep && k >= a.first ? np - (a.keep - k) : k];
  }
  if (m == 0) return;
  __syncthreads();
  float bound;
  int left;
  want_th(sh, reinterpret_cast<const float *>(scores), m, a.keep - a.first - a.last, low, high, bound, left);
  // scores above the bound, and the first `left` that equal it: every warp a stretch, a lane four in a row; counts of those above in
  // the low and of equal ones in the high half
  const int per = (m4 + T - 1) / T * 32, f0 = min(warp * per, m4), f1 = min(f0 + per, m4);
  auto counts = [&](const float4 &v) {
    return (v.x > bound) + (v.y > bound) + (v.z > bound) + (v.w > bound) +
           (((v.x == bound) + (v.y == bound) + (v.z == bound) + (v.w == bound)) << 16);
  };
  uint32_t both = 0u;
#pragma unroll 4
  for (int k = f0 + lane; k < f1; k += 32) both += counts(scores[k]);
  const uint32_t above = __reduce_add_sync(0xffffffffu, both & 0xFFFFu), equal = __reduce_add_sync(0xffffffffu, both >> 16);
  if (lane == 0) {
    sh.count[warp][0] = above;
    sh.count[warp][1] = equal;
  }
  __syncthreads();
  uint32_t at = 0u, ties = 0u;  // in front of this warp's: scores above, equal ones
  for (int w = 0; w < warp; ++w) {
    at += sh.count[w][0];
    ties += sh.count[w][1];
  }
  // (a stretch without one to take is passed over: equal ones behind the first `left` are not taken)
  const bool some = above > 0u || (equal > 0u && ties < static_cast<uint32_t>(left));
  for (int k = f0; some && k < f1; k += 32) {
    const float4 v = k + lane < f1 ? scores[k + lane] : make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t own = k + lane < f1 ? counts(v) : 0u;
    if (!__any_sync(0xffffffffu, own != 0u)) continue;
    uint32_t sum = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += o;
    }
    uint32_t up = at + ((sum - own) & 0xFFFFu), eq = ties + ((sum - own) >> 16);
    const float x[4] = {v.x, v.y, v.z, v.w};
    if (own != 0u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool is = x[j] == bound;
        if (x[j] > bound || (is && eq < static_cast<uint32_t>(left)))
          out[a.first + up + min(eq, static_cast<uint32_t>(left))] = a.first + 4 * (k + lane) + j;
        up += x[j] > bound;
        eq += is;
      }
    const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
    at += all & 0xFFFFu;
    ties += all >> 16;
  }
  // places in the sequence's row become pages, all at once
  __syncthreads();
  for (int k = a.first + threadIdx.x; k < a.keep - a.last; k += T) out[k] = table[out[k]];
}

template <int T>
cudaError_t launch_list(const SelectArgs &a, int64_t lists, cudaStream_t s) {
  static std::atomic<unsigned long long> smem_set{0};
  if (cudaError_t e = set_smem_limit_once(select_list_kernel<T>, SEL_PAGES * 4, smem_set); e != cudaSuccess) return e;
  return launch_dependent(select_list_kernel<T>, dim3(static_cast<unsigned>(lists)), T, static_cast<size_t>((a.width + 3) / 4 * 16), s, a);
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
  a.B = static_cast<int>(B);
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

size_t sparge_cache4_select_workspace_bytes(int64_t B, int64_t Hkv, int64_t Nq, int64_t width) {
  if (B < 0 || B > 65535 || Hkv <= 0 || Hkv > 65535 || Nq < 0 || Nq > (int64_t(1) << 30) || width < 0 || width > SEL_PAGES ||
      B * Nq * Hkv > INT_MAX)
    return 0;
  return static_cast<size_t>(B * Nq * Hkv) * static_cast<size_t>((width + 3) / 4 * 16);
}

int sparge_cache4_select(const sparge_tensor *q, const sparge_cache4 *cache, const void *bounds, size_t bounds_bytes,
                         const int32_t *table, int64_t width, int64_t table_stride, const int32_t *kv_lens, int64_t keep,
                         int64_t first, int64_t last, int32_t *pages, int32_t *lens, void *ws, size_t ws_bytes,
                         sparge_stream_t stream) {
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
  const int64_t lists = qv.B * qv.N * c.H;
  if (lists > INT_MAX) return fail(SPARGE_ERR_UNSUPPORTED, "too many queries");
  if (lists == 0) return SPARGE_OK;
  const size_t need = sparge_cache4_select_workspace_bytes(qv.B, c.H, qv.N, width);
  if (need && (!ws || ws_bytes < need)) return fail(SPARGE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", ws_bytes, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(SPARGE_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  if (!pages || !lens) return fail(SPARGE_ERR_INVALID_ARG, "pages or lens is NULL");
  if (lens == kv_lens) return fail(SPARGE_ERR_INVALID_ARG, "lens must not be kv_lens: every list reads those");
  SelectArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(qv.data);
  a.q_sb = qv.sb; a.q_sh = qv.sh; a.q_sn = qv.sn;
  a.bounds = static_cast<const uint8_t *>(bounds);
  a.table = table;
  a.lens = kv_lens;
  a.table_stride = table_stride;
  a.n_pages = c.n_pages;
  a.row = bounds_row(c.H, c.d);
  a.B = static_cast<int>(qv.B);
  a.width = static_cast<int>(width);
  a.page_shift = c.page_shift;
  a.Hkv = c.H;
  a.G = static_cast<int>(qv.H / c.H);
  a.Nq = static_cast<int>(qv.N);
  a.keep = static_cast<int>(keep);
  a.first = static_cast<int>(first);
  a.last = static_cast<int>(last);
  a.keys = static_cast<float *>(ws);
  a.pitch = static_cast<int>((width + 3) / 4 * 4);
  a.pages = pages;
  a.out_lens = lens;
  a.status = status_ptr();
  a.rows_log = a.G == 1 ? 0 : a.G == 2 ? 1 : 2;
  a.tiles = a.G <= 4 ? 0 : (a.G + 7) / 8;
  const int row = a.tiles ? 8 * a.tiles : 1 << a.rows_log;
  a.at_once = SEL_ROWS / row < a.Nq ? SEL_ROWS / row : a.Nq;
  const int rounds = (a.Nq + a.at_once - 1) / a.at_once;
  if (rounds > 65535) return fail(SPARGE_ERR_UNSUPPORTED, "too many queries");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (width > keep && keep > first + last) {  // else there is nothing to choose
    const int64_t most = qv.B * c.H * ((width + SEL_STRETCH - 1) / SEL_STRETCH), full = 152 * sel_ctas(c.d), ctas = most < full ? most : full;
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(rounds));
    e = c.d == 128 ? launch_dependent(select_score_kernel<128>, grid, SEL_THREADS, 0, s, a)
                   : launch_dependent(select_score_kernel<64>, grid, SEL_THREADS, 0, s, a);
  }
  // threads of a list, the list kernel alone with 256 and 512 in us: 8 lists of 1024 pages 4.4 and 4.7, 2048 5.2 and 5.0, 4096 6.4 and
  // 6.0, 8192 9.5 and 8.4; 512 lists of 512 11.4 and 13.9, 2048 18.6 and 19.8, 2560 21.4 and 23.2, 4096 32 and 31.4, 8192 36 and 40, but 384 of 32
  // to 8192, whose longest ends last, 66 and 58 with scores and attention: the edge lies between those of few and of many lists
  if (e == cudaSuccess) e = width > 2048 ? launch_list<512>(a, lists, s) : launch_list<256>(a, lists, s);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "page selection launch");
}

}  // extern "C"
