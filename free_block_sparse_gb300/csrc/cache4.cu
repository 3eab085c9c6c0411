// The 4-bit key/value cache: storing tokens, reading them back, and the tables of its pages.
//
// Store: each token's 64-channel groups of K and V become 4-bit codes,
//   minimum = min x, scale = bf16((max x - min x) / 15), n = round((x - minimum) / scale) in 0..15
// (rounded to even; scale 0: n = 0), and go to the token's slot (page * page_size + place in the page).
// The minimum is a bf16 input and stays exact; the scale is rounded before the codes are taken, so
// the codes are nearest to what the cache will read back.  A group with an infinity or a NaN gets a
// NaN scale and minimum: it reads back as NaN instead of a plausible number.
// Load: x^ = n * scale + minimum (one rounding to bf16) from the slots.
// Both are bound by memory: 2 d bytes of bf16 and 9 d/16 bytes of cache per token, head and side.
#include <climits>
#include <cmath>

#include "../../include/sparge.h"
#include "cache4.cuh"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace sparge {
namespace {

struct Rows4 {  // K and V rows and the cache they go to or come from
  const __nv_bfloat16 *x[2];
  __nv_bfloat16 *y[2];
  int64_t sb[2], sh[2], sn[2];
  const int64_t *slots;
  uint8_t *pool;
  int64_t n_slots;
  int page_shift, H, N, B, recs;  // recs: records of a page
  int zero;                       // load: rows of left-out slots become zero
  int wide;                       // every row's 16-channel pieces are 32-byte aligned
  int *status;
};

__device__ __forceinline__ uint8_t *record_of(const Rows4 &a, int64_t slot, int h, int bytes) {
  const int64_t page = slot >> a.page_shift;
  const int g = static_cast<int>(slot & ((1 << a.page_shift) - 1)) / C4_TOKENS;
  return a.pool + ((page * a.H + h) * a.recs + g) * static_cast<int64_t>(bytes);
}

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 16 channels of a row, 32 bytes: in one piece where the rows allow it (a warp's accesses then fill whole sectors).
__device__ __forceinline__ void load16(const __nv_bfloat16 *p, bool wide, uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "l"(p));
  } else {
    const uint4 a = *reinterpret_cast<const uint4 *>(p), b = reinterpret_cast<const uint4 *>(p)[1];
    u[0] = a.x; u[1] = a.y; u[2] = a.z; u[3] = a.w;
    u[4] = b.x; u[5] = b.y; u[6] = b.z; u[7] = b.w;
  }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *p, bool wide, const uint32_t (&u)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]),
                 "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(p)[0] = make_uint4(u[0], u[1], u[2], u[3]);
    reinterpret_cast<uint4 *>(p)[1] = make_uint4(u[4], u[5], u[6], u[7]);
  }
}

// Four words of four bytes as their transpose: z[b] holds byte b of a, b, c, d.
__device__ __forceinline__ void transpose_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&z)[4]) {
  const uint32_t x0 = __byte_perm(a, b, 0x5140), x1 = __byte_perm(a, b, 0x7362);
  const uint32_t y0 = __byte_perm(c, d, 0x5140), y1 = __byte_perm(c, d, 0x7362);
  z[0] = __byte_perm(x0, y0, 0x5410);
  z[1] = __byte_perm(x0, y0, 0x7632);
  z[2] = __byte_perm(x1, y1, 0x5410);
  z[3] = __byte_perm(x1, y1, 0x7632);
}

// Place of channel ch's code among the 16 of a thread, 4 bits each: K in order; V, whose bytes hold channels g and
// g + 8, at byte g.
__device__ __forceinline__ constexpr int nibble_of(bool v, int ch) { return v ? 2 * (ch & 7) + (ch >> 3) : ch; }

// The groups that quantise16 leaves: no range, one past fp32's middle, an infinity or a NaN.  Codes in x and y; the
// word is z with the minimum's bits under the mask w.  (Out of line: the callers' loops hold the other case eight times.)
template <bool V>
__device__ __noinline__ uint4 quantise_rest(uint4 a, uint4 b, float lo, float hi) {
  if (!(fabsf(lo) <= 3.4028235e38f && fabsf(hi) <= 3.4028235e38f)) return make_uint4(0u, 0u, 0x7FC07FC0u, 0u);
  // a difference beyond fp32 (bf16 values near 3e38 of both signs) is held at the largest fp32
  const uint32_t sbits = pack_bf16x2(__fdiv_rn(fminf(hi - lo, 3.4028235e38f), 15.f), 0.f) & 0xFFFFu;
  const float s = __uint_as_float(sbits << 16);
  uint32_t n[2] = {0u, 0u};
  if (s > 0.f) {
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int ch = 0; ch < 16; ++ch) {
      const float f = ((ch & 1) ? bf16hi(u[ch / 2]) : bf16lo(u[ch / 2])) - lo;
      const int at = nibble_of(V, ch);
      n[at / 8] |= static_cast<uint32_t>(min(max(__float2int_rn(fminf(__fdiv_rn(f, s), 15.f)), 0), 15)) << (4 * (at % 8));
    }
  }
  return make_uint4(n[0], n[1], sbits, 0xFFFF0000u);
}

// Codes of a thread's 16 channels (n[0]: nibbles 0 - 7, n[1]: 8 - 15) and its group's word; the 4 threads of a
// group are adjacent lanes.  Minimum and maximum are taken on packed bf16 pairs, NaN winning, then
// together as the maximum of (max, -min), so two shuffles serve both and one test of the two
// finds an infinity or a NaN anywhere in the group.
template <bool V>
__device__ __forceinline__ uint32_t quantise16(const uint32_t (&u)[8], uint32_t (&n)[2]) {
  uint32_t lo2 = u[0], hi2 = u[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    lo2 = min2_nan(lo2, u[j]);
    hi2 = max2_nan(hi2, u[j]);
  }
  lo2 = min2_nan(lo2, lo2 >> 16);
  hi2 = max2_nan(hi2, hi2 >> 16);
  uint32_t m = __byte_perm(hi2, lo2, 0x5410) ^ 0x80000000u;  // max, -min
#pragma unroll
  for (int off = 2; off > 0; off >>= 1) m = max2_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  m ^= 0x80000000u;
  const float lo = bf16hi(m), hi = bf16lo(m);
  const float range = hi - lo;  // an infinity or a NaN if there is one in the group
  n[0] = n[1] = 0u;
  if (range >= 1e-28f && range < 1e38f) {
    // Quotients by the reciprocal and one correction by the exact remainder (Markstein, 1990: q' = q + (a - q b) r).  Rounded
    // correctly here: q is within two ulps, the fma's remainder is exact, so q' before its rounding is off by
    // about 2^-22 ulp, and a 24-bit a over an 8-bit b lies no closer than 2^-9 ulp to the middle between two floats (a - m b is a
    // whole multiple of a's last place, and not 0: an odd 25-bit m times b has more bits than a).  Where the quotient is
    // representable (a tie of codes is) it is exactly it.  scale = range / 15 (b = 15) to bf16; adding 1.5 * 2^23 to
    // (x - lo) / scale rounds it to even and leaves it in the sum's low bits (at most 15 (1 + 2^-8): no code passes 15).
    constexpr float MAGIC = 12582912.f;
    constexpr uint32_t MAGIC_BITS = 0x4B400000u;
    constexpr float R15 = 1.f / 15.f;
    const float sq = range * R15;
    const uint32_t sbits = pack_bf16x2(fmaf(fmaf(-15.f, sq, range), R15, sq), 0.f) & 0xFFFFu;
    const float s = __uint_as_float(sbits << 16);
    float r1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(s));  // the correction makes up for its last bit
    const float2 r = make_float2(r1, r1), ns = make_float2(-s, -s), nl = make_float2(-lo, -lo);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = fadd2(make_float2(bf16lo(u[j]), bf16hi(u[j])), nl);
      float2 q = fmul2(f, r);
      q = ffma2(ffma2(q, ns, f), r, q);
      const float2 t = fadd2(q, make_float2(MAGIC, MAGIC));
      const int a = nibble_of(V, 2 * j), b = nibble_of(V, 2 * j + 1);
      n[a / 8] += __float_as_uint(t.x) << (4 * (a % 8));
      n[b / 8] += __float_as_uint(t.y) << (4 * (b % 8));
    }
    uint32_t magic = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) magic += MAGIC_BITS << (4 * j);
    n[0] -= magic;
    n[1] -= magic;
    return sbits | (m & 0xFFFF0000u);
  }
  const uint4 r = quantise_rest<V>(make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7]), lo, hi);
  n[0] = r.x;
  n[1] = r.y;
  return r.z | (m & r.w);
}

// A thread's 16 channels (piece i of the row) inside a record.  K codes: two words, bytes k_at and k_at + D/8 of the
// token's.  V codes: byte v_at + 64 g holds channels g (low) and g + 8 (high).
template <int D>
__device__ __forceinline__ int k_at(int t, int i) {
  return Rec4<D>::K + t * (D / 2) + (i & 1) * (D / 4) + (i >> 1) * 4;
}
template <int D>
__device__ __forceinline__ int v_at(int t, int i) {
  return Rec4<D>::V + (i >> 2) * 512 + ((t & 7) >> 1) * 16 + (i & 3) * 4 + ((t & 1) << 1) + (t >> 3);
}
template <int D>
__device__ __forceinline__ int word_at(bool v, int t, int i) {
  return (v ? Rec4<D>::VW : Rec4<D>::KW) + (t * Rec4<D>::NG + (i >> 2)) * 4;
}

// Writes a thread's 16 channels of token t; reads them back as codes.
template <int D, bool V>
__device__ __forceinline__ void put16(uint8_t *rec, int t, int i, const uint32_t (&n)[2], uint32_t word) {
  if constexpr (V) {
    uint8_t *p = rec + v_at<D>(t, i);
#pragma unroll
    for (int g = 0; g < 8; ++g) p[64 * g] = static_cast<uint8_t>(n[g / 4] >> (8 * (g % 4)));
  } else {
    uint8_t *p = rec + k_at<D>(t, i);
    *reinterpret_cast<uint32_t *>(p) = n[0];
    *reinterpret_cast<uint32_t *>(p + D / 8) = n[1];
  }
  if ((i & 3) == 0) *reinterpret_cast<uint32_t *>(rec + word_at<D>(V, t, i)) = word;
}
template <int D, bool V>
__device__ __forceinline__ uint32_t get16(const uint8_t *rec, int t, int i, uint32_t (&n)[2]) {
  if constexpr (V) {
    const uint8_t *p = rec + v_at<D>(t, i);
    uint32_t w[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) w[g] = p[64 * g];
#pragma unroll
    for (int k = 0; k < 2; ++k) n[k] = w[4 * k] | (w[4 * k + 1] << 8) | (w[4 * k + 2] << 16) | (w[4 * k + 3] << 24);
  } else {
    const uint8_t *p = rec + k_at<D>(t, i);
    n[0] = *reinterpret_cast<const uint32_t *>(p);
    n[1] = *reinterpret_cast<const uint32_t *>(p + D / 8);
  }
  return *reinterpret_cast<const uint32_t *>(rec + word_at<D>(V, t, i));
}

// Codes to bf16.  A code's byte becomes the low byte of 2^23 (code + 2^23, exactly).
template <bool V>
__device__ __forceinline__ void expand16(const uint32_t (&n)[2], uint32_t word, uint32_t (&o)[8]) {
  const uint32_t even[2] = {n[0] & 0x0F0F0F0Fu, n[1] & 0x0F0F0F0Fu}, odd[2] = {(n[0] >> 4) & 0x0F0F0F0Fu, (n[1] >> 4) & 0x0F0F0F0Fu};
  const float2 s = make_float2(bf16lo(word), bf16lo(word)), m = make_float2(bf16hi(word), bf16hi(word));
  auto code = [&](int ch) {
    const int a = nibble_of(V, ch);
    return __uint_as_float(__byte_perm((a & 1) ? odd[a / 8] : even[a / 8], 0x4B000000u, 0x7650 + (a % 8) / 2));
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = fadd2(make_float2(code(2 * j), code(2 * j + 1)), make_float2(-8388608.f, -8388608.f));
    const float2 x = ffma2(f, s, m);
    o[j] = pack_bf16x2(x.x, x.y);
  }
}

// The slot of token m; negative: padding (the token is left out).  A slot past the pool is never
// used as an address: it is reported and left out.
__device__ __forceinline__ int64_t slot_of(const Rows4 &a, int64_t m, bool report) {
  const int64_t s = a.slots[m];
  if (s >= a.n_slots) {
    if (report) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
    return -1;
  }
  return s;
}

// Few tokens of each sequence (N < 16, decoding steps): one row (token, head) per D / 16 threads, K and V
// by blockIdx.y, straight between the rows and the cache's bytes.
template <int D, bool LOAD, bool V>
__device__ __forceinline__ void row4(const Rows4 &a) {
  constexpr int TR = D / 16;
  const int i = threadIdx.x % TR;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / TR;
  const int64_t m = row / a.H;
  const int h = static_cast<int>(row % a.H);
  const bool in = m < static_cast<int64_t>(a.B) * a.N;
  const int64_t slot = in ? slot_of(a, m, i == 0 && h == 0 && !V) : -1;
  const int b = in ? static_cast<int>(m / a.N) : 0, n = in ? static_cast<int>(m % a.N) : 0;
  const int64_t at = b * a.sb[V] + h * a.sh[V] + n * a.sn[V] + 16 * i;
  const bool live = slot >= 0;
  uint8_t *rec = record_of(a, live ? slot : 0, h, Rec4<D>::BYTES);
  const int t = static_cast<int>(slot & 15);
  uint32_t u[8], c[2];
#pragma unroll
  for (int j = 0; j < 8; ++j) u[j] = 0u;
  if (LOAD) {
    if (live) {
      const uint32_t word = get16<D, V>(rec, t, i, c);
      expand16<V>(c, word, u);
    }
    if (live || (in && a.zero)) store16(a.y[V] + at, a.wide, u);
  } else {
    if (live) load16(a.x[V] + at, a.wide, u);
    const uint32_t word = quantise16<V>(u, c);
    if (live) put16<D, V>(rec, t, i, c, word);
  }
}
template <int D, bool LOAD>
__global__ void __launch_bounds__(256) rows4_kernel(const Rows4 a) {
  let_dependents_start();
  wait_for_earlier();
  if (blockIdx.y == 0)
    row4<D, LOAD, false>(a);
  else
    row4<D, LOAD, true>(a);
}

// Longer rows: D / 4 threads take the tokens that fall on one record of one head, K or V (the parity of blockIdx.x),
// with nothing between the threads but the groups' shuffles.  A thread holds 16 channels (piece i) of the four tokens
// 2j, 2j + 1, 2j + 8, 2j + 9, whose V codes lie in the same 32-bit words.  A token's place among the 16 follows the
// slots (the last one's place in its record lines the chunks up).  A record whose 16 slots run on is moved in
// words; else (a sequence's ends, slots that do not run on) the V codes go byte by byte.
// Measured, 4 x 8192 tokens of 8 heads, d = 128, K and V stored and read back: 59 us for 344 MB, 86% of the
// measured copy rate (cold: store 33 us at 65% of its issue slots, load 29, bound by the latency of last slot, slots,
// record).  K and V in the same threads: 104 registers, store 36 us; several heads one after another in a
// thread: the same; 8 channels a thread with the record put together in shared memory: 43 and 38.
template <int D, bool LOAD, bool V>
__device__ __forceinline__ void record4(const Rows4 &a) {
  using R = Rec4<D>;
  constexpr int TR = D / 16, UNIT = D / 4;  // threads of a row, of a record
  const int lane = threadIdx.x & 31, i = lane % TR, j = (lane / TR) & 3, b = blockIdx.z;
  const int h = static_cast<int>(blockIdx.y * blockDim.x + threadIdx.x) / UNIT;
  const int64_t *slots = a.slots + static_cast<int64_t>(b) * a.N;
  const int64_t last = slots[a.N - 1];
  const int shift = last < 0 ? 0 : static_cast<int>((last - (a.N - 1)) & 15);
  const int n0 = static_cast<int>(blockIdx.x >> 1) * C4_TOKENS - shift;
  auto place = [&](int k) { return 2 * j + (k & 1) + 8 * (k >> 1); };
  bool in[4];
  int64_t slot[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int n = n0 + place(k);
    in[k] = h < a.H && n >= 0 && n < a.N;
    slot[k] = in[k] ? slot_of(a, static_cast<int64_t>(b) * a.N + n, i == 0 && h == 0 && !V) : -1;
  }
  const int64_t hoff = b * a.sb[V] + min(h, a.H - 1) * a.sh[V] + 16 * i;
  uint32_t x[4][8], c[4][2], word[4];
  if constexpr (!LOAD) {  // every row of the tensors may be read: places in front, behind and left out give codes that go nowhere
#pragma unroll
    for (int k = 0; k < 4; ++k) load16(a.x[V] + hoff + min(max(n0 + place(k), 0), a.N - 1) * a.sn[V], a.wide, x[k]);
  }
  const int64_t first = __shfl_sync(0xffffffffu, slot[0], lane & ~(UNIT - 1));
  bool run = first >= 0 && (first & 15) == 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) run = run && slot[k] == first + place(k);
  const uint32_t unit = UNIT == 32 ? 0xffffffffu : 0xffffu << (lane & 16);
  const bool whole = (__ballot_sync(0xffffffffu, run) & unit) == unit;
  uint8_t *mem = record_of(a, whole ? first : 0, h, R::BYTES);
  // V codes of a whole record: bytes 0 - 3 of word g are tokens 2j, 2j + 8, 2j + 1, 2j + 9
  uint8_t *vp = mem + v_at<D>(2 * j, i);
  constexpr int ORDER[4] = {0, 2, 1, 3};
  if constexpr (LOAD) {
    if (whole) {
      if constexpr (V) {
        uint32_t w[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) w[g] = *reinterpret_cast<const uint32_t *>(vp + 64 * g);
#pragma unroll
        for (int k = 0; k < 4; ++k) word[k] = *reinterpret_cast<const uint32_t *>(mem + word_at<D>(true, place(k), i));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t z[4];
          transpose_bytes(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3], z);
#pragma unroll
          for (int k = 0; k < 4; ++k) c[ORDER[k]][q] = z[k];
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) word[k] = get16<D, false>(mem, place(k), i, c[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k][0] = c[k][1] = word[k] = 0u;  // left out: zeros
        if (slot[k] >= 0) word[k] = get16<D, V>(record_of(a, slot[k], h, R::BYTES), static_cast<int>(slot[k] & 15), i, c[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      expand16<V>(c[k], word[k], x[k]);
      if (slot[k] >= 0 || (in[k] && a.zero)) store16(a.y[V] + hoff + (n0 + place(k)) * a.sn[V], a.wide, x[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) word[k] = quantise16<V>(x[k], c[k]);
    if (whole) {
      if constexpr (V) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t z[4];
          transpose_bytes(c[ORDER[0]][q], c[ORDER[1]][q], c[ORDER[2]][q], c[ORDER[3]][q], z);
#pragma unroll
          for (int g = 0; g < 4; ++g) *reinterpret_cast<uint32_t *>(vp + 64 * (4 * q + g)) = z[g];
        }
        if ((i & 3) == 0)
#pragma unroll
          for (int k = 0; k < 4; ++k) *reinterpret_cast<uint32_t *>(mem + word_at<D>(true, place(k), i)) = word[k];
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) put16<D, false>(mem, place(k), i, c[k], word[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (slot[k] >= 0) put16<D, V>(record_of(a, slot[k], h, R::BYTES), static_cast<int>(slot[k] & 15), i, c[k], word[k]);
    }
  }
}
template <int D, bool LOAD>
__global__ void __launch_bounds__(128) records4_kernel(const Rows4 a) {
  let_dependents_start();
  wait_for_earlier();
  if (blockIdx.x & 1)
    record4<D, LOAD, true>(a);
  else
    record4<D, LOAD, false>(a);
}

template <int D, bool LOAD>
cudaError_t launch_rows4(const Rows4 &a, cudaStream_t s) {
  if (a.N >= C4_TOKENS) {
    constexpr int HW = 128 / D;  // heads of a warp
    const int warps = (a.H + HW - 1) / HW < 4 ? (a.H + HW - 1) / HW : 4;
    const dim3 grid(static_cast<unsigned>(2 * (a.N / C4_TOKENS + 2)), static_cast<unsigned>((a.H + warps * HW - 1) / (warps * HW)),
                    static_cast<unsigned>(a.B));
    return launch_dependent(records4_kernel<D, LOAD>, grid, static_cast<unsigned>(warps * 32), 0, s, a);
  }
  const int64_t rows = static_cast<int64_t>(a.B) * a.N * a.H, per = 256 / (D / 16);
  return launch_dependent(rows4_kernel<D, LOAD>, dim3(static_cast<unsigned>((rows + per - 1) / per), 2), 256, 0, s, a);
}

}  // namespace

// Pool rules: page sizes 16, 32, 64, 128 or 256, d 64 or 128, 16-byte aligned.
int check_cache4(const sparge_cache4 *c, Cache4 *out) {
  if (!c) return fail(SPARGE_ERR_INVALID_ARG, "cache is NULL");
  if (c->d != 64 && c->d != 128) return fail(SPARGE_ERR_UNSUPPORTED, "cache: head dim %d not in {64,128}", c->d);
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return fail(SPARGE_ERR_UNSUPPORTED, "cache: page_size %d not in {16,32,64,128,256}", c->page_size);
  if (c->n_pages < 0 || c->H <= 0) return fail(SPARGE_ERR_INVALID_ARG, "cache: bad shape n_pages=%lld H=%d", (long long)c->n_pages, c->H);
  if (c->n_pages > INT32_MAX || c->H > 65535) return fail(SPARGE_ERR_UNSUPPORTED, "cache: too large");
  if (!c->data && c->n_pages) return fail(SPARGE_ERR_INVALID_ARG, "cache->data is NULL");
  if (reinterpret_cast<uintptr_t>(c->data) & 15u) return fail(SPARGE_ERR_INVALID_ARG, "cache->data not 16-byte aligned");
  out->data = static_cast<uint8_t *>(c->data);
  out->n_pages = c->n_pages;
  out->page_size = c->page_size;
  out->page_shift = 0;
  while ((1 << out->page_shift) < c->page_size) ++out->page_shift;
  out->H = c->H;
  out->d = c->d;
  return SPARGE_OK;
}

namespace {

int rows4(const sparge_tensor *k, const sparge_tensor *v, const int64_t *slots, const sparge_cache4 *cache, bool load,
          int zero, sparge_stream_t stream) {
  clear_error();
  View x[2];
  Cache4 c;
  int rc;
  if ((rc = check_tensor(k, "k", &x[0])) || (rc = check_tensor(v, "v", &x[1])) || (rc = check_cache4(cache, &c))) return rc;
  if (x[0].B != x[1].B || x[0].H != x[1].H || x[0].N != x[1].N || x[0].d != x[1].d)
    return fail(SPARGE_ERR_INVALID_ARG, "k and v have different shapes");
  if (x[0].H != c.H || x[0].d != c.d) return fail(SPARGE_ERR_INVALID_ARG, "k and v disagree with the cache in H or d");
  if (x[0].B * x[0].N == 0) return SPARGE_OK;
  if (!slots) return fail(SPARGE_ERR_INVALID_ARG, "slots is NULL");
  Rows4 a;
  for (int s = 0; s < 2; ++s) {
    a.x[s] = static_cast<const __nv_bfloat16 *>(x[s].data);
    a.y[s] = static_cast<__nv_bfloat16 *>(const_cast<void *>(x[s].data));
    a.sb[s] = x[s].sb; a.sh[s] = x[s].sh; a.sn[s] = x[s].sn;
  }
  a.slots = slots;
  a.pool = c.data;
  a.n_slots = c.n_pages * c.page_size;
  a.page_shift = c.page_shift;
  a.H = c.H; a.N = static_cast<int>(x[0].N); a.B = static_cast<int>(x[0].B);
  a.recs = c.page_size / C4_TOKENS;
  a.status = status_ptr();
  a.zero = zero;
  a.wide = 1;  // 32-byte pieces: base and strides allow it
  for (int t = 0; t < 2; ++t)
    if ((reinterpret_cast<uintptr_t>(x[t].data) & 31u) || ((x[t].sb | x[t].sh | x[t].sn) & 15)) a.wide = 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c.d == 128)
    e = load ? launch_rows4<128, true>(a, s) : launch_rows4<128, false>(a, s);
  else
    e = load ? launch_rows4<64, true>(a, s) : launch_rows4<64, false>(a, s);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, load ? "cache load launch" : "cache store launch");
}

// --------------------------------------------------------------------------------------------
// Tables.  Bound by latency: 256 decoding requests take 2.7 us, 64 chunks of 4096 tokens (3.2 MB written) 4.7.
// One launch: every CTA sums the pages that the requests before its own need, so no
// pass over the requests precedes it (a few thousand lengths come from L2 faster than a second
// launch starts), then writes its requests' new table entries, slots and positions.  Nothing is
// read that another CTA writes: a slot on a new page takes it from the free list itself.
// --------------------------------------------------------------------------------------------
struct TablesArgs {
  const int32_t *lens, *new_lens, *free_pages;
  int32_t *table, *positions, *kv_lens, *used;
  int64_t *slots;
  int64_t stride;
  int R, N, width, n_free, shift, chunk;  // chunk: requests of a CTA
  int *status;
};

constexpr int TB_THREADS = 256;
constexpr int TB_CHUNK = 512;  // most requests of a CTA

struct Request {
  int64_t len, add;
  int have, need;  // pages held before, pages taken now
  bool bad;
};

__device__ __forceinline__ Request request_of(const TablesArgs &a, int r) {
  Request q;
  const int len = a.lens[r], add = a.new_lens[r];
  q.bad = len < 0 || add < 0 || add > a.N || static_cast<int64_t>(len) + add > INT32_MAX;
  q.len = q.bad ? 0 : len;
  q.add = q.bad ? 0 : add;
  const int64_t p = (int64_t(1) << a.shift) - 1;
  q.have = static_cast<int>((q.len + p) >> a.shift);
  q.need = static_cast<int>((q.len + q.add + p) >> a.shift) - q.have;
  return q;
}

__global__ void __launch_bounds__(TB_THREADS) cache_tables_kernel(const TablesArgs a) {
  __shared__ int64_t part[TB_THREADS / 32];
  __shared__ int64_t first[TB_CHUNK + 1];
  const int r0 = blockIdx.x * a.chunk, r1 = min(a.R, r0 + a.chunk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  let_dependents_start();
  wait_for_earlier();
  int64_t sum = 0;
  for (int r = threadIdx.x; r < r0; r += TB_THREADS) sum += request_of(a, r).need;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the CTA's own requests
    int64_t base = 0;
    for (int u = 0; u < TB_THREADS / 32; ++u) base += part[u];
    for (int r = r0; r < r1; r += 32) {
      const int64_t need = r + lane < r1 ? request_of(a, r + lane).need : 0;
      int64_t inc = need;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
      }
      if (r + lane < r1) first[r + lane - r0] = base + inc - need;
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0 && blockIdx.y == 0 && r1 == a.R && a.used) {
      *a.used = static_cast<int>(base < INT_MAX ? base : INT_MAX);
    }
  }
  __syncthreads();
  // new token places n of requests r0..r1, this CTA's share of the N
  const int per = (a.N + static_cast<int>(gridDim.y) - 1) / static_cast<int>(gridDim.y);
  const int n0 = min(a.N, static_cast<int>(blockIdx.y) * per), cnt = min(per, a.N - n0);
  const int64_t mask = (int64_t(1) << a.shift) - 1;
  auto place = [&](int k, const Request &q, int n) {  // place n of request r0 + k
    const int r = r0 + k;
    int64_t slot = -1;
    int32_t where = -1;
    if (n >= a.N - q.add) {
      const int64_t pos = q.len + n - (a.N - q.add), col = pos >> a.shift;
      where = static_cast<int32_t>(pos);
      int64_t page = -1;
      if (col < a.width) {
        if (col < q.have) page = a.table[r * a.stride + col];
        else if (first[k] + col - q.have < a.n_free) page = a.free_pages[first[k] + col - q.have];
      }
      if (page >= 0) slot = (page << a.shift) + (pos & mask);
    }
    if (a.slots) a.slots[static_cast<int64_t>(r) * a.N + n] = slot;
    if (a.positions) a.positions[static_cast<int64_t>(r) * a.N + n] = where;
  };
  if (cnt >= TB_THREADS) {  // long chunks: a request after the other
    for (int k = 0; k < r1 - r0; ++k) {
      const Request q = request_of(a, r0 + k);
      for (int n = threadIdx.x; n < cnt; n += TB_THREADS) place(k, q, n0 + n);
    }
  } else {                  // decoding steps: all requests' places in one line (at most TB_CHUNK TB_THREADS)
    for (int e = threadIdx.x; e < (r1 - r0) * cnt; e += TB_THREADS) {
      const int k = e / cnt;
      place(k, request_of(a, r0 + k), n0 + e - k * cnt);
    }
  }
  if (blockIdx.y != 0) return;
  for (int k = warp; k < r1 - r0; k += TB_THREADS / 32) {
    const int r = r0 + k;
    const Request q = request_of(a, r);
    if (lane == 0) {
      if (a.kv_lens) a.kv_lens[r] = static_cast<int32_t>(q.len + q.add);
      if (q.bad || q.have + q.need > a.width) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
    }
    for (int j = lane; j < q.need && q.have + j < a.width; j += 32)
      a.table[r * a.stride + q.have + j] = first[k] + j < a.n_free ? a.free_pages[first[k] + j] : -1;
  }
}

}  // namespace
}  // namespace sparge

using namespace sparge;

extern "C" {

size_t sparge_cache4_bytes(int64_t n_pages, int page_size, int H, int d) {
  if (n_pages < 0 || n_pages > INT32_MAX || H <= 0 || H > 65535 || (d != 64 && d != 128) || page_size < 16 ||
      page_size > 256 || (page_size & (page_size - 1)))
    return 0;
  return static_cast<size_t>(n_pages) * H * (page_size / C4_TOKENS) * (18 * static_cast<size_t>(d));
}

int sparge_cache4_store(const sparge_tensor *k, const sparge_tensor *v, const int64_t *slots, const sparge_cache4 *cache,
                        sparge_stream_t stream) {
  return rows4(k, v, slots, cache, false, 0, stream);
}

int sparge_cache4_load(const sparge_cache4 *cache, const int64_t *slots, int zero_left_out, sparge_tensor *k,
                       sparge_tensor *v, sparge_stream_t stream) {
  return rows4(k, v, slots, cache, true, zero_left_out ? 1 : 0, stream);
}

int sparge_cache_tables(const int32_t *lens, const int32_t *new_lens, int64_t R, int64_t N, int page_size,
                        const int32_t *free_pages, int64_t n_free, int32_t *table, int64_t width, int64_t table_stride,
                        int64_t *slots, int32_t *positions, int32_t *kv_lens, int32_t *used, sparge_stream_t stream) {
  clear_error();
  if (R < 0 || N < 0 || width < 0 || n_free < 0 || table_stride < width)
    return fail(SPARGE_ERR_INVALID_ARG, "bad shape R=%lld N=%lld width=%lld table_stride=%lld n_free=%lld", (long long)R,
                (long long)N, (long long)width, (long long)table_stride, (long long)n_free);
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(SPARGE_ERR_UNSUPPORTED, "page_size %d not in {16,32,64,128,256}", page_size);
  if (R > 65535 || N > (int64_t(1) << 30) || width > INT32_MAX || n_free > INT32_MAX)
    return fail(SPARGE_ERR_UNSUPPORTED, "shape too large");
  if (R > 0 && (!lens || !new_lens)) return fail(SPARGE_ERR_INVALID_ARG, "lens or new_lens is NULL");
  if (R > 0 && kv_lens && (kv_lens == lens || kv_lens == new_lens))
    return fail(SPARGE_ERR_INVALID_ARG, "kv_lens must not be lens or new_lens (every CTA reads them all)");
  if (R > 0 && width > 0 && !table) return fail(SPARGE_ERR_INVALID_ARG, "table is NULL");
  if (n_free > 0 && !free_pages) return fail(SPARGE_ERR_INVALID_ARG, "free_pages is NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  TablesArgs a;
  a.lens = lens; a.new_lens = new_lens; a.free_pages = free_pages;
  a.table = table; a.positions = positions; a.kv_lens = kv_lens; a.used = used;
  a.slots = slots;
  a.stride = table_stride;
  a.R = static_cast<int>(R); a.N = static_cast<int>(N); a.width = static_cast<int>(width); a.n_free = static_cast<int>(n_free);
  a.shift = 0;
  while ((1 << a.shift) < page_size) ++a.shift;
  a.status = status_ptr();
  // requests of a CTA: one until the CTAs outnumber two for each of the 152 SMs
  int64_t chunk = (R + 303) / 304;
  if (chunk < 1) chunk = 1;
  a.chunk = static_cast<int>(chunk);
  const int64_t gx = R > 0 ? (R + chunk - 1) / chunk : 1;
  int64_t gy = chunk * N / (4 * TB_THREADS);  // about 4 places per thread
  const int64_t most = 4 * 152 / gx;
  gy = gy > most ? most : gy;
  gy = gy < 1 ? 1 : gy;
  const cudaError_t e = launch_dependent(cache_tables_kernel, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)),
                                         TB_THREADS, 0, s, a);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "cache tables launch");
}

}  // extern "C"
