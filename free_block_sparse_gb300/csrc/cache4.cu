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
  int per;                        // heads of a CTA
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

// Codes of a thread's 8 channels (nibble j: channel j) and its group's word; the 8 threads of a
// group are adjacent lanes.  Minimum and maximum are taken on packed bf16 pairs, NaN winning, then
// together as the maximum of (max, -min), so three shuffles serve both and one test of the two
// finds an infinity or a NaN anywhere in the group.
__device__ __forceinline__ uint32_t quantise8(uint4 v, uint32_t &word) {
  uint32_t lo2 = min2_nan(min2_nan(v.x, v.y), min2_nan(v.z, v.w));
  uint32_t hi2 = max2_nan(max2_nan(v.x, v.y), max2_nan(v.z, v.w));
  lo2 = min2_nan(lo2, lo2 >> 16);
  hi2 = max2_nan(hi2, hi2 >> 16);
  uint32_t m = __byte_perm(hi2, lo2, 0x5410) ^ 0x80000000u;  // max, -min
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) m = max2_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
  m ^= 0x80000000u;
  const float lo = bf16hi(m), hi = bf16lo(m);
  const float range = hi - lo;  // an infinity or a NaN if there is one in the group
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t n = 0u;
  if (range >= 1e-28f && range < 1e38f) {
    // A quotient from the reciprocal and one correction is the correctly rounded one, or where the quotient
    // is representable (a tie of codes is) exactly it.  scale = range / 15 to bf16; adding 1.5 * 2^23 to (x - lo) / scale rounds it to even and leaves it in the
    // sum's low bits (at most 15 (1 + 2^-8): no code passes 15).
    constexpr float MAGIC = 12582912.f;
    constexpr uint32_t MAGIC_BITS = 0x4B400000u;
    constexpr float R15 = 1.f / 15.f;
    const float sq = range * R15;
    const uint32_t sbits = pack_bf16x2(fmaf(fmaf(-15.f, sq, range), R15, sq), 0.f) & 0xFFFFu;
    const float s = __uint_as_float(sbits << 16);
    float r1;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(s));  // the correction makes up for its last bit
    word = sbits | (m & 0xFFFF0000u);
    const float2 r = make_float2(r1, r1), ns = make_float2(-s, -s), nl = make_float2(-lo, -lo);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = fadd2(make_float2(bf16lo(u[j]), bf16hi(u[j])), nl);
      float2 q = fmul2(f, r);
      q = ffma2(ffma2(q, ns, f), r, q);
      const float2 t = fadd2(q, make_float2(MAGIC, MAGIC));
      n += (__float_as_uint(t.x) << (8 * j)) + (__float_as_uint(t.y) << (8 * j + 4));
    }
    uint32_t magic = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) magic += MAGIC_BITS << (4 * j);
    return n - magic;
  }
  if (!(fabsf(lo) <= 3.4028235e38f && fabsf(hi) <= 3.4028235e38f)) {
    word = 0x7FC07FC0u;
    return 0u;
  }
  // a difference beyond fp32 (bf16 values near 3e38 of both signs) is held at the largest fp32
  const uint32_t sbits = pack_bf16x2(__fdiv_rn(fminf(range, 3.4028235e38f), 15.f), 0.f) & 0xFFFFu;
  const float s = __uint_as_float(sbits << 16);
  word = sbits | (m & 0xFFFF0000u);
  if (!(s > 0.f)) return n;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float f = ((j & 1) ? bf16hi(u[j / 2]) : bf16lo(u[j / 2])) - lo;
    n |= static_cast<uint32_t>(min(max(__float2int_rn(fminf(__fdiv_rn(f, s), 15.f)), 0), 15)) << (4 * j);
  }
  return n;
}

// Byte of V codes that holds channels 16 (i / 2) + g (low) and + 8 (high) of token t, i = channel / 8.
__device__ __forceinline__ int v_byte(int t, int i, int g) {
  const int u = i >> 1;
  return (u >> 2) * 512 + (4 * g + ((t & 7) >> 1)) * 16 + (u & 3) * 4 + ((t & 1) << 1) + (t >> 3);
}

// Writes a thread's 8 channels (piece i of token t's row) of K or V into a record, in global or
// shared memory.  Called by all threads of a row together (V bytes join two threads' nibbles).
template <int D>
__device__ __forceinline__ void put8(uint8_t *rec, bool v, int t, int i, uint32_t n, uint32_t word, bool live) {
  using R = Rec4<D>;
  const uint32_t other = __shfl_xor_sync(0xffffffffu, n, 1);
  if (!live) return;
  if (!v) {
    *reinterpret_cast<uint32_t *>(rec + R::K + t * (D / 2) + (i & 3) * (D / 8) + (i >> 2) * 4) = n;
  } else {
    // this thread's four bytes, rows g0 .. g0 + 3: the even piece's code below the odd piece's.  The four
    // codes' bytes side by side, then the middle nibbles of each half exchanged
    const int g0 = (i & 1) ? 4 : 0;
    uint32_t z = __byte_perm(n, other, (i & 1) ? 0x3726 : 0x5140);
    const uint32_t x = (z ^ (z >> 4)) & 0x00F000F0u;
    z ^= x ^ (x << 4);
    uint8_t *p = rec + R::V + v_byte(t, i, g0);
#pragma unroll
    for (int g = 0; g < 4; ++g) p[64 * g] = static_cast<uint8_t>(z >> (8 * g));
  }
  if ((i & 7) == 0) *reinterpret_cast<uint32_t *>(rec + (v ? R::VW : R::KW) + (t * R::NG + (i >> 3)) * 4) = word;
}

// A thread's 8 channels back from a record.  A code's byte becomes the low byte of 2^23 (code + 2^23, exactly).
template <int D>
__device__ __forceinline__ uint4 get8(const uint8_t *rec, bool v, int t, int i) {
  using R = Rec4<D>;
  uint32_t a, b;      // codes, a byte each: channels 0, 2, 4, 6 and 1, 3, 5, 7 (K), 0 - 3 and 4 - 7 (V)
  if (!v) {
    const uint32_t n = *reinterpret_cast<const uint32_t *>(rec + R::K + t * (D / 2) + (i & 3) * (D / 8) + (i >> 2) * 4);
    a = n & 0x0F0F0F0Fu;
    b = (n >> 4) & 0x0F0F0F0Fu;
  } else {
    const uint8_t *p = rec + R::V + v_byte(t, i, 0);
    uint32_t w[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) w[g] = p[64 * g];
    a = w[0] | (w[1] << 8) | (w[2] << 16) | (w[3] << 24);
    b = w[4] | (w[5] << 8) | (w[6] << 16) | (w[7] << 24);
    a = (a >> ((i & 1) * 4)) & 0x0F0F0F0Fu;
    b = (b >> ((i & 1) * 4)) & 0x0F0F0F0Fu;
  }
  const uint32_t word = *reinterpret_cast<const uint32_t *>(rec + (v ? R::VW : R::KW) + (t * R::NG + (i >> 3)) * 4);
  const float2 s = make_float2(bf16lo(word), bf16lo(word)), m = make_float2(bf16hi(word), bf16hi(word));
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t x = v ? (j < 2 ? a : b) : a, y = v ? (j < 2 ? a : b) : b;
    const int bx = v ? 2 * (j & 1) : j, by = v ? 2 * (j & 1) + 1 : j;
    float2 f = make_float2(__uint_as_float(__byte_perm(x, 0x4B000000u, 0x7650 + bx) ),
                           __uint_as_float(__byte_perm(y, 0x4B000000u, 0x7650 + by)));
    f = ffma2(fadd2(f, make_float2(-8388608.f, -8388608.f)), s, m);
    o[j] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The slot of token m; negative: padding (the token is left out).  A slot past the pool is never
// used as an address: it is reported and left out.
__device__ __forceinline__ int64_t slot_of(const Rows4 &a, int64_t m, bool report) {
  const int64_t s = __ldg(a.slots + m);
  if (s >= a.n_slots) {
    if (report) record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
    return -1;
  }
  return s;
}

// Few tokens of each sequence (N < 16, decoding steps): one row (token, head) per D / 8 threads, K and V
// by blockIdx.y, straight between the rows and the cache's bytes.
template <int D, bool LOAD>
__global__ void __launch_bounds__(256) rows4_kernel(const Rows4 a) {
  constexpr int TR = D / 8;
  let_dependents_start();
  wait_for_earlier();
  const int side = blockIdx.y, i = threadIdx.x % TR;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / TR;
  const int64_t m = row / a.H;
  const int h = static_cast<int>(row % a.H);
  const bool in = m < static_cast<int64_t>(a.B) * a.N;
  const int64_t slot = in ? slot_of(a, m, i == 0 && h == 0 && side == 0) : -1;
  const int b = in ? static_cast<int>(m / a.N) : 0, n = in ? static_cast<int>(m % a.N) : 0;
  const int64_t at = b * a.sb[side] + h * a.sh[side] + n * a.sn[side] + 8 * i;
  const bool live = slot >= 0;
  uint8_t *rec = record_of(a, live ? slot : 0, h, Rec4<D>::BYTES);
  const int t = static_cast<int>(slot & 15);
  if (LOAD) {
    if (live) *reinterpret_cast<uint4 *>(a.y[side] + at) = get8<D>(rec, side != 0, t, i);
    else if (in && a.zero) *reinterpret_cast<uint4 *>(a.y[side] + at) = make_uint4(0u, 0u, 0u, 0u);
  } else {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (live) v = ld_stream_v4(a.x[side] + at);
    uint32_t word;
    const uint32_t c = quantise8(v, word);
    put8<D>(rec, side != 0, t, i, c, word, live);
  }
}

// Longer rows: a CTA takes the tokens that fall on one record, K and V together, for a few heads one
// after another (the slots are looked up once, and a head's rows or record come while the one before it
// is worked on).  A row's place among the 16 tokens follows the slots (the last one's place in its record lines the
// chunks up; slots that do not run on are still handled, token by token).  A whole record is put
// together or taken apart in shared memory and moved in 16-byte pieces; single tokens go straight
// to the cache's bytes.
// Measured, 4 x 8192 tokens of 8 heads, d = 128, K and V stored and read back: 69 us for 344 MB, 74% of the
// measured copy rate (cold: store 43 us, load 38): the store is bound by its arithmetic (16 instructions per value),
// the load by the latency of its two steps.
constexpr int R4_HEADS = 8;  // most heads of a CTA (8 heads: 68 us, 4: 70, 2: 79)
template <int D, bool LOAD>
__global__ void __launch_bounds__(2 * D) records4_kernel(const Rows4 a) {
  using R = Rec4<D>;
  constexpr int TR = D / 8, PIECES = (R::BYTES / 16 + 2 * D - 1) / (2 * D);
  __shared__ __align__(16) uint8_t rec[2][R::BYTES];
  __shared__ int64_t first;
  let_dependents_start();
  wait_for_earlier();
  const int t = threadIdx.x / TR, i = threadIdx.x % TR, b = blockIdx.z;
  const int h0 = blockIdx.y * a.per, h1 = min(h0 + a.per, a.H);
  const int64_t *slots = a.slots + static_cast<int64_t>(b) * a.N;
  const int64_t last = __ldg(slots + a.N - 1);
  const int shift = last < 0 ? 0 : static_cast<int>((last - (a.N - 1)) & 15);
  const int n = static_cast<int>(blockIdx.x) * C4_TOKENS - shift + t;
  const bool in = n >= 0 && n < a.N;
  const int64_t slot = in ? slot_of(a, static_cast<int64_t>(b) * a.N + n, i == 0 && h0 == 0) : -1;
  const bool live = slot >= 0;
  if (threadIdx.x == 0) first = slot;
  __syncthreads();
  const bool whole = __syncthreads_and(live && (first & 15) == 0 && slot == first + t);
  uint8_t *mem = record_of(a, live ? slot : 0, h0, R::BYTES);
  const int64_t hstep = static_cast<int64_t>(a.recs) * R::BYTES;  // the next head's record of the page
  const int at = static_cast<int>(slot & 15);
  const int64_t o0 = b * a.sb[0] + h0 * a.sh[0] + n * a.sn[0] + 8 * i, o1 = b * a.sb[1] + h0 * a.sh[1] + n * a.sn[1] + 8 * i;
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  if (LOAD) {
    __nv_bfloat16 *y0 = a.y[0] + o0, *y1 = a.y[1] + o1;
    uint4 piece[PIECES];
    auto fetch = [&](const uint8_t *from) {
#pragma unroll
      for (int e = 0; e < PIECES; ++e)
        if (whole && e * 2 * D + threadIdx.x < R::BYTES / 16) piece[e] = ld_stream_v4(from + 16 * (e * 2 * D + threadIdx.x));
    };
    fetch(mem);
    for (int h = h0; h < h1; ++h) {
      uint8_t *buf = rec[h & 1];
      if (whole) {
#pragma unroll
        for (int e = 0; e < PIECES; ++e)
          if (e * 2 * D + threadIdx.x < R::BYTES / 16) reinterpret_cast<uint4 *>(buf)[e * 2 * D + threadIdx.x] = piece[e];
        __syncthreads();
        if (h + 1 < h1) fetch(mem + hstep);
      }
      uint4 k = none, v = none;
      if (live) {
        const uint8_t *src = whole ? buf : mem;
        k = get8<D>(src, false, at, i);
        v = get8<D>(src, true, at, i);
      }
      if (live || (in && a.zero)) {
        *reinterpret_cast<uint4 *>(y0) = k;
        *reinterpret_cast<uint4 *>(y1) = v;
      }
      mem += hstep;
      y0 += a.sh[0];
      y1 += a.sh[1];
    }
  } else {
    const __nv_bfloat16 *x0 = a.x[0] + o0, *x1 = a.x[1] + o1;
    uint4 k = live ? ld_stream_v4(x0) : none, v = live ? ld_stream_v4(x1) : none;
    for (int h = h0; h < h1; ++h) {
      const uint4 k0 = k, v0 = v;
      if (live && h + 1 < h1) {
        x0 += a.sh[0];
        x1 += a.sh[1];
        k = ld_stream_v4(x0);
        v = ld_stream_v4(x1);
      }
      uint8_t *dst = whole ? rec[h & 1] : mem;
      uint32_t word;
      uint32_t c = quantise8(k0, word);
      put8<D>(dst, false, at, i, c, word, live);
      c = quantise8(v0, word);
      put8<D>(dst, true, at, i, c, word, live);
      if (whole) {
        __syncthreads();
        for (int e = threadIdx.x; e < R::BYTES / 16; e += 2 * D)
          *reinterpret_cast<uint4 *>(mem + 16 * e) = reinterpret_cast<const uint4 *>(rec[h & 1])[e];
      }
      mem += hstep;
    }
  }
}

template <int D, bool LOAD>
cudaError_t launch_rows4(Rows4 a, cudaStream_t s) {
  if (a.N >= C4_TOKENS) {
    // as many heads per CTA as leave 8 CTAs for each of the 152 SMs
    const int64_t chunks = a.N / C4_TOKENS + 2, per = chunks * a.B * a.H / (8 * 152);
    a.per = static_cast<int>(per < 1 ? 1 : (per > R4_HEADS ? R4_HEADS : per));
    if ((a.H + a.per - 1) / a.per > 65535) a.per = R4_HEADS;
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>((a.H + a.per - 1) / a.per), static_cast<unsigned>(a.B));
    return launch_dependent(records4_kernel<D, LOAD>, grid, 2 * D, 0, s, a);
  } else {
    const int64_t rows = static_cast<int64_t>(a.B) * a.N * a.H, per = 256 / (D / 8);
    return launch_dependent(rows4_kernel<D, LOAD>, dim3(static_cast<unsigned>((rows + per - 1) / per), 2), 256, 0, s, a);
  }
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
  a.per = 1;
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
  const int len = __ldg(a.lens + r), add = __ldg(a.new_lens + r);
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
        else if (first[k] + col - q.have < a.n_free) page = __ldg(a.free_pages + first[k] + col - q.have);
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
      a.table[r * a.stride + q.have + j] = first[k] + j < a.n_free ? __ldg(a.free_pages + first[k] + j) : -1;
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
