// Attention over the paged 4-bit cache (decoding steps and short chunks).
//
//   O = softmax(scale Q K^^T) V^,  K^, V^ = code * scale + minimum per token and 64 channels,
// causal with the last query on the last token of its sequence, optionally over a window and a few
// first tokens.  Each cache byte is read once per tile of 8 or 16 query rows (the Nq rows of all heads
// of a KV head), so for a decoding step memory bounds it: 18 d / 16 bytes per token and KV head.
//
// The products run on mma.sync with the codes as they lie in memory: a 4-bit code in the low bits of
// an f16 is the subnormal code * 2^-24 (bits 4-7: code * 2^-20), so two ANDs and one shift per 4
// codes make the operands - no conversion, no subtraction of a bias - and scales and minima enter in
// fp32 on the small side, where each applies to a whole 64-channel dot product.  tcgen05 would want
// the codes widened into shared memory first, 4 times their size through a port that then feeds
// the tensor core from it again; for 1 to 16 rows that traffic, not the products, would bound it.
//   S^T = K^ Q^T: A = 16 tokens x 16 channels of codes, B = Q^T (f16, each row scaled by a power of two
//         to a maximum in [2^14, 2^15); the odd channels' 1/16 of that, as their codes come 16 times as
//         large: the 8 significant bits stay whole down to 2^-27 of the maximum, in even channels to 2^-31).
//         x = k (sum_g s_g acc_g) + sum_g m_g (scale * sum of q over group g).
//   O^T = V^T P^T: A = 16 channels x 16 tokens of codes, B = P^T s (f16: 11 bits, an eighth of the
//         output's rounding: against 64 bits 1.79e-3 in place of the 1.66e-3 of an fp32 form, 64 sequences)
//         transposed in registers by movmatrix; the minima add sum P m per row.
// P lies in [0, 2^8] (the reference follows the running maximum lazily).  P s is scaled by a power of two per row and
// channel group that follows its own running maximum the same way, so the largest P s of a row stays in
// [2^3, 2^15]: what is less than 2^-17 of it loses bits in f16, what is less than 2^-28 is lost.
//
// Work: the (sequence, KV head, row tile) items' tiles in one line, cut into equal shares, one per CTA
// (2 to 4 CTAs per SM), so ragged lengths fill the part evenly; every warp sums the lengths
// itself.  A warp takes every fourth step of its CTA's share (two 16-token records)
// through a ring of its own of bulk copies, without any synchronisation among warps until an item
// ends; then the four warps' sums are merged in shared memory, and an item cut between CTAs is put
// together by a second kernel (rowsplit.cuh).
// Measured: 64 sequences of 1K to 32K tokens, 32 + 8 heads, d = 128: 206 us for 1.25 GB, 90% of the
// measured copy rate; one sequence of 4K 9.8 us, of which the chain length -> page -> record -> merge ->
// combine is nearly all; 128 x 4 queries under a window of 4096, d = 64: 58 us, 38% (16 rows of 64 channels bring two
// and a half times the arithmetic per byte: the ALU is 43% busy, the tensor pipe 28%).  One power of two per warp in place
// of one per row and group: 9.2, 206 and 57 us, but hidden and improbable tokens took bits from the others.
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/sparge.h"
#include "cache4.cuh"
#include "common.cuh"
#include "kernels.h"
#include "rowsplit.cuh"

namespace sparge {
int check_cache4(const ::sparge_cache4 *c, Cache4 *out);
namespace {

// Tiles that an item's start and end weigh in a CTA's share (128 ragged sequences of 4 queries, d = 64, under a window of
// 4096: 0 66 us, 2 58, 3 57; 64 sequences of up to 32K: 0 213, 3 206; measured before the powers of two went by row).
constexpr int CA_ITEM = 3;
// Where a row's largest P s goes when its power of two is set (to 2^(CA_ROOM - 1) .. 2^CA_ROOM), and how far it may grow before
// that moves: to 2^15, within f16.
constexpr int CA_ROOM = 4, CA_GROW = 15 - CA_ROOM;
constexpr float CA_SBOUND = 128.f;  // 2^15 / 2^CA_RESCALE

// The records a sequence's queries see: the first `ns` (tokens that stay visible), then lo..hi-1.
struct Span {
  int len, ns, lo, recs;
};

struct CacheAttnArgs : SplitArgs {
  const __nv_bfloat16 *q;
  int64_t q_sb, q_sh, q_sn;
  const uint8_t *pool;
  const int32_t *table, *lens;
  int64_t table_stride, n_pages;
  int width, rec_shift;  // records of a page: 1 << rec_shift
  int window, sinks;     // window 0: none
  float scale_log2;
  int *status;
  __device__ __forceinline__ bool empty(int b) const { return width == 0 || lens[b] <= 0; }
  __device__ __forceinline__ const int32_t *pages(int b, int) const { return table + static_cast<int64_t>(b) * table_stride; }
  __device__ __forceinline__ const __nv_bfloat16 *queries(int b, int h) const { return q + b * q_sb + h * q_sh; }
  __device__ __forceinline__ int length(int b) const {
    const int len = lens[b];
    const int64_t cap = static_cast<int64_t>(width) << (rec_shift + 4);
    return max(len > cap ? static_cast<int>(cap) : len, 0);
  }
  __device__ __forceinline__ Span span(int b) const {
    Span s;
    s.len = length(b);
    const int hi = static_cast<int>((static_cast<int64_t>(s.len) + 15) >> 4);
    s.ns = 0;
    s.lo = 0;
    if (window > 0) {
      const int64_t first = static_cast<int64_t>(s.len) - Nq - window + 1;
      s.lo = first > 0 ? static_cast<int>(first >> 4) : 0;
      s.ns = min(s.lo, static_cast<int>((static_cast<int64_t>(sinks) + 15) >> 4));
    }
    s.recs = s.ns + hi - s.lo;
    return s;
  }
};

// Every query and KV head with a page list of its own: "sequence" b is query b % queries_of of sequence b / queries_of, the
// last token of its list.  (G rows each, so the selected bytes of a KV head are read once for its heads.)  512 lists of 64 pages of
// 64 tokens, d = 128: 60 us for 302 MB, 75 % of the copy rate; 384 of 128 pages of 16, d = 64: 21 us for 57 MB, bound by starts and ends.
struct CacheListArgs : CacheAttnArgs {
  int queries_of;
  __device__ __forceinline__ const int32_t *pages(int b, int kvh) const {
    return table + (static_cast<int64_t>(b) * Hkv + kvh) * width;
  }
  __device__ __forceinline__ const __nv_bfloat16 *queries(int b, int h) const {
    return q + (b / queries_of) * q_sb + static_cast<int64_t>(b % queries_of) * q_sn + h * q_sh;
  }
  __device__ __forceinline__ __nv_bfloat16 *row(int b, int kvh, int r) const {
    return o + (b / queries_of) * o_sb + static_cast<int64_t>(b % queries_of) * o_sn + (kvh * G + r) * o_sh;
  }
};

// What stands behind a prefix that is attended elsewhere: a sequence's records from first_rec on (all of them if its queries do
// not all stand behind the prefix), as shares for another kernel to combine.  64 sequences of 64 to 2048 own tokens, 32 over 8 heads,
// d = 128: 22 to 26 us for 78 MB: an item of one head and sequence is a few steps, so starts and ends bound it.  (It starts behind the
// prefix kernel.  Beside that one's last CTAs, reading before its wait what calls in front had written, it gained 2 us; that order is not promised.)
struct CacheTailArgs : CacheAttnArgs {
  int first_rec;
  static constexpr bool PARTIAL = true;
  __device__ __forceinline__ Span span(int b) const {
    Span s;
    s.len = length(b);
    s.ns = 0;
    s.lo = (s.len - Nq) >= first_rec * 16 ? first_rec : 0;
    s.recs = static_cast<int>((static_cast<int64_t>(s.len) + 15) >> 4) - s.lo;
    return s;
  }
};

// CTAs per SM, by registers: the sums of 16 rows of 128 channels alone take 64 per thread.  (16 rows of
// d = 128, 4 queries of 128 sequences of 4100 with 4 KV heads: 2 CTAs 93 us, 3 with one record a step and spills 113; with 8, 180;
// d = 64: 3 CTAs 56 us, 2 65.)
constexpr int ca_ctas(int D, int RT) { return RT == 1 ? 4 : D == 64 ? 3 : 2; }

// Shared memory and the step of a warp: U = 2 records at a time (a CTA's tile is 4 U records, one step of each
// warp), which keeps two chains of dependent products in flight and halves the waits, votes and
// branches per record; ST steps in a warp's ring.
template <int D, int RT>
struct CaSmem {
  static constexpr int U = 2;
  static constexpr int ST = D == 64 ? 5 : 3;
  static constexpr int REC = Rec4<D>::BYTES;
  static constexpr int WRING = ST * U * REC;  // of one warp; the item's sums go there at its end
  static constexpr int OROW = D + 4;          // floats of a row of sums, padded against bank conflicts
  static_assert(8 * RT * OROW * 4 <= WRING, "a warp's sums fit its ring");
  static_assert(ST <= 6 && ST * U <= 12, "barriers and flags");
  static constexpr int OFF_ML = CA_WARPS * WRING, OFF_CTRL = OFF_ML + CA_WARPS * 8 * RT * 8;
  static constexpr int TOTAL = OFF_CTRL + 512;
};
struct CaCtrl {
  uint64_t full[CA_WARPS][6];
  int abort;
  uint8_t bad[CA_WARPS][12];  // the record's page lies outside the pool: its tokens are left out
};
static_assert(sizeof(CaCtrl) <= 512, "control block");

// The line that is cut into shares: every item counts its tiles (4 U records each) and CA_ITEM more, about
// the time that a CTA spends on an item apart from its tiles, so a CTA of many short items gets fewer tiles.
// A place in those CA_ITEM stands for no work.
template <int U>
__device__ __forceinline__ int tiles_of(const Span &sp) {
  return (sp.recs + 4 * U - 1) / (4 * U);
}
template <int U, typename Args>
__device__ __forceinline__ int64_t units_of(const Args &a, int b) {
  const int t = tiles_of<U>(a.span(b));
  return t == 0 ? 0 : static_cast<int64_t>(t + CA_ITEM) * (a.Hkv * a.ntile);
}
// x / y for non-negative x and positive y, in 32 bits where they do
__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? static_cast<uint32_t>(x) / static_cast<uint32_t>(y) : x / y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with a zero accumulator
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// scale words of tokens g (u) and g + 8 (v) of this lane, g = lane / 4
template <int NG>
__device__ __forceinline__ void words(const uint8_t *p, uint32_t (&u)[NG], uint32_t (&v)[NG]) {
  const int g = (threadIdx.x & 31) >> 2;
  if constexpr (NG == 2) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p + g * 8), b = *reinterpret_cast<const uint2 *>(p + 64 + g * 8);
    u[0] = a.x; u[1] = a.y;
    v[0] = b.x; v[1] = b.y;
  } else {
    u[0] = *reinterpret_cast<const uint32_t *>(p + g * 4);
    v[0] = *reinterpret_cast<const uint32_t *>(p + 32 + g * 4);
  }
}
// 2^e / f for a power of two f
__device__ __forceinline__ float over2(float f, int e) {
  return __uint_as_float((static_cast<uint32_t>(254 + e) << 23) - __float_as_uint(f));
}

// The power of two f on a row's P s of one channel group, set anew when y, the largest score + log2 s (a maximum over the
// warp's tokens, reduced here), is 2^CA_GROW above what it was set for, and when the exponent reference (its negative m)
// has moved, by al on what was summed (0: nothing before).  A row's f depends on the row's own P s alone: y that far above
// means a scale past CA_SBOUND, and moves of the reference are the row's own.  Returns the factor on the sums.
__device__ __forceinline__ float follow_scale(float &f, float y, float m, float al) {
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, o));
  const int e0 = CA_ROOM - exponent_of(f);
  const float top = y + m;
  if (!(top > static_cast<float>(e0 + CA_GROW)) && al == 1.f) return 1.f;
  const int e = min(max(__float2int_ru(fmaxf(top, static_cast<float>(e0) + __log2f(al))), -100), 108);
  f = pow2i(CA_ROOM - e);
  return al * pow2i(min(max(e0 - e, -126), 127));
}

template <int D, int RT, typename Args>
__global__ void __launch_bounds__(CA_WARPS * 32, ca_ctas(D, RT)) cache4_attn_kernel(const Args a) {
  using S = CaSmem<D, RT>;
  using R = Rec4<D>;
  constexpr int NG = D / 64, NW = D / 32, MT = D / 16, U = S::U, ST = S::ST;
  extern __shared__ __align__(128) uint8_t smem[];
  CaCtrl &cs = *reinterpret_cast<CaCtrl *>(smem + S::OFF_CTRL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t *ring = smem + warp * S::WRING;

  let_dependents_start();
  wait_for_earlier();

  // ---- this CTA's share [start, end) of the line of tiles, and the sequence it starts in; every warp for
  // itself, so that no barrier holds up the first loads ----
  if (lane == 0) {
    cs.abort = 0;
    for (int s = 0; s < ST; ++s) mbar_init(&cs.full[warp][s], U);
    fence_barrier_init();
  }
  __syncwarp();
  const int per = (a.B + 31) / 32, bt = min(a.B, lane * per), bu = min(a.B, bt + per);
  int64_t own = 0;
  for (int b = bt; b < bu; ++b) own += units_of<U>(a, b);
  int64_t inc = own;
  if (a.B > 1) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
  }
  const int64_t total = __shfl_sync(0xffffffffu, inc, a.B > 1 ? 31 : 0);
  // shares only for as many CTAs as there are places: between an item's first and last CTA each holds some of it
  const int64_t shares = total < gridDim.x ? total : gridDim.x;
  if (blockIdx.x >= shares) return;
  const int64_t start = divide(total * blockIdx.x, shares), end = divide(total * (blockIdx.x + 1), shares);
  int b = bt;
  int64_t off = start - (inc - own), left = end - start;
  const uint32_t here = __ballot_sync(0xffffffffu, off >= 0 && off < own);  // the lane whose sequences hold the start
  if (off >= 0 && off < own)
    for (int64_t u; off >= (u = units_of<U>(a, b)); ++b) off -= u;
  b = __shfl_sync(0xffffffffu, b, __ffs(here) - 1);
  off = __shfl_sync(0xffffffffu, off, __ffs(here) - 1);
  uint32_t used = 0;  // steps this warp has taken through its ring (stage used % ST)

  // ---- the item at the front of what is left of the share, and its first loads ----
  Span sp;
  int item, kvh, row0, tiles, tile0, nt;  // this CTA holds tiles tile0 .. tile0 + nt - 1 of the item
  int k0, kend, nstep;                    // this warp's steps; step i: records k0 + 4 U i .. + U - 1, those below kend
  auto locate = [&]() -> bool {           // false: nothing left
    while (left > 0) {
      sp = a.span(b);
      tiles = tiles_of<U>(sp);
      const int64_t in_b = tiles ? divide(off, tiles + CA_ITEM) : INT_MAX;
      if (in_b >= a.Hkv * a.ntile) {
        off -= units_of<U>(a, b);
        ++b;
        continue;
      }
      const int place = static_cast<int>(off - in_b * (tiles + CA_ITEM));
      if (place < CA_ITEM) {
        const int64_t skip = left < CA_ITEM - place ? left : CA_ITEM - place;
        off += skip;
        left -= skip;
        if (left == 0) return false;
      }
      tile0 = max(place - CA_ITEM, 0);
      nt = static_cast<int>(left < tiles - tile0 ? left : tiles - tile0);
      off += nt;
      left -= nt;
      kvh = static_cast<int>(in_b) / a.ntile;
      row0 = (static_cast<int>(in_b) - kvh * a.ntile) * 8 * RT;
      item = b * (a.Hkv * a.ntile) + static_cast<int>(in_b);
      k0 = (tile0 * 4 + warp) * U;
      kend = min(sp.recs, (tile0 + nt) * 4 * U);
      nstep = kend > k0 ? (kend - k0 + 4 * U - 1) / (4 * U) : 0;
      return true;
    }
    return false;
  };
  auto record_at = [&](int k) { return k < sp.ns ? k : sp.lo + k - sp.ns; };
  // The warp looks up the pages of 32 records at a time; the lane that holds a record's address issues
  // its copy.
  const uint8_t *src = nullptr;  // record lane % U of step sbase + lane / U (null: no such page, no such record)
  int sbase = 0;
  bool has_bad = false, had_bad = true;  // some page of the item (of the one before) was outside the pool: the flags count
  auto look_up = [&](int i) {
    sbase = i;
    const int k = k0 + 4 * U * (i + lane / U) + lane % U;
    src = nullptr;
    bool bad = false;
    if (k < kend) {
      const int r = record_at(k);
      const int page = a.pages(b, kvh)[r >> a.rec_shift];
      bad = page < 0 || page >= a.n_pages;
      if (bad)
        record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
      else
        src = a.pool + (((static_cast<int64_t>(page) * a.Hkv + kvh) << a.rec_shift) + (r & ((1 << a.rec_shift) - 1))) * S::REC;
    }
    has_bad = __any_sync(0xffffffffu, bad) || has_bad;
  };
  auto issue = [&](int i) {  // called by the whole warp for i = 0, 1, ... in order
    if (i >= sbase + 32 / U) look_up(i);
    if (lane / U == i - sbase) {
      const uint32_t st = (used + i) % ST;
      uint64_t *bar = &cs.full[warp][st];
      if (has_bad) cs.bad[warp][st * U + lane % U] = src == nullptr;
      if (src != nullptr) {
        mbar_arrive_expect_tx(bar, S::REC);
        bulk_load(ring + (st * U + lane % U) * S::REC, src, S::REC, bar);
      } else {
        mbar_arrive(bar);
      }
    }
  };
  // this lane's query row of row tile j (null: there is none) and its place among the Nq queries
  auto query_of = [&](int j, int &qi) -> const uint4 * {
    const int r = row0 + 8 * j + g;
    const int hg = a.Nq == 1 ? r : r / a.Nq;
    qi = a.Nq == 1 ? 0 : r - hg * a.Nq;
    if (r >= a.rows) {
      qi = 0;
      return nullptr;
    }
    return reinterpret_cast<const uint4 *>(a.queries(b, kvh * a.G + hg) + static_cast<int64_t>(qi) * a.q_sn);
  };
  // Q rows of the next item: carried in registers over the end of the one before where they fit (d = 64),
  // else only fetched ahead of their use
  constexpr bool CARRY = D == 64;
  uint4 qraw[RT][NW];
  auto load_q = [&](int j) {
    int qi;
    const uint4 *qrow = query_of(j, qi);
#pragma unroll
    for (int w = 0; w < NW; ++w) qraw[j][w] = qrow != nullptr ? qrow[4 * w + c] : make_uint4(0u, 0u, 0u, 0u);
  };

  // The next item's first loads (queries, page numbers) go out before the end of the one before.
  bool ending = false, first = false, last = false;
  int item_done = 0, b_done = 0, kvh_done = 0, row_done = 0;
  for (;;) {
    const bool more = locate();
    if (more) {
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        if constexpr (CARRY) {
          load_q(j);
        } else {
          int qi;
          const uint4 *qrow = query_of(j, qi);
          if (qrow != nullptr && (c & 1) == 0)
#pragma unroll
            for (int w = 0; w < NW; ++w) asm volatile("prefetch.global.L1 [%0];" ::"l"(qrow + 4 * w + c));
        }
      }
      has_bad = false;
      look_up(0);
    }
    if (ending) {
      end_item<D, RT>(a, smem, S::WRING, S::OROW, reinterpret_cast<const float2 *>(smem + S::OFF_ML), item_done, b_done,
                      kvh_done, row_done, first, last);
      if (*reinterpret_cast<volatile int *>(&cs.abort)) break;
    }
    if (!more) break;
    if (had_bad) {  // flags of an earlier item
      if (lane < 12) cs.bad[warp][lane] = 0;
      __syncwarp();
    }
    const int ahead = min(nstep, ST);
    for (int i = 0; i < ahead; ++i) issue(i);

    // ---- Q: B operands of the score product, and per query row the multiplier and the group sums ----
    uint32_t qf[RT][NW][4];
    float2 qk[RT], qz[RT][NG];  // of this lane's rows 2c, 2c + 1 of each row tile
    int pos[RT][2];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      if constexpr (!CARRY) load_q(j);
      int qi;
      query_of(j, qi);
      float x[NW][8];
      float mx = 0.f, sum[NG];
#pragma unroll
      for (int w = 0; w < NG; ++w) sum[w] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint32_t u[4] = {qraw[j][w].x, qraw[j][w].y, qraw[j][w].z, qraw[j][w].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[w][2 * k] = bf16lo(u[k]);
          x[w][2 * k + 1] = bf16hi(u[k]);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          mx = fmaxf(mx, fabsf(x[w][k]));
          sum[w / 2] += x[w][k];
        }
      }
#pragma unroll
      for (int o = 1; o <= 2; o <<= 1) {
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
        for (int w = 0; w < NG; ++w) sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], o);
      }
      // a power of two that takes the row's maximum to [2^14, 2^15)
      const int e = min(max(exponent_of(mx), -100), 116);
      const float f = pow2i(14 - e);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f16 = f * 0.0625f;  // the odd channels' codes come 16 times as large
        qf[j][w][0] = half2_of(x[w][0] * f, x[w][4] * f);
        qf[j][w][1] = half2_of(x[w][1] * f16, x[w][5] * f16);
        qf[j][w][2] = half2_of(x[w][2] * f, x[w][6] * f);
        qf[j][w][3] = half2_of(x[w][3] * f16, x[w][7] * f16);
      }
      const float mult = a.scale_log2 * pow2i(e + 10);  // 2^24 / f
      const int p = sp.len - a.Nq + qi;                   // rows past the last are computed and dropped
      const int from = 8 * c;  // the lanes of rows 2c and 2c + 1
      qk[j] = make_float2(__shfl_sync(0xffffffffu, mult, from), __shfl_sync(0xffffffffu, mult, from + 4));
      pos[j][0] = __shfl_sync(0xffffffffu, p, from);
      pos[j][1] = __shfl_sync(0xffffffffu, p, from + 4);
#pragma unroll
      for (int w = 0; w < NG; ++w)
        qz[j][w] = make_float2(__shfl_sync(0xffffffffu, sum[w], from) * a.scale_log2,
                               __shfl_sync(0xffffffffu, sum[w], from + 4) * a.scale_log2);
    }

    float acc[MT][RT][4];   // O^T: rows g (channels 16 u + g, times 2^-24 vfac) and g + 8 (times 2^-20 vfac), columns 2c, 2c + 1
    float2 zero[RT][NG];    // sum of P times the minima, and the sum of P (this lane's tokens, rows 2c and 2c + 1)
    float2 l[RT];
    float2 nref[RT], thr[RT];  // minus the exponent references, and the scores that move them
    // per row and channel group: the power of two on P s.  It follows what the row itself sees, weighed by P, so neither a
    // hidden token nor an improbable one nor the other group takes bits from the rest.
    float2 vfac[NG][RT];
    float sbound = 0.f;  // d = 64, where there is a register for it: CA_SBOUND over the largest of this lane's powers
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      nref[j] = both(0.f);
      thr[j] = both(-INFINITY);  // nothing seen yet: the first score moves it
      l[j] = both(0.f);
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        zero[j][w] = both(0.f);
        vfac[w][j] = both(1.f);
      }
    }
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[u][j][k] = 0.f;

    // One step: tokens g and g + 8 of each of its records in this lane.  EDGE: some of its tokens are
    // hidden from some row, or lie behind the sequence, or on no page.
    auto step = [&](auto edge_tag, const uint8_t *p, int k) {
      constexpr bool EDGE = decltype(edge_tag)::value;
      int tok[U];
      bool gone[U];  // EDGE: the record is not there
#pragma unroll
      for (int e = 0; e < U; ++e) {
        tok[e] = record_at(k + e) * 16;
        gone[e] = EDGE && (k + e >= kend || (has_bad && cs.bad[warp][static_cast<int>(p - ring) / S::REC + e] != 0));
      }
      // ---- scores ----
      float2 x0[U][RT], x1[U][RT];
#pragma unroll
      for (int e = 0; e < U; ++e) {
        const uint8_t *pe = p + e * S::REC;
        uint32_t ka[NW], kb[NW];
        if constexpr (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4 *>(pe + R::K + lane * 16);
          const uint4 v = *reinterpret_cast<const uint4 *>(pe + R::K + 512 + lane * 16);
          ka[0] = u.x; ka[1] = u.y; ka[2] = u.z; ka[3] = u.w;
          kb[0] = v.x; kb[1] = v.y; kb[2] = v.z; kb[3] = v.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2 *>(pe + R::K + lane * 8);
          const uint2 v = *reinterpret_cast<const uint2 *>(pe + R::K + 256 + lane * 8);
          ka[0] = u.x; ka[1] = u.y;
          kb[0] = v.x; kb[1] = v.y;
        }
        float sc[NG][RT][4];
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const uint32_t va = ka[w] >> 8, vb = kb[w] >> 8;
#pragma unroll
          for (int j = 0; j < RT; ++j) {
            if (w % 2 == 0)
              mma_f16_zero(sc[w / 2][j], ka[w] & 0x000F000Fu, kb[w] & 0x000F000Fu, ka[w] & 0x00F000F0u, kb[w] & 0x00F000F0u,
                           qf[j][w][0], qf[j][w][1]);
            else
              mma_f16(sc[w / 2][j], ka[w] & 0x000F000Fu, kb[w] & 0x000F000Fu, ka[w] & 0x00F000F0u, kb[w] & 0x00F000F0u,
                      qf[j][w][0], qf[j][w][1]);
            mma_f16(sc[w / 2][j], va & 0x000F000Fu, vb & 0x000F000Fu, va & 0x00F000F0u, vb & 0x00F000F0u, qf[j][w][2],
                    qf[j][w][3]);
          }
        }
        uint32_t u[NG], v[NG];
        words(pe + R::KW, u, v);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          float2 t0 = fmul2(both(bf16lo(u[0])), make_float2(sc[0][j][0], sc[0][j][1]));
          float2 t1 = fmul2(both(bf16lo(v[0])), make_float2(sc[0][j][2], sc[0][j][3]));
          float2 z0 = fmul2(both(bf16hi(u[0])), qz[j][0]), z1 = fmul2(both(bf16hi(v[0])), qz[j][0]);
          if constexpr (NG == 2) {
            t0 = ffma2(both(bf16lo(u[1])), make_float2(sc[1][j][0], sc[1][j][1]), t0);
            t1 = ffma2(both(bf16lo(v[1])), make_float2(sc[1][j][2], sc[1][j][3]), t1);
            z0 = ffma2(both(bf16hi(u[1])), qz[j][1], z0);
            z1 = ffma2(both(bf16hi(v[1])), qz[j][1], z1);
          }
          x0[e][j] = ffma2(t0, qk[j], z0);
          x1[e][j] = ffma2(t1, qk[j], z1);
        }
        // hidden tokens: past the row's position, or between the first tokens and the window
        if constexpr (EDGE) {
          auto hide = [&](float &x, int t, int q) {
            if (!(t <= q && (a.window == 0 || t < a.sinks || q - t < a.window)) || gone[e]) x = -INFINITY;
          };
#pragma unroll
          for (int j = 0; j < RT; ++j) {
            hide(x0[e][j].x, tok[e] + g, pos[j][0]);
            hide(x0[e][j].y, tok[e] + g, pos[j][1]);
            hide(x1[e][j].x, tok[e] + g + 8, pos[j][0]);
            hide(x1[e][j].y, tok[e] + g + 8, pos[j][1]);
          }
        }
      }
      // ---- the exponent reference and the powers of two on P s follow lazily ----
      uint32_t vu[U][NG], vv[U][NG];
#pragma unroll
      for (int e = 0; e < U; ++e) words(p + e * S::REC + R::VW, vu[e], vv[e]);
      bool move = false;
      float2 xm[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        xm[j] = make_float2(fmaxf(x0[0][j].x, x1[0][j].x), fmaxf(x0[0][j].y, x1[0][j].y));
        if constexpr (U == 2) {
          xm[j].x = fmax3(xm[j].x, x0[U - 1][j].x, x1[U - 1][j].x);
          xm[j].y = fmax3(xm[j].y, x0[U - 1][j].y, x1[U - 1][j].y);
        }
        move = move || xm[j].x > thr[j].x || xm[j].y > thr[j].y;
      }
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        float smax = fmaxf(fabsf(bf16lo(vu[0][w])), fabsf(bf16lo(vv[0][w])));
        if constexpr (U == 2) smax = fmax3(smax, fabsf(bf16lo(vu[U - 1][w])), fabsf(bf16lo(vv[U - 1][w])));
        // while P is at most 2^CA_RESCALE this bounds P s of every row of this lane
        if constexpr (NG == 1) {
          move = move || smax > sbound;
        } else {
          float f = fmaxf(vfac[w][0].x, vfac[w][0].y);
          if constexpr (RT == 2) f = fmax3(f, vfac[w][RT - 1].x, vfac[w][RT - 1].y);
          move = move || smax * f > CA_SBOUND;
        }
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          float2 al;
          al.x = follow(thr[j].x, nref[j].x, xm[j].x);
          al.y = follow(thr[j].y, nref[j].y, xm[j].y);
          l[j] = fmul2(l[j], al);
#pragma unroll
          for (int w = 0; w < NG; ++w) {
            zero[j][w] = fmul2(zero[j][w], al);
            float2 y = both(-INFINITY);  // score + log2 s, token by token (a hidden one: -inf)
#pragma unroll
            for (int e = 0; e < U; ++e) {
              const float lu = __log2f(fabsf(bf16lo(vu[e][w]))), lv = __log2f(fabsf(bf16lo(vv[e][w])));
              y.x = fmax3(y.x, x0[e][j].x + lu, x1[e][j].x + lv);
              y.y = fmax3(y.y, x0[e][j].y + lu, x1[e][j].y + lv);
            }
            const float fx = follow_scale(vfac[w][j].x, y.x, nref[j].x, al.x);
            const float fy = follow_scale(vfac[w][j].y, y.y, nref[j].y, al.y);
#pragma unroll
            for (int u = 4 * w; u < 4 * w + 4; ++u) {
              acc[u][j][0] *= fx;
              acc[u][j][1] *= fy;
              acc[u][j][2] *= fx;
              acc[u][j][3] *= fy;
            }
          }
        }
        if constexpr (NG == 1) {
          float f = fmaxf(vfac[0][0].x, vfac[0][0].y);
          if constexpr (RT == 2) f = fmax3(f, vfac[0][RT - 1].x, vfac[0][RT - 1].y);
          sbound = CA_SBOUND * over2(f, 0);
        }
      }
      // ---- per record: P, its sums and the B operands of the second product, then O^T += V^T P^T ----
#pragma unroll
      for (int e = 0; e < U; ++e) {
        uint32_t pb[NG][RT][2];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const float2 y0 = fadd2(x0[e][j], nref[j]), y1 = fadd2(x1[e][j], nref[j]);
          const float2 p0 = make_float2(fast_exp2(y0.x), fast_exp2(y0.y));
          const float2 p1 = make_float2(fast_exp2(y1.x), fast_exp2(y1.y));
          l[j] = fadd2(l[j], fadd2(p0, p1));
#pragma unroll
          for (int w = 0; w < NG; ++w) {
            const float m0 = bf16hi(vu[e][w]), m1 = bf16hi(vv[e][w]);
            float2 e0 = fmul2(fmul2(p0, vfac[w][j]), both(bf16lo(vu[e][w]))), e1 = fmul2(fmul2(p1, vfac[w][j]), both(bf16lo(vv[e][w])));
            if constexpr (EDGE) {  // a hidden token adds nothing, whatever its scale and minimum are (behind the sequence: anything)
              float2 z0 = fmul2(p0, both(m0)), z1 = fmul2(p1, both(m1));
              if (p0.x == 0.f) e0.x = z0.x = 0.f;
              if (p0.y == 0.f) e0.y = z0.y = 0.f;
              if (p1.x == 0.f) e1.x = z1.x = 0.f;
              if (p1.y == 0.f) e1.y = z1.y = 0.f;
              zero[j][w] = fadd2(zero[j][w], fadd2(z0, z1));
            } else {
              zero[j][w] = ffma2(p0, both(m0), ffma2(p1, both(m1), zero[j][w]));
            }
            pb[w][j][0] = transpose8x8(half2_of(e0.x, e0.y));
            pb[w][j][1] = transpose8x8(half2_of(e1.x, e1.y));
          }
        }
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          const uint4 v4 = *reinterpret_cast<const uint4 *>(p + e * S::REC + R::V + w * 512 + lane * 16);
          const uint32_t v[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t hi = v[u] >> 8;
#pragma unroll
            for (int j = 0; j < RT; ++j)
              mma_f16(acc[4 * w + u][j], v[u] & 0x000F000Fu, v[u] & 0x00F000F0u, hi & 0x000F000Fu, hi & 0x00F000F0u,
                      pb[w][j][0], pb[w][j][1]);
          }
        }
      }
    };

    // records that every row sees whole: up to r_full, and (window) up to r_sinks or from r_win on
    const int r_full = (sp.len - a.Nq - 15) >> 4;
    const int r_win = a.window > 0 ? ((sp.len - 1 - a.window) >> 4) + 1 : INT_MIN;
    const int r_sinks = a.sinks >> 4;
    for (int i = 0; i < nstep; ++i) {
      const uint32_t n = used + i, st = n % ST;
      const bool landed = mbar_wait(&cs.full[warp][st], (n / ST) & 1, &cs.abort, a.status);
      if (!__all_sync(0xffffffffu, landed)) break;
      const uint8_t *p = ring + st * (U * S::REC);
      const int k = k0 + 4 * U * i, r = record_at(k), r1 = record_at(k + U - 1);
      // (a step that holds the last of the first tokens and the window's first record is an edge)
      if (has_bad || k + U > kend || r1 > r_full || (r < r_win && (r1 >= r_sinks)))
        step(std::true_type{}, p, k);
      else
        step(std::false_type{}, p, k);
      __syncwarp();  // every lane has read the stage
      if (i + ST < nstep) issue(i + ST);
    }
    had_bad = has_bad;
    used += nstep;

    // ---- the item's (or its share's) end: the warps' sums into shared memory, then merged ----
    float *mo = reinterpret_cast<float *>(ring);  // every copy of the item has landed and been read
    float2 *ml = reinterpret_cast<float2 *>(smem + S::OFF_ML);
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 8 * j + 2 * c + k;
        float ls = k ? l[j].y : l[j].x;
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        float z[NG];
#pragma unroll
        for (int w = 0; w < NG; ++w) {
          z[w] = k ? zero[j][w].y : zero[j][w].x;
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) z[w] += __shfl_xor_sync(0xffffffffu, z[w], o);
        }
        if (g == 0) ml[warp * 8 * RT + row] = make_float2((k ? thr[j].y : thr[j].x) == -INFINITY ? -INFINITY : -(k ? nref[j].y : nref[j].x), ls);
        float back[NG];
#pragma unroll
        for (int w = 0; w < NG; ++w) back[w] = over2(k ? vfac[w][j].y : vfac[w][j].x, 24);
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          mo[row * S::OROW + 16 * u + g] = fmaf(acc[u][j][k], back[u / 4], z[u / 4]);
          mo[row * S::OROW + 16 * u + 8 + g] = fmaf(acc[u][j][2 + k], back[u / 4] * 0.0625f, z[u / 4]);
        }
      }
    ending = true;
    item_done = item;
    b_done = b;
    kvh_done = kvh;
    row_done = row0;
    first = tile0 == 0;
    last = tile0 + nt == tiles;
  }
  if (*reinterpret_cast<volatile int *>(&cs.abort)) {  // let copies already in flight land before the CTA exits
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
}

// Query rows of a KV head and items that a call takes (its places are 32-bit numbers).
bool too_many(int64_t B, int64_t Hkv, int64_t rows) {
  const int64_t rt = row_tile(rows);
  return rows > INT_MAX || B * Hkv > (int64_t(1) << 24) || B * Hkv * ((rows + 8 * rt - 1) / (8 * rt)) > INT_MAX / 2;
}

SplitWs ws_layout(int64_t B, int64_t Hkv, int64_t rows, int64_t d) {
  const int rt = row_tile(rows);
  return split_ws(B * Hkv * ((rows + 8 * rt - 1) / (8 * rt)), CA_SMS * ca_ctas(static_cast<int>(d), rt), rt, d);
}

template <int D, int RT, typename Args>
cudaError_t launch_cache_attn(const Args &a, int64_t tiles, cudaStream_t st) {
  using S = CaSmem<D, RT>;
  static std::atomic<unsigned long long> smem_set{0};
  if (cudaError_t e = set_smem_limit_once(cache4_attn_kernel<D, RT, Args>, S::TOTAL, smem_set); e != cudaSuccess) return e;
  const int64_t most = CA_SMS * ca_ctas(D, RT), ctas = tiles < most ? tiles : most;
  if (cudaError_t e = launch_dependent(cache4_attn_kernel<D, RT, Args>, dim3(static_cast<unsigned>(ctas)), CA_WARPS * 32, S::TOTAL, st, a);
      e != cudaSuccess)
    return e;
  if constexpr (Args::PARTIAL)
    return cudaSuccess;
  else
    return launch_split_combine<D, RT>(a, ctas, st);
}

// recs: an upper bound of the records that a sequence's queries see, for the number of CTAs (the lengths are on the device)
template <typename Args>
cudaError_t run_cache_attn(const Args &a, int d, int64_t recs, cudaStream_t s) {
  const int64_t step = 4 * CaSmem<128, 1>::U;  // records of a CTA's tile
  const int64_t tiles = ((recs + step - 1) / step + CA_ITEM) * a.B * a.Hkv * a.ntile;
  if (d == 128) return row_tile(a.rows) == 1 ? launch_cache_attn<128, 1>(a, tiles, s) : launch_cache_attn<128, 2>(a, tiles, s);
  return row_tile(a.rows) == 1 ? launch_cache_attn<64, 1>(a, tiles, s) : launch_cache_attn<64, 2>(a, tiles, s);
}

// The tensors, the pool and the scale of a call over the cache: checked, and what of its arguments follows from them (pages,
// lengths and the split's rows are the caller's).
int checked_args(const sparge_tensor *q, const sparge_cache4 *cache, float scale, sparge_tensor *o, View &qv, Cache4 &c,
                 CacheAttnArgs &a) {
  View ov;
  int rc;
  if ((rc = check_tensor(q, "q", &qv)) || (rc = check_tensor(o, "o", &ov)) || (rc = check_cache4(cache, &c))) return rc;
  if (qv.B != ov.B || qv.H != ov.H || qv.N != ov.N || qv.d != ov.d) return fail(SPARGE_ERR_INVALID_ARG, "o disagrees with q");
  if (qv.d != c.d) return fail(SPARGE_ERR_INVALID_ARG, "q and the cache disagree in d");
  if (qv.H % c.H) return fail(SPARGE_ERR_UNSUPPORTED, "Hq=%lld not a multiple of the cache's %d heads", (long long)qv.H, c.H);
  if (std::isnan(scale) || scale < 0.f || std::isinf(scale)) return fail(SPARGE_ERR_INVALID_ARG, "scale must be finite and >= 0");
  a.q = static_cast<const __nv_bfloat16 *>(qv.data);
  a.o = static_cast<__nv_bfloat16 *>(const_cast<void *>(ov.data));
  a.q_sb = qv.sb; a.q_sh = qv.sh; a.q_sn = qv.sn;
  a.o_sb = ov.sb; a.o_sh = ov.sh; a.o_sn = ov.sn;
  a.pool = c.data;
  a.n_pages = c.n_pages;
  a.rec_shift = c.page_shift - 4;
  a.Hkv = c.H;
  a.G = static_cast<int>(qv.H / c.H);
  a.window = a.sinks = 0;
  a.scale_log2 = (scale > 0.f ? scale : 1.f / sqrtf(static_cast<float>(qv.d))) * 1.4426950408889634f;
  return SPARGE_OK;
}
int checked_table(const Cache4 &c, int64_t width, int64_t table_stride) {
  if (width < 0 || table_stride < width || width > INT_MAX / c.page_size)
    return fail(SPARGE_ERR_INVALID_ARG, "table width %lld and stride %lld: the stride must reach the width, the width 2^31 tokens at most",
                (long long)width, (long long)table_stride);
  return SPARGE_OK;
}
// B sequences of Nq queries, and the workspace of their split
int set_split(CacheAttnArgs &a, int64_t B, int64_t Nq, int64_t d, void *ws, size_t ws_bytes) {
  const int64_t rows = a.G * Nq, rt = row_tile(rows);
  if (too_many(B, a.Hkv, rows)) return fail(SPARGE_ERR_UNSUPPORTED, "too many query rows");
  const SplitWs w = ws_layout(B, a.Hkv, rows, d);
  if (!ws || ws_bytes < w.total) return fail(SPARGE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", ws_bytes, w.total);
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(SPARGE_ERR_INVALID_ARG, "workspace not 256-byte aligned");
  a.B = static_cast<int>(B);
  a.Nq = static_cast<int>(Nq);
  a.rows = static_cast<int>(rows);
  a.ntile = static_cast<int>((rows + 8 * rt - 1) / (8 * rt));
  a.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.o);
  a.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + w.ml);
  a.ends = reinterpret_cast<int2 *>(static_cast<uint8_t *>(ws) + w.ends);
  return SPARGE_OK;
}

// Whether a call attends its prefix of `recs` records once for all sequences (rows: query rows of a KV head and sequence).
bool shares_prefix(int path, int64_t B, int64_t rows, int64_t Hkv, int64_t d, int64_t recs) {
  return recs > 0 && B * rows > 0 && (path == SPARGE_PREFIX_SHARED || prefix_shared(B, rows, Hkv, d, recs));
}

}  // namespace
}  // namespace sparge

using namespace sparge;

extern "C" {

size_t sparge_cache4_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || (d != 64 && d != 128) || Hq % Hkv || B > 65535 || Hq > 65535 ||
      Nq > (int64_t(1) << 30) || too_many(B, Hkv, Hq / Hkv * Nq))
    return 0;
  return ws_layout(B, Hkv, Hq / Hkv * Nq, d).total;
}

int sparge_cache4_attn(const sparge_tensor *q, const sparge_cache4 *cache, const int32_t *table, int64_t width,
                       int64_t table_stride, const int32_t *kv_lens, int64_t window, int64_t sinks, float scale,
                       sparge_tensor *o, void *ws, size_t ws_bytes, sparge_stream_t stream) {
  clear_error();
  View qv;
  Cache4 c;
  CacheAttnArgs a;
  int rc;
  if ((rc = checked_args(q, cache, scale, o, qv, c, a))) return rc;
  if (window < 0 || sinks < 0 || window > INT_MAX || sinks > INT_MAX)
    return fail(SPARGE_ERR_INVALID_ARG, "window=%lld and sinks=%lld must be in 0..2^31-1", (long long)window, (long long)sinks);
  if (window == 0 && sinks != 0) return fail(SPARGE_ERR_INVALID_ARG, "sinks need a window");
  if ((rc = checked_table(c, width, table_stride)) || (rc = set_split(a, qv.B, qv.N, qv.d, ws, ws_bytes))) return rc;
  if (qv.B == 0 || qv.N == 0) return SPARGE_OK;
  if (!kv_lens || (width && !table)) return fail(SPARGE_ERR_INVALID_ARG, "table or kv_lens is NULL");
  a.table = table;
  a.lens = kv_lens;
  a.table_stride = table_stride;
  a.width = static_cast<int>(width);
  a.window = static_cast<int>(window);
  a.sinks = static_cast<int>(sinks);
  a.status = status_ptr();
  int64_t recs = (width * c.page_size + 15) / 16;
  if (window > 0) {
    const int64_t most = (window + qv.N + 15) / 16 + 1 + (sinks + 15) / 16;
    recs = recs < most ? recs : most;
  }
  const cudaError_t e = run_cache_attn(a, static_cast<int>(qv.d), recs, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "cache attention launch");
}

size_t sparge_cache4_pages_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Nq < 0 || (d != 64 && d != 128) || Hq % Hkv || B > 65535 || Hq > 65535 ||
      Nq > (int64_t(1) << 30) || too_many(B * Nq, Hkv, Hq / Hkv))
    return 0;
  return ws_layout(B * Nq, Hkv, Hq / Hkv, d).total;
}

int sparge_cache4_pages_attn(const sparge_tensor *q, const sparge_cache4 *cache, const int32_t *pages, int64_t keep,
                             const int32_t *lens, float scale, sparge_tensor *o, void *ws, size_t ws_bytes,
                             sparge_stream_t stream) {
  clear_error();
  View qv;
  Cache4 c;
  CacheListArgs a;
  int rc;
  if ((rc = checked_args(q, cache, scale, o, qv, c, a))) return rc;
  if (keep < 0 || keep > INT_MAX / c.page_size)
    return fail(SPARGE_ERR_INVALID_ARG, "keep=%lld pages: 0 to 2^31 - 1 tokens", (long long)keep);
  if ((rc = set_split(a, qv.B * qv.N, 1, qv.d, ws, ws_bytes))) return rc;
  if (qv.B == 0 || qv.N == 0) return SPARGE_OK;
  if (!lens || (keep && !pages)) return fail(SPARGE_ERR_INVALID_ARG, "pages or lens is NULL");
  a.table = pages;
  a.lens = lens;
  a.table_stride = 0;
  a.width = static_cast<int>(keep);
  a.queries_of = static_cast<int>(qv.N);
  a.status = status_ptr();
  const cudaError_t e = run_cache_attn(a, static_cast<int>(qv.d), keep * c.page_size / 16, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "attention over selected pages: launch");
}

size_t sparge_cache4_prefix_attn_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d) {
  const size_t own = sparge_cache4_attn_workspace_bytes(B, Hq, Hkv, Nq, d);
  return own == 0 || B * (Hq / Hkv) * Nq > INT_MAX / 2 ? 0 : own + prefix_ws_bytes(B * (Hq / Hkv) * Nq, Hkv, d);
}

size_t sparge_cache4_prefix_attn_workspace_bytes_of(int64_t B, int64_t Hq, int64_t Hkv, int64_t Nq, int64_t d, int64_t prefix_tokens,
                                                    int path) {
  const size_t most = sparge_cache4_prefix_attn_workspace_bytes(B, Hq, Hkv, Nq, d);
  if (most == 0 || prefix_tokens < 0 || prefix_tokens > INT_MAX || (path != SPARGE_PREFIX_AUTO && path != SPARGE_PREFIX_SHARED)) return 0;
  const bool shared = shares_prefix(path, B, Hq / Hkv * Nq, Hkv, d, prefix_tokens / 16);
  return shared ? most : sparge_cache4_attn_workspace_bytes(B, Hq, Hkv, Nq, d);
}

int sparge_cache4_prefix_attn(const sparge_tensor *q, const sparge_cache4 *cache, const int32_t *prefix_pages, int64_t n_prefix,
                              const int32_t *table, int64_t width, int64_t table_stride, const int32_t *kv_lens, float scale,
                              int path, sparge_tensor *o, void *ws, size_t ws_bytes, sparge_stream_t stream) {
  clear_error();
  View qv;
  Cache4 c;
  CacheTailArgs a;
  int rc;
  if ((rc = checked_args(q, cache, scale, o, qv, c, a)) || (rc = checked_table(c, width, table_stride))) return rc;
  if (n_prefix < 0 || n_prefix > width)
    return fail(SPARGE_ERR_INVALID_ARG, "n_prefix=%lld pages not in 0..%lld, the table's width", (long long)n_prefix, (long long)width);
  if (path != SPARGE_PREFIX_AUTO && path != SPARGE_PREFIX_SHARED)
    return fail(SPARGE_ERR_INVALID_ARG, "path=%d: SPARGE_PREFIX_AUTO or SPARGE_PREFIX_SHARED", path);
  if (n_prefix && !prefix_pages) return fail(SPARGE_ERR_INVALID_ARG, "prefix_pages is NULL");
  if (qv.B * a.G * qv.N > INT_MAX / 2) return fail(SPARGE_ERR_UNSUPPORTED, "too many query rows");
  if ((rc = set_split(a, qv.B, qv.N, qv.d, ws, ws_bytes))) return rc;
  const int d = static_cast<int>(qv.d), per = c.page_size / 16;
  const bool shared = shares_prefix(path, qv.B, a.rows, c.H, d, n_prefix * per);
  const size_t own = ws_layout(qv.B, c.H, a.rows, d).total, need = own + (shared ? prefix_ws_bytes(qv.B * a.rows, c.H, d) : 0);
  if (ws_bytes < need) return fail(SPARGE_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes, need %zu", ws_bytes, need);
  if (qv.B == 0 || qv.N == 0) return SPARGE_OK;
  if (!kv_lens || (width && !table)) return fail(SPARGE_ERR_INVALID_ARG, "table or kv_lens is NULL");
  a.table = table;
  a.lens = kv_lens;
  a.table_stride = table_stride;
  a.width = static_cast<int>(width);
  a.status = status_ptr();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (!shared) {
    e = run_cache_attn(static_cast<const CacheAttnArgs &>(a), d, width * per, s);
    return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "cache attention launch");
  }
  a.first_rec = static_cast<int>(n_prefix) * per;
  PrefixAttn l;
  l.q = qv.data;
  l.q_sb = qv.sb; l.q_sh = qv.sh; l.q_sn = qv.sn;
  l.pool = c.data;
  l.pages = prefix_pages;
  l.lens = kv_lens;
  l.n_pages = c.n_pages;
  l.rec_shift = a.rec_shift;
  l.prefix = a.first_rec * 16;
  l.width = a.width;
  l.d = d;
  l.scale_log2 = a.scale_log2;
  l.ws = static_cast<uint8_t *>(ws) + own;
  l.status = a.status;
  e = launch_prefix_attn(l, a, s);
  if (e == cudaSuccess) e = run_cache_attn(a, d, (width - n_prefix) * per, s);
  if (e == cudaSuccess) e = launch_prefix_combine(l, a, s);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "attention behind a prefix: launch");
}

}  // extern "C"
