// Attention of a whole batch over a prefix that its sequences share, from the paged 4-bit cache, on tcgen05 tensor cores.
//
//   O = softmax(scale Q K^^T) V^ over the shared tokens for all B G Nq query rows of a KV head at once, K^ and V^ = code * scale +
//   minimum; left as shares (reference m, sum l, sum P V) that prefix_combine_kernel puts together with those of the
//   sequences' own tokens, which the cache attention makes.
//
// A sequence by itself reads every shared record again: 64 sequences over 32K tokens of 8 heads are 2.4 GB from L2, 370 us.  Here a
// record is read once, and its codes, widened once, serve 256 rows.
//
// Widening.  A code n is the subnormal f16 n 2^-24 once its four bits are masked out in place, so one fma.rn.f16x2 with (s 2^(f + 24),
// m 2^f) makes two elements of s n + m times 2^f: no conversion, one rounding, to f16.  f, one number for a tile's K and one for its V,
// takes the tile's largest scale to [2^-9, 2^-8), the most that s 2^(f + 24) allows (or the largest minimum: K's below 2^14, V's to
// 2^-3).  An element is off by at most 2^-11 of itself and 2^-15 of the largest scale.  So that no token takes bits from smaller ones, a
// tile whose tokens' sizes are more than 2^PF_EVEN apart is an uneven one: the warp that finds the powers scales the smaller tokens' words to
// the size of the largest, and the softmax takes each token's own powers from shared memory.  (It passes twice over the scores, in
// a function of its own: within the even tiles' code it cost those 5 % as a loop, up to 20 % unrolled or with the scores in local memory.  64 over
// 32K with every tile uneven: 78 us in place of 38, one of 16 tiles 43.)  Words give the
// channels of eight in the order 0 4 1 5 2 6 3 7, so Q is stored in that order; tokens of a tile stand in the order that the
// V records give (position 32 p + 8 c + 4 r + 2 h + i: token 2 c + 8 h + i of record 2 p + r), for K and V alike.
//
// Products.  S = Q K'^T (M = 128 rows, N = 64 tokens) and O += P' V' (N = d), kind::f16 with fp32 sums in TMEM.  P' = 2^(x + g - ref),
// g = -f of V, the token's own in an uneven tile: V's powers enter through P, and ref follows the row's largest x + g (of one token) when a P'
// passes 2^15, so O needs no rescaling when V's sizes change from tile to tile.  l is summed in fp32 against a reference m of its own.  Q is f16 times a power of two per row.
//
// A CTA holds two streams, each with its softmax warps, its warp that issues products, and its S, P and O: two tiles of 128 rows
// over the same tokens (more than 128 rows) or one tile of rows whose streams take the token tiles in turns.  The line of all
// (KV head, row group) items' tiles is cut into equal shares, so any batch fills all SMs.
//
// What bounds it.  64 sequences over 32K tokens of 8 heads, 4 rows each, d = 128, so 256 rows: 37.7 us (3.5e10 flops would take 18.5), of which
// 26.9 tiles of a CTA take 0.95 us each and 12 us are fixed: launch, Q, the first tiles' way through the roles, the shares' way out (63.2 us
// over 64K).  Over the kernel the tensor unit works 40 %, the schedulers issue 48 %, the special function unit 21 %, DRAM 12 %: no unit, but
// each stream's chain of scores, their way to registers, exponentials, P's way to TMEM and P V, with a wait at each step, that the other
// stream's alone does not cover.  12 over 128K (48 rows of 128 in use): 84.6 us, 0.70 a tile and 9 fixed; bytes would take 25.7.  Two
// streams take turns there, so a job of one takes 1.4 us, longer than with all rows in use; why is not known (more widening warps
// took it to 83 us in an earlier state, and fewer exponentials to nothing).  Every role is a warp or four that take the tiles one by one,
// so none may take longer than the rest: powers of two word by word, 1100 cycles a tile, took the kernel from 85 to 95 us.
// The code of the roles' loops is larger than what the SM's instruction cache holds: shorter code pays by itself (waits of ten
// instructions instead of forty and no second path for tiny V: hits 80 -> 96 %, 43 -> 41 and 104 -> 94 us; tiles that miss records by way of the
// uneven ones', and those in a function of their own: 40.3 -> 37.7 and 90.7 -> 84.6), and so do products that a whole warp issues, with descriptors in uniform registers
// (41 -> 38.7).  Tried and not faster: P in two places so that it need not wait for P V (39.1), scores in two places with P over them (39.0),
// two threads a row (46), eight warps that widen, in turns (39.5 and 83) or together (41 and 84), K and V freed apart (+5 %), powers of two
// per record (maxima no longer come with the load: +15 %), one product of 128 tokens for both streams of one row tile (they then wait for one another: +30 %).
#include <climits>
#include <cmath>
#include <type_traits>

#include "cache4.cuh"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"
#include "rowsplit.cuh"

namespace sparge {
namespace {

// Warps: softmax (4 per stream, a row a thread), widening, products (one per stream), loads, powers of two.
constexpr int PF_SOFT = 8, PF_WIDE = 4, PF_PROD = PF_SOFT + PF_WIDE, PF_LOAD = PF_PROD + 2;
constexpr int PF_THREADS = (PF_LOAD + 2) * 32;
constexpr int PF_ROWS = 256;     // rows of a slot: two streams of 128
// The references move when a P or a P' passes 2^15, the last power of two within f16, and the row's largest P' then stands at 2^8: with
// 2^7 to grow before the next move, and 22 powers of two below it that f16 holds whole.
constexpr float PF_TOP = 15.f, PF_ROOM = 8.f;
// Tokens of a tile whose sizes' exponents are no further apart share its powers of two; in an uneven tile each has its own.
constexpr int PF_EVEN = 4;

struct PrefixArgs {
  const __nv_bfloat16 *q;
  int64_t q_sb, q_sh, q_sn;
  const uint8_t *pool;
  const int32_t *pages;
  int64_t n_pages;
  int rec_shift, recs, tiles;       // records of a page (1 << rec_shift), of the prefix; 64-token tiles
  int Hkv, G, Nq, rows, groups;     // rows of a KV head: B G Nq; groups of them: items of a KV head
  float scale_log2;
  float *part_o, *part_ml;          // [CTA + item][D / 32][256][32], [CTA + item][256] (reference, sum)
  int *status;
};

// D channels; R = 2: the streams are two tiles of 128 rows, each over every 64-token tile; R = 1: one tile of rows, the
// streams take turns over the token tiles.
template <int D, int R>
struct PfCfg {
  static constexpr int PITCH = Rec4<D>::BYTES + 64;  // of a record in the ring, so that two of them fall on different banks
  static constexpr int RAW = 4 * PITCH;
  static constexpr int RS = 6, NS = R == 2 ? 3 : 4;  // stages of raw tiles, of widened ones: of K, and of V
  static constexpr bool QSMEM = D == 128 && R == 2;  // no room in TMEM for two tiles of Q
  static constexpr uint32_t TILE = 64 * D * 2;       // of K or V, f16
  static constexpr uint32_t OUT = 128 * 32 * 4;      // 32 channels of a stream's O on their way out; over its Q where that lies here
  static constexpr uint32_t K = 0, V = K + NS * TILE, Q = V + NS * TILE, QB = QSMEM ? 128 * D * 2 : OUT, RING = Q + 2 * QB;
  static constexpr uint32_t CTRL = RING + RS * RAW, SMEM = CTRL + 9216;
  // TMEM columns
  static constexpr uint32_t O = 0, S = 2 * D, P = S + 128, QC = P + 64, QCOLS = D / 2;
  static_assert(QC + (QSMEM ? 0 : R) * QCOLS <= 512, "TMEM");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
// What goes with a tile: K = K' 2^-kf, V = V' 2^-vf; bit r of missing: its record r is not there.  In an uneven tile (one that misses
// records is) a token's are K' 2^-kf k_by and V' 2^v_by.
struct alignas(16) PfInfo {
  int kf, vf;
  uint32_t missing, uneven;
};
struct PfCtrl {
  PfInfo info[16];  // (tile % 16: a tile that far behind has been turned into P)
  alignas(16) float k_by[16][64], v_by[16][64];  // of uneven tiles, in the order of the scores' columns
  uint64_t raw_full[8], raw_free[8], info_full[8], kv_full[4], kv_free[4];
  uint64_t q_full[2], q_free, s_full[2], s_free[2], p_full[2], pv_done[2], drained[2];
  uint8_t bad[8][4];
  uint32_t tmem;
  int abort, no_abort;
};
static_assert(sizeof(PfCtrl) <= 9216, "control block");

__device__ __forceinline__ void pf_bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
// mbar_wait in few instructions: the loop's code of all roles has to stay in the instruction cache.
__device__ __forceinline__ bool pf_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  uint32_t t0, t;
  asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t0));
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
    if (t - t0 > 2000000000u) *abort = 1;
    if (*abort) return false;
  }
  return true;
}
// One lane of the warp, always the same one.  The products' warps run as a whole and branch on values that are the same in all lanes, so
// that descriptors are made in uniform registers.
__device__ __forceinline__ bool pf_one_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0u;
}
__device__ __forceinline__ uint32_t pf_hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t pf_sixteenth2(uint32_t a) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x2C002C00u));
  return r;
}
__device__ __forceinline__ void pf_sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 pf_lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
// tcgen05.wait::ld that the loaded registers pass through, so nothing that uses them moves in front of it.
__device__ __forceinline__ void pf_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void pf_ld_wait_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

__device__ __forceinline__ void pf_ld_wait_for(uint32_t (&r)[32], float &m) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+f"(m)
               :
               : "memory");
}
// What a power of two f has to keep to, from the exponents of scales and minima: f <= -need, so that a code's 2^-24 code * s 2^(f + 24)
// is within f16 and K's minimum below 2^14.  V's minimum goes to 2^-3, where its scale's codes are, so that x - f says within a
// few powers of two what a token of score x can add to O.
template <bool V>
__device__ __forceinline__ int pf_need(uint32_t word) {
  return max(static_cast<int>((word >> 7) & 0xFFu) + 9, static_cast<int>((word >> 23) & 0xFFu) + (V ? 4 : -13)) - 127;
}
// Nothing: a scale or minimum that is not finite makes its own values NaN, whatever the power.
constexpr int PF_NO_NEED = -200;
template <bool V>
__device__ __forceinline__ int pf_finite_need(uint32_t word) {
  return ((word & 0x7F80u) == 0x7F80u || (word & 0x7F800000u) == 0x7F800000u) ? PF_NO_NEED : pf_need<V>(word);
}
__device__ __forceinline__ int pf_power(int need) { return min(max(-need, -126), 100); }
// A scale and a minimum times 2^by, exactly.
__device__ __forceinline__ uint32_t pf_word_by(uint32_t word, int by) {
  const float f = pow2i(by);
  return pack_bf16x2(bf16lo(word) * f, bf16hi(word) * f);
}

// An uneven tile's scores, 64 columns of TMEM: l and m take them in, then x + g of each token stands in their place.
__device__ __noinline__ float2 pf_uneven(uint32_t sc, const float *k_by, const float *v_by, uint32_t missing, float mult, float m, float l) {
  float xm = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 128; i += 16) {  // every 16 columns for the maximum, then again for the sum
    uint32_t x[16];
    tmem_ld16(sc + (i & 63), x);
    pf_ld_wait_for(x);
    if (i == 64) {
      const float mn = fmaxf(m, xm);
      l *= m == -INFINITY ? 0.f : fast_exp2(m - mn);
      m = mn;
    }
    const float *by = (i < 64 ? k_by : v_by) + (i & 63);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float y = __uint_as_float(x[k]);
      if (i < 64) {  // column 32 h + 8 c + 4 r + i is a token of record 2 h + r
        y = ((missing >> (2 * (i >> 5) + ((k >> 2) & 1))) & 1u) ? -INFINITY : y * by[k] * mult;
        xm = fmaxf(xm, y);
      } else {
        l += fast_exp2(m == -INFINITY ? y : y - m);
        y += by[k];
      }
      x[k] = __float_as_uint(y);
    }
    tmem_st16(sc + (i & 63), x);
    tmem_st_wait();
  }
  return make_float2(m, l);
}

// A CTA's share of the line of all items' tiles, and its pieces: item, first tile, tiles.
struct PfShare {
  int64_t at, end;
  __host__ __device__ __forceinline__ static int64_t cut(int64_t total, int cta, int ctas) { return total * cta / ctas; }
  __device__ __forceinline__ PfShare(const PrefixArgs &a) {
    const int64_t total = static_cast<int64_t>(a.Hkv) * a.groups * a.tiles;
    at = cut(total, blockIdx.x, gridDim.x);
    end = cut(total, blockIdx.x + 1, gridDim.x);
  }
  __device__ __forceinline__ bool next(const PrefixArgs &a, int &item, int &tile0, int &n) {
    if (at >= end) return false;
    item = static_cast<int>(at / a.tiles);
    tile0 = static_cast<int>(at - static_cast<int64_t>(item) * a.tiles);
    n = static_cast<int>(min(end - at, static_cast<int64_t>(a.tiles - tile0)));
    at += n;
    return true;
  }
};

template <int D, int R>
__global__ void __launch_bounds__(PF_THREADS, 1) prefix_attn_kernel(const PrefixArgs a) {
  using C = PfCfg<D, R>;
  using Rec = Rec4<D>;
  constexpr int NG = D / 64, NS = C::NS, RS = C::RS;
  constexpr uint32_t IDESC_S = idesc_f32acc(128, 64, FMT_F16, false);
  constexpr uint32_t IDESC_PV = idesc_f32acc(128, D, FMT_F16, false);
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzle of the MMA descriptors assumes 1024-byte aligned tiles
    start_after_earlier();
    if (threadIdx.x == 0) record_status(a.status, -4 /* SPARGE_ERR_CUDA */);
    return;
  }
  PfCtrl &cs = *reinterpret_cast<PfCtrl *>(smem + C::CTRL);
  volatile int *abort = &cs.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < RS; ++s) {
      mbar_init(&cs.raw_full[s], 4);
      mbar_init(&cs.raw_free[s], PF_WIDE);
      mbar_init(&cs.info_full[s], 1);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&cs.kv_full[s], PF_WIDE);
      mbar_init(&cs.kv_free[s], R);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&cs.q_full[t], 4);
      mbar_init(&cs.s_full[t], 1);
      mbar_init(&cs.s_free[t], 4);
      mbar_init(&cs.p_full[t], 4);
      mbar_init(&cs.pv_done[t], 1);
      mbar_init(&cs.drained[t], 1);
    }
    mbar_init(&cs.q_free, 1);
    cs.abort = 0;
    cs.no_abort = 0;
    fence_barrier_init();
  }
  if (warp == PF_PROD) {
    tmem_alloc(&cs.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  start_after_earlier();
  const uint32_t tmem = cs.tmem;
  PfShare share(a);
  int item, tile0, n;  // the piece: tiles tile0 .. tile0 + n - 1 of the item
  uint32_t tc = 0;     // tiles of the CTA's pieces before this one

  if (warp < PF_SOFT) {
    // ------------------------------------ softmax ------------------------------------
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t oc = tl + C::O + t * D, sc = tl + C::S + t * 64, pc = tl + C::P + t * 32;
    const uint32_t qb = base + C::Q + t * C::QB;  // the stream's Q or, at a piece's end, its O
    uint32_t done = 0, piece = 0;                 // jobs of this stream so far, pieces
    bool ok = true;
    for (; share.next(a, item, tile0, n); ++piece) {
      const int kvh = item / a.groups, r = (item % a.groups) * (128 * R) + (R == 2 ? t * 128 : 0) + row;
      const bool live = r - lane < a.rows;  // a warp past the last row takes part in the waits alone
      // ---- the row's queries: to their place as they are, then in place f16, times a power of two that takes the maximum to [2^14, 2^15),
      // in each 8 channels in the order 0 4 1 5 2 6 3 7, in which the codes' words give them ----
      float rm;  // 2^(e - 14) scale: what a product of the scaled row counts
      {
        if (R == 1 && t == 0 && piece > 0) {  // the other stream's products with the rows before these have been made (this one's have)
          ok = __all_sync(0xffffffffu, pf_wait(&cs.q_free, (piece - 1) & 1, abort));
          if (bar_red_or(1 + t, 128, !ok)) {  // (all four warps leave, or none)
            ok = false;
            break;
          }
          tc_fence_after();
        }
        const bool keep = R == 2 || t == 0;  // (the second stream of one row tile wants the power alone)
        const uint32_t qc = tl + C::QC + (R == 2 ? t * C::QCOLS : 0);
        const int b = r / (a.G * a.Nq), rr = r % (a.G * a.Nq);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + b * a.q_sb + (kvh * a.G + rr / a.Nq) * a.q_sh +
                                                           static_cast<int64_t>(rr % a.Nq) * a.q_sn);
        auto place = [&](int i) { return qb + (i / 8) * 16384 + row * 128 + (((i & 7) ^ (row & 7)) << 4); };
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; i += 8) {
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = r < a.rows ? src[i + k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(u[x])), fabsf(bf16hi(u[x]))));
          }
          if (keep) {
            if (C::QSMEM) {
#pragma unroll
              for (int k = 0; k < 8; ++k) pf_sts128(place(i + k), v[k].x, v[k].y, v[k].z, v[k].w);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  w[4 * k] = v[4 * h + k].x;
                  w[4 * k + 1] = v[4 * h + k].y;
                  w[4 * k + 2] = v[4 * h + k].z;
                  w[4 * k + 3] = v[4 * h + k].w;
                }
                tmem_st16(qc + 4 * i + 16 * h, w);
              }
            }
          }
        }
        const int e = min(max(exponent_of(mx), -100), 116);
        const float f = pow2i(14 - e);
        rm = a.scale_log2 * pow2i(e - 14);
        auto scaled = [&](uint4 u) {
          return make_uint4(half2_of(bf16lo(u.x) * f, bf16lo(u.z) * f), half2_of(bf16hi(u.x) * f, bf16hi(u.z) * f),
                            half2_of(bf16lo(u.y) * f, bf16lo(u.w) * f), half2_of(bf16hi(u.y) * f, bf16hi(u.w) * f));
        };
        if (keep) {
          if (C::QSMEM) {
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              const uint4 u = scaled(pf_lds128(place(i)));
              pf_sts128(place(i), u.x, u.y, u.z, u.w);
            }
          } else {
            tmem_st_wait();
#pragma unroll 1
            for (int i = 0; i < D / 2; i += 16) {
              uint32_t w[16];
              tmem_ld16(qc + i, w);
              pf_ld_wait_for(w);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                const uint4 u = scaled(make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]));
                w[k] = u.x;
                w[k + 1] = u.y;
                w[k + 2] = u.z;
                w[k + 3] = u.w;
              }
              tmem_st16(qc + i, w);
            }
            tmem_st_wait();
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&cs.q_full[t]);
        }
      }
      // m: the reference of l = sum of P, P = 2^(x - m); ref: that of O = sum of P' V', P' = 2^(x + g - ref).  When a term passes 2^15 of
      // them, m is set to the largest x that the row sees and ref to 2^PF_ROOM below its largest x + g; what the sums hold is then scaled down.
      float m = -INFINITY, ref = -INFINITY, l = 0.f;
      const int jobs = R == 2 ? n : (n - t + 1) / 2;
      for (int j = 0; j < jobs; ++j, ++done) {
        const uint32_t tile = tc + (R == 2 ? j : 2 * j + t), st = tile % NS;
        // (what the widened tile's barrier orders, its powers among it, is there before its scores are)
        ok = pf_wait(&cs.s_full[t], done & 1, abort) && pf_wait(&cs.kv_full[st], (tile / NS) & 1, abort);
        const PfInfo info = cs.info[tile & 15];
        float mult = fminf(fmaxf(rm * pow2i(-info.kf), 0x1p-126f), 0x1p127f);  // (no 0 times -inf, no infinity times 0)
        float g = static_cast<float>(-info.vf), apart = 0.f;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[2][32];
        float mh[2];
        if (live) {
          if (info.uneven) [[unlikely]] {
            const float2 ml = pf_uneven(sc, cs.k_by[tile & 15], cs.v_by[tile & 15], info.missing, mult, m, l);
            m = ml.x;
            l = ml.y;
            mult = 1.f;
            g = 0.f;
            apart = -INFINITY;
          }
          tmem_ld32_max(sc, v[0], mh[0]);
          tmem_ld32_max(sc + 32, v[1], mh[1]);
          pf_ld_wait_for(v[0], mh[0]);
          pf_ld_wait_for(v[1], mh[1]);
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&cs.s_free[t]);
        if (j > 0) {  // the product before this one has read its P and added to O
          ok = ok && pf_wait(&cs.pv_done[t], (done - 1) & 1, abort);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (live) {
          const float top = fmaxf(mh[0], mh[1]) * mult, ym = top + g, xm = top + apart;
          const bool move = xm > m + PF_TOP || ym > ref + PF_TOP;
          if (__any_sync(0xffffffffu, move)) {
            float f = 1.f;
            if (move) {
              const float mn = fmaxf(m, xm), rn = fmaxf(ym - PF_ROOM, ref);
              l *= m == -INFINITY ? 0.f : fast_exp2(m - mn);
              f = ref == -INFINITY ? 0.f : fast_exp2(ref - rn);
              m = mn;
              ref = rn;
            }
            if (j > 0) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(oc + 16 * q, o);
                pf_ld_wait_for(o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(oc + 16 * q, o);
              }
            }
          }
          // (a row whose references are still -inf has only hidden columns, or NaN)
          const bool none = ref == -INFINITY;
          // P' = 2^(x + nr), P = P' 2^back; where V of this tile is so small beside what O holds that its P' is 0, back stops where l's terms do not
          const float back = none ? 0.f : fminf((ref - m) - g, 60.f - apart), nr = none ? 0.f : -m - back;
          const float2 m2 = make_float2(mult, mult), n2 = make_float2(nr, nr);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 e2 = ffma2(make_float2(__uint_as_float(v[h][2 * k]), __uint_as_float(v[h][2 * k + 1])), m2, n2);
              const float2 p2 = make_float2(fast_exp2(e2.x), fast_exp2(e2.y));
              sum[k & 1] = fadd2(sum[k & 1], p2);
              pk[k] = pack_f16x2(p2.x, p2.y);
            }
            tmem_st16(pc + 16 * h, pk);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&cs.p_full[t]);
          const float2 s2 = fadd2(sum[0], sum[1]);
          l = fmaf(s2.x + s2.y, fast_exp2(back + apart), l);
        } else {
          if (lane == 0) mbar_arrive(&cs.p_full[t]);
        }
      }
      // ---- the piece's end: O against m, 32 channels of the stream's rows at a time through shared memory, then the references and
      // sums.  (The four warps leave together if one's wait gave up.) ----
      if (ok && jobs > 0) {
        ok = __all_sync(0xffffffffu, pf_wait(&cs.pv_done[t], (done - 1) & 1, abort));
        tc_fence_after();
      }
      if (bar_red_or(1 + t, 128, !ok)) {
        ok = false;
        break;
      }
      const int64_t slot = static_cast<int64_t>(blockIdx.x) + item;
      if (r < a.rows) *reinterpret_cast<float2 *>(a.part_ml + 2 * (slot * PF_ROWS + t * 128 + row)) = make_float2(m, l);
      if (jobs > 0) {
        const float back = ref == -INFINITY ? 1.f : fast_exp2(ref - m);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          if (live) {
            uint32_t o[32];
            tmem_ld32(oc + 32 * q, o);
            pf_ld_wait_for(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * back);
#pragma unroll
            for (int k = 0; k < 8; ++k) pf_sts128(qb + row * 128 + ((k ^ (row & 7)) << 4), o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          fence_proxy_async_smem();
          bar_sync(1 + t, 128);
          if ((threadIdx.x & 127) == 0) {
            pf_bulk_store(a.part_o + ((slot * (D / 32) + q) * PF_ROWS + t * 128) * 32, qb, C::OUT);
            bulk_commit();
            bulk_wait_read_all();
          }
          bar_sync(1 + t, 128);
        }
        tc_fence_before();
      }
      tc += n;
    }
    if ((threadIdx.x & 127) == 0) bulk_wait_all();
  } else if (warp < PF_PROD) {
    // ------------------------------------ widening: codes to f16 tiles ------------------------------------
    // K and V have stages of their own, so that K's is free with the scores, and V's is not held while they are turned into P.
    const int w4 = warp & 3;
    const uint32_t total = static_cast<uint32_t>(share.end - share.at);  // tiles of all the CTA's pieces
    for (uint32_t tile = 0; tile < total; ++tile) {
      const uint32_t rs = tile % RS, st = tile % NS;
      bool ok = pf_wait(&cs.info_full[rs], (tile / RS) & 1, abort) && pf_wait(&cs.raw_full[rs], (tile / RS) & 1, abort);
      if (tile >= NS) ok = ok && pf_wait(&cs.kv_free[st], (tile / NS - 1) & 1, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t *raw = smem + C::RING + rs * C::RAW;
      const PfInfo info = cs.info[tile & 15];
      const int pk = w4 & 1;  // the pair of records whose K this warp takes
      // ---- K: a lane takes the codes of 8-channel piece c of every 32 channels of a token ----
      {
        const int c = lane & 3, r = (lane >> 2) & 1;
        const int f = info.kf;
        const bool there = !((info.missing >> (2 * pk + r)) & 1u);
        const float fs = there ? pow2i(f + 24) : 0.f, fm = there ? pow2i(f) : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int t = ((w4 >> 1) + 2 * k) * 4 + (lane >> 3);
          const int pos = 32 * pk + 8 * ((t & 7) >> 1) + 4 * r + 2 * (t >> 3) + (t & 1);
          const uint8_t *from = raw + (2 * pk + r) * C::PITCH, *src = from + Rec::K + t * (D / 2) + c * (D / 8);
          uint32_t code[2 * NG], word[NG];
          if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src);
            const uint2 x = *reinterpret_cast<const uint2 *>(from + Rec::KW + t * 8);
            code[0] = u.x; code[1] = u.y; code[2] = u.z; code[3] = u.w;
            word[0] = x.x; word[1] = x.y;
          } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(src);
            code[0] = u.x; code[1] = u.y;
            word[0] = *reinterpret_cast<const uint32_t *>(from + Rec::KW + t * 4);
          }
          const uint32_t to = base + C::K + st * C::TILE + pos * 128;
#pragma unroll
          for (int w = 0; w < 2 * NG; ++w) {
            const float sf = there ? bf16lo(word[w / 2]) * fs : 0.f, mf = there ? bf16hi(word[w / 2]) * fm : 0.f;
            const uint32_t lo = half2_of(sf, sf), hi = pf_sixteenth2(lo), m = half2_of(mf, mf), u = code[w], u8 = u >> 8;
            pf_sts128(to + (w >> 1) * 8192 + (((4 * (w & 1) + c) ^ (pos & 7)) << 4), pf_hfma2(u & 0x000F000Fu, lo, m),
                      pf_hfma2(u & 0x00F000F0u, hi, m), pf_hfma2(u8 & 0x000F000Fu, lo, m), pf_hfma2(u8 & 0x00F000F0u, hi, m));
          }
        }
      }
      // ---- V, transposed: lane 4 g + c holds channels g and g + 8 of every 16 for tokens 2c, 2c + 1, 2c + 8, 2c + 9 of two records ----
      {
        const int g = lane >> 2, c = lane & 3;
        constexpr int NU = 2 * NG;  // words of a warp: d = 128: a half of the channels and a pair of records; d = 64: a quarter
        const int part = D == 128 ? w4 >> 1 : 0, u0 = D == 128 ? 0 : 2 * (w4 >> 1), pr = (w4 & 1) ^ (g & 1);
        uint32_t ss[4], sh[4], mm[4], code[2][NU];  // of tokens (2c, 2c + 1) and (2c + 8, 2c + 9) of either record
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint8_t *from = raw + (2 * pr + r) * C::PITCH, *src = from + Rec::V + part * 512 + 16 * lane + 4 * u0;
          const int f = info.vf;
          const bool there = !((info.missing >> (2 * pr + r)) & 1u);
          const float fs = pow2i(f + 24), fm = pow2i(f);
          if constexpr (NU == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src);
            code[r][0] = u.x; code[r][1] = u.y; code[r][2] = u.z; code[r][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(src);
            code[r][0] = u.x; code[r][1] = u.y;
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t x, y;
            if constexpr (NG == 2) {
              const uint4 u = *reinterpret_cast<const uint4 *>(from + Rec::VW + (2 * c + 8 * k) * 8);
              x = part ? u.y : u.x;
              y = part ? u.w : u.z;
            } else {
              const uint2 u = *reinterpret_cast<const uint2 *>(from + Rec::VW + (2 * c + 8 * k) * 4);
              x = u.x;
              y = u.y;
            }
            if (!there) x = y = 0u;
            ss[2 * r + k] = half2_of(bf16lo(x) * fs, bf16lo(y) * fs);
            mm[2 * r + k] = half2_of(bf16hi(x) * fm, bf16hi(y) * fm);
            sh[2 * r + k] = pf_sixteenth2(ss[2 * r + k]);
          }
        }
        const uint32_t to = base + C::V + st * C::TILE + (((4 * pr + c) ^ g) << 4);
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          const uint32_t at = to + (64 * part + 16 * (u0 + u) + g) * 128;
          const uint32_t a0 = code[0][u], a8 = a0 >> 8, b0 = code[1][u], b8 = b0 >> 8;
          pf_sts128(at, pf_hfma2(a0 & 0x000F000Fu, ss[0], mm[0]), pf_hfma2(a8 & 0x000F000Fu, ss[1], mm[1]),
                    pf_hfma2(b0 & 0x000F000Fu, ss[2], mm[2]), pf_hfma2(b8 & 0x000F000Fu, ss[3], mm[3]));
          pf_sts128(at + 8 * 128, pf_hfma2(a0 & 0x00F000F0u, sh[0], mm[0]), pf_hfma2(a8 & 0x00F000F0u, sh[1], mm[1]),
                    pf_hfma2(b0 & 0x00F000F0u, sh[2], mm[2]), pf_hfma2(b8 & 0x00F000F0u, sh[3], mm[3]));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&cs.kv_full[st]);
        mbar_arrive(&cs.raw_free[rs]);
      }
    }
  } else if (warp < PF_LOAD) {
    // ------------------------------------ products of one stream ------------------------------------
    // (a warp for each stream: waits, fences and issue of a job take it about as long as the tensor unit takes the products)
    const int t = __shfl_sync(0xffffffffu, warp - PF_PROD, 0);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t dk = smem_desc_sw128(base + C::K, 16, 1024), dv = smem_desc_sw128(base + C::V, 16, 1024);
    const uint64_t dq = smem_desc_sw128(base + C::Q + (C::QSMEM ? t * C::QB : 0), 16, 1024);
    const uint32_t sc = tm + C::S + t * 64, oc = tm + C::O + t * D, pc = tm + C::P + t * 32;
    const uint32_t qc = tm + C::QC + (R == 2 ? t * C::QCOLS : 0);
    uint32_t done = 0, piece = 0;  // jobs so far, pieces
    bool ok = true;
    for (; ok && share.next(a, item, tile0, n); ++piece) {
      const int jobs = R == 2 ? n : (n - t + 1) / 2;
      ok = __all_sync(0xffffffffu, pf_wait(&cs.q_full[R == 2 ? t : 0], piece & 1, abort));
      for (int j = 0; ok && j <= jobs; ++j) {
        if (j < jobs) {  // scores of job j, once the softmax has read those before
          const uint32_t tile = tc + (R == 2 ? j : 2 * j + t), st = tile % NS;
          ok = pf_wait(&cs.kv_full[st], (tile / NS) & 1, abort) && (done == 0 || pf_wait(&cs.s_free[t], (done - 1) & 1, abort));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (pf_one_lane()) {
            const uint64_t b = dk + st * (C::TILE >> 4);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              if (C::QSMEM)
                mma_bf16_ss(sc, dq + (s >> 2) * (16384 >> 4) + (s & 3) * 2, b + (s >> 2) * (8192 >> 4) + (s & 3) * 2, IDESC_S, s > 0 ? 1u : 0u);
              else
                mma_bf16_ts(sc, qc + s * 8, b + (s >> 2) * (8192 >> 4) + (s & 3) * 2, IDESC_S, s > 0 ? 1u : 0u);
            }
            mma_commit(&cs.s_full[t]);
            if (R == 1 && t == 1 && j == jobs - 1) mma_commit(&cs.q_free);
          }
          __syncwarp();
          ++done;
        }
        if (j > 0) {  // P V of job j - 1
          const uint32_t tile = tc + (R == 2 ? j - 1 : 2 * (j - 1) + t), st = tile % NS, nth = done - (j < jobs ? 2 : 1);
          ok = __all_sync(0xffffffffu, pf_wait(&cs.p_full[t], nth & 1, abort));
          if (!ok) break;
          tc_fence_after();
          if (pf_one_lane()) {
            const uint64_t b = dv + st * (C::TILE >> 4);
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_bf16_ts(oc, pc + s * 8, b + s * 2, IDESC_PV, s > 0 || j > 1 ? 1u : 0u);
            mma_commit(&cs.pv_done[t]);
            mma_commit(&cs.kv_free[st]);
          }
          __syncwarp();
        }
      }
      if (R == 1 && t == 1 && jobs == 0 && pf_one_lane()) mma_commit(&cs.q_free);
      __syncwarp();
      tc += n;
    }
    if (!ok) {  // products in flight end before the CTA gives its TMEM back
      if (pf_one_lane()) mma_commit(&cs.drained[t]);
      __syncwarp();
      pf_wait(&cs.drained[t], 0, &cs.no_abort);
    }
    __syncwarp();
  } else if (warp == PF_LOAD) {
    // ------------------------------------ loads ------------------------------------
    bool ok = true;
    while (ok && share.next(a, item, tile0, n)) {
      const int kvh = item / a.groups;
      const uint8_t *src = nullptr;  // of record 4 (j0 + lane / 4) + lane % 4 of the piece's tiles
      int j0 = -8;
      for (int j = 0; j < n; ++j) {
        if (j >= j0 + 8) {  // the pages of 32 records at a time
          j0 = j;
          src = nullptr;
          const int r = 4 * (tile0 + j) + lane;
          if (r < a.recs && j + lane / 4 < n) {
            const int page = a.pages[r >> a.rec_shift];
            if (page < 0 || page >= a.n_pages)
              record_status(a.status, -1 /* SPARGE_ERR_INVALID_ARG */);
            else
              src = a.pool + (((static_cast<int64_t>(page) * a.Hkv + kvh) << a.rec_shift) + (r & ((1 << a.rec_shift) - 1))) * Rec::BYTES;
          }
        }
        const uint32_t tile = tc + j, rs = tile % RS;
        if (tile >= RS) ok = pf_wait(&cs.raw_free[rs], (tile / RS - 1) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane / 4 == j - j0) {
          uint64_t *bar = &cs.raw_full[rs];
          cs.bad[rs][lane & 3] = src == nullptr;
          if (src != nullptr) {
            mbar_arrive_expect_tx(bar, Rec::BYTES);
            bulk_load(smem + C::RING + rs * C::RAW + (lane & 3) * C::PITCH, src, Rec::BYTES, bar);
          } else {
            mbar_arrive(bar);
          }
        }
        __syncwarp();
      }
      tc += n;
    }
    if (!ok) {  // let copies in flight land before the CTA exits
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 1000000ull) {
      }
    }
  } else {
    // ------------------------------------ powers of two ------------------------------------
    // A tile's K and its V get one each from its 64 tokens' words: the largest scale to [2^-9, 2^-8), which is what a code of
    // 2^-24 code leaves in f16, or where the minima are larger the largest of them to [2^13, 2^14).
    const uint32_t total = static_cast<uint32_t>(share.end - share.at);
    for (uint32_t tile = 0; tile < total; ++tile) {
      const uint32_t rs = tile % RS;
      if (!__all_sync(0xffffffffu, pf_wait(&cs.raw_full[rs], (tile / RS) & 1, abort))) break;
      const uint32_t bad = *reinterpret_cast<const uint32_t *>(cs.bad[rs]);  // a byte a record
      // lane 8 rec + k looks at the words of tokens 2k and 2k + 1 of a record
      const int rec = lane >> 3;
      const uint8_t *at = smem + C::RING + rs * C::RAW + rec * C::PITCH + (lane & 7) * (8 * NG);
      uint32_t u[2][2 * NG];
      if constexpr (NG == 2) {
        const uint4 x = *reinterpret_cast<const uint4 *>(at + Rec::KW), y = *reinterpret_cast<const uint4 *>(at + Rec::VW);
        u[0][0] = x.x; u[0][1] = x.y; u[0][2] = x.z; u[0][3] = x.w;
        u[1][0] = y.x; u[1][1] = y.y; u[1][2] = y.z; u[1][3] = y.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(at + Rec::KW), y = *reinterpret_cast<const uint2 *>(at + Rec::VW);
        u[0][0] = x.x; u[0][1] = x.y;
        u[1][0] = y.x; u[1][1] = y.y;
      }
      const bool there = ((bad >> (8 * rec)) & 1u) == 0u;
      int own[2][2], top[2], low[2];  // of K, V: the two tokens' needs, the tile's largest and (but for tokens of zeros) smallest
      uint32_t some[2][2];            // a token's scales and minima
      auto reduce = [&] {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          top[s] = __reduce_max_sync(0xffffffffu, there ? max(own[s][0], own[s][1]) : PF_NO_NEED);
          low[s] = __reduce_min_sync(0xffffffffu, min(there && some[s][0] != 0u ? own[s][0] : 255, there && some[s][1] != 0u ? own[s][1] : 255));
        }
      };
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          some[s][k] = NG == 2 ? __vmaxu2(u[s][NG * k] & 0x7F807F80u, u[s][NG * k + NG - 1] & 0x7F807F80u) : u[s][k] & 0x7F807F80u;
        own[0][k] = pf_need<false>(some[0][k]);
        own[1][k] = pf_need<true>(some[1][k]);
      }
      reduce();
      if (max(top[0], top[1]) >= 100) [[unlikely]] {  // words that are not finite may be among them, and are passed over
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          own[0][k] = max(pf_finite_need<false>(u[0][NG * k]), pf_finite_need<false>(u[0][NG * k + NG - 1]));
          own[1][k] = max(pf_finite_need<true>(u[1][NG * k]), pf_finite_need<true>(u[1][NG * k + NG - 1]));
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (own[s][k] == PF_NO_NEED) some[s][k] = 0u;
        }
        reduce();
      }
      const int f[2] = {pf_power(top[0]), pf_power(top[1])};
      const bool uneven = bad != 0u || low[0] < top[0] - PF_EVEN || low[1] < top[1] - PF_EVEN;
      if (uneven) [[unlikely]] {  // the smaller tokens' words take their own powers here, so that widening knows one for all
        const int col = 32 * (rec >> 1) + 8 * (lane & 3) + 4 * (rec & 1) + 2 * ((lane >> 2) & 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t *to = reinterpret_cast<uint32_t *>(smem + C::RING + rs * C::RAW + rec * C::PITCH + (s ? Rec::VW : Rec::KW)) + (lane & 7) * (2 * NG);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int by = there && some[s][k] != 0u ? min(max(min(-own[s][k], 100) - f[s], 0), 126) : 0;
            (s ? cs.v_by : cs.k_by)[tile & 15][col + k] = s ? static_cast<float>(-f[1] - by) : pow2i(-by);
#pragma unroll
            for (int w = 0; w < NG; ++w)
              if (by > 0) to[NG * k + w] = pf_word_by(to[NG * k + w], by);
          }
        }
        fence_proxy_async_smem();  // before the ring's next copy
        __syncwarp();
      }
      if (lane == 0) {
        cs.info[tile & 15] = {f[0], f[1], (bad & 1u) | ((bad >> 7) & 2u) | ((bad >> 14) & 4u) | ((bad >> 21) & 8u), uneven ? 1u : 0u};
        mbar_arrive(&cs.info_full[rs]);
      }
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && (cs.abort | cs.no_abort)) record_status(a.status, -5 /* SPARGE_ERR_DEVICE_TIMEOUT */);
  if (warp == PF_PROD) tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------------------------------------
// Every row's shares - of the prefix from each CTA that held some of it, of the sequence's own tokens from those of the
// cache attention - weighted by 2^(m - M) and divided by the weighted sum.  W warps per row, each loads eight shares at a time: loads of a
// microsecond each bound it, so a row of many shares wants many of them in flight.
// --------------------------------------------------------------------------------------------
struct PfCombineArgs {
  SplitArgs own;
  const float *part_o, *part_ml;
  const int32_t *lens;
  int64_t total;  // tiles of all items
  int tiles, ctas, groups, R, rt, width, rec_shift, prefix;
};

constexpr int PC_THREADS = 256, PC_FEW = 8;
template <int D, int W>
__global__ void __launch_bounds__(PC_THREADS, 4) prefix_combine_kernel(const PfCombineArgs a) {
  constexpr int NL = D / 4, ROWS = PC_THREADS / 32 / W;
  __shared__ float4 part[W > 1 ? PC_THREADS : 1];
  __shared__ float2 part_ml[PC_THREADS / 32];
  start_after_earlier();
  const int lane = threadIdx.x & 31, sub = (threadIdx.x >> 5) % W;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * ROWS + (threadIdx.x >> 5) / W;
  const int rows = a.own.rows;                      // of a sequence and KV head
  const int64_t per = static_cast<int64_t>(a.own.B) * rows;
  const int kvh = static_cast<int>(i / per);
  const bool mine = kvh < a.own.Hkv;
  if (!mine && W == 1) return;
  const int r = mine ? static_cast<int>(i - kvh * per) : 0, b = r / rows, rr = r % rows;
  const int64_t cap = static_cast<int64_t>(a.width) << (a.rec_shift + 4);
  const int len = max(a.lens[b] > cap ? static_cast<int>(cap) : a.lens[b], 0);
  const int tile = 8 * a.rt, oitem = (b * a.own.Hkv + kvh) * a.own.ntile + rr / tile;
  int n_own = 0, n = 0, prow = 0;
  int64_t own0 = 0, slot0 = 0;
  if (mine && len > 0) {
    const int2 ends = a.own.ends[oitem];
    n = n_own = ends.y - ends.x + 1;
    own0 = (static_cast<int64_t>(ends.x) + oitem) * tile + rr % tile;
  }
  if (mine && len > 0 && len - a.own.Nq >= a.prefix) {
    const int item = kvh * a.groups + r / (128 * a.R);
    // CTA c holds tiles total c / ctas .. total (c + 1) / ctas - 1
    const int64_t t0 = static_cast<int64_t>(item) * a.tiles, t1 = t0 + a.tiles - 1;
    const int c0 = static_cast<int>(((t0 + 1) * a.ctas - 1) / a.total), c1 = static_cast<int>(((t1 + 1) * a.ctas - 1) / a.total);
    slot0 = static_cast<int64_t>(c0) + item;
    prow = r % (128 * a.R);
    n += (c1 - c0 + 1) * (a.R == 2 ? 1 : 2);
  }
  // share k of the prefix: a slot's row or, with one row tile, the rows of its two streams
  auto at = [&](int k, int &in) {
    in = a.R == 2 ? prow : (k & 1) * 128 + prow;
    return slot0 + (a.R == 2 ? k : k >> 1);
  };
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = sub * PC_FEW; w < n; w += W * PC_FEW) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < PC_FEW && w + lane < n) {
      const int k = w + lane;
      int in;
      const int64_t slot = at(k - n_own, in);
      ml = k < n_own ? *reinterpret_cast<const float2 *>(a.own.part_ml + 2 * (own0 + static_cast<int64_t>(k) * tile))
                     : *reinterpret_cast<const float2 *>(a.part_ml + 2 * (slot * PF_ROWS + in));
    }
    float4 v[PC_FEW];
#pragma unroll
    for (int u = 0; u < PC_FEW; ++u) {
      const int k = w + u;
      int in;
      const int64_t slot = at(k - n_own, in);
      if (k < n && lane < NL)
        v[u] = k < n_own ? *reinterpret_cast<const float4 *>(a.own.part_o + (own0 + static_cast<int64_t>(k) * tile) * D + 4 * lane)
                         : *reinterpret_cast<const float4 *>(a.part_o + ((slot * (D / 32) + lane / 8) * PF_ROWS + in) * 32 +
                                                             4 * ((lane & 7) ^ (in & 7)));
    }
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
    for (int u = 0; u < PC_FEW; ++u) {
      const float fu = __shfl_sync(0xffffffffu, f, u);
      if (w + u < n && lane < NL) add_share(s, fu, v[u]);
    }
    o = s;
  }
  if constexpr (W > 1) {  // the first warp of a row puts its warps' sums together
    part[threadIdx.x] = o;
    if (lane == 0) part_ml[threadIdx.x >> 5] = make_float2(M, L);
    __syncthreads();
    if (sub > 0 || !mine) return;
    float m = -INFINITY;
#pragma unroll
    for (int k = 0; k < W; ++k) m = fmaxf(m, part_ml[(threadIdx.x >> 5) + k].x);
    L = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float2 ml = part_ml[(threadIdx.x >> 5) + k];
      const float f = share_weight(ml.x, ml.y, m);
      if (f != 0.f) L = fmaf(f, ml.y, L);
      add_share(o, f, part[threadIdx.x + 32 * k]);
    }
  }
  if (lane < NL) put_row(a.own.row(b, kvh, rr) + 4 * lane, o, L == 0.f ? 0.f : 1.f / L);
}

// Row tiles of a CTA, groups of rows and CTAs of a call.
struct PfPlan {
  int R, groups, ctas;
  int64_t items;
};
PfPlan plan(int64_t rows, int64_t Hkv, int64_t tiles) {
  PfPlan p;
  p.R = rows > 128 ? 2 : 1;
  p.groups = static_cast<int>((rows + 128 * p.R - 1) / (128 * p.R));
  p.items = Hkv * p.groups;
  const int64_t total = p.items * tiles, most = total / 2 > 1 ? total / 2 : 1;
  p.ctas = static_cast<int>(most < CA_SMS ? most : CA_SMS);
  return p;
}

// What one of the paths takes beyond what both do, in us, fitted to 115 pairs of times: 2 to 64 sequences with 1K to 64K shared tokens, 8
// to 64 query heads over 1 to 8 KV heads, 1 to 4 queries (d = 128, 32 over 8 heads, alone and shared: 4 sequences over 64K tokens
// 57 and 59, 8 over 64K 103 and 60, 8 over 16K 34 and 30, 16 over 4K 23.1 and 23.0, 2 over 4K 12 and 20).  The rule takes the slower
// path in two of the pairs, by 8 and 15 %.
double alone_us(int64_t B, int64_t rows, int64_t Hkv, int64_t d, int64_t recs) {  // the records of every sequence, from L2 for the most part
  const double mb = 18e-6 * static_cast<double>(B) * Hkv * d * recs;
  return mb * (rows <= 8 ? 0.165 : 0.24 * ((rows + 15) / 16));
}
double shared_us(const PfPlan &p, int64_t rows, int64_t Hkv, int64_t d, int64_t tiles) {  // two launches more, tiles, rows put together
  const double tile = d == 128 ? (p.R == 2 ? 1.0 : 0.8) : (p.R == 2 ? 0.85 : 0.55);
  return 9. + tile * static_cast<double>(p.items) * tiles / CA_SMS + 0.0022 * static_cast<double>(rows) * Hkv;
}

template <int D, int R>
cudaError_t launch_t(const PrefixArgs &a, int ctas, cudaStream_t st) {
  static std::atomic<unsigned long long> smem_set{0};
  if (cudaError_t e = set_smem_limit_once(prefix_attn_kernel<D, R>, static_cast<int>(PfCfg<D, R>::SMEM), smem_set); e != cudaSuccess)
    return e;
  return launch_dependent(prefix_attn_kernel<D, R>, dim3(static_cast<unsigned>(ctas)), PF_THREADS, PfCfg<D, R>::SMEM, st, a);
}

}  // namespace

// rows: B G Nq of a KV head
size_t prefix_ws_bytes(int64_t rows, int64_t Hkv, int64_t d) {
  const PfPlan p = plan(rows, Hkv, INT_MAX);
  const size_t slots = static_cast<size_t>(p.items + CA_SMS);
  return ((slots * PF_ROWS * d * 4 + 255) & ~size_t(255)) + ((slots * PF_ROWS * 8 + 255) & ~size_t(255));
}

// Whether B sequences of `rows` query rows per KV head gain from a prefix of `recs` records being attended once for all of them.
bool prefix_shared(int64_t B, int64_t rows, int64_t Hkv, int64_t d, int64_t recs) {
  const int64_t tiles = (recs + 3) / 4;
  return alone_us(B, rows, Hkv, d, recs) > shared_us(plan(B * rows, Hkv, tiles), B * rows, Hkv, d, tiles);
}

cudaError_t launch_prefix_attn(const PrefixAttn &l, const SplitArgs &own, cudaStream_t st) {
  PrefixArgs a;
  a.q = static_cast<const __nv_bfloat16 *>(l.q);
  a.q_sb = l.q_sb; a.q_sh = l.q_sh; a.q_sn = l.q_sn;
  a.pool = l.pool;
  a.pages = l.pages;
  a.n_pages = l.n_pages;
  a.rec_shift = l.rec_shift;
  a.recs = l.prefix / C4_TOKENS;
  a.tiles = (a.recs + 3) / 4;
  a.Hkv = own.Hkv; a.G = own.G; a.Nq = own.Nq;
  a.rows = own.B * own.rows;
  const PfPlan p = plan(a.rows, a.Hkv, a.tiles);
  a.groups = p.groups;
  a.scale_log2 = l.scale_log2;
  a.part_o = static_cast<float *>(l.ws);
  a.part_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(l.ws) +
                                        ((static_cast<size_t>(p.items + CA_SMS) * PF_ROWS * l.d * 4 + 255) & ~size_t(255)));
  a.status = l.status;
  if (l.d == 128) return p.R == 2 ? launch_t<128, 2>(a, p.ctas, st) : launch_t<128, 1>(a, p.ctas, st);
  return p.R == 2 ? launch_t<64, 2>(a, p.ctas, st) : launch_t<64, 1>(a, p.ctas, st);
}

cudaError_t launch_prefix_combine(const PrefixAttn &l, const SplitArgs &own, cudaStream_t st) {
  PfCombineArgs a;
  a.own = own;
  const int64_t rows = static_cast<int64_t>(own.B) * own.rows;
  a.tiles = (l.prefix / C4_TOKENS + 3) / 4;
  const PfPlan p = plan(rows, own.Hkv, a.tiles);
  a.part_o = static_cast<const float *>(l.ws);
  a.part_ml = reinterpret_cast<const float *>(static_cast<const uint8_t *>(l.ws) +
                                              ((static_cast<size_t>(p.items + CA_SMS) * PF_ROWS * l.d * 4 + 255) & ~size_t(255)));
  a.lens = l.lens;
  a.total = p.items * a.tiles;
  a.ctas = p.ctas;
  a.groups = p.groups;
  a.R = p.R;
  a.rt = row_tile(own.rows);
  a.width = l.width;
  a.rec_shift = l.rec_shift;
  a.prefix = l.prefix;
  // Warps of a row: by its shares of the prefix and the rows in all.  Measured with one, two and eight (d = 128): 256 rows of 153 shares 33,
  // 25 and 16 us, 608 of 52 23, 17 and 11; 1024 of 39 20, 16 and 15 (two waves of blocks with eight, and ahead all the same); 1200 of 20 17, 13.5 and
  // 14.4; 2400 of 17 17.5, 14.6 and 23, with 2432 of two warps resident at once; 2800 of 15 16.1, 16.3 and 25; 3000 of 12 13.7, 14.5 and 24.
  const int64_t shares = ((p.ctas + p.items - 1) / p.items + 1) * (p.R == 2 ? 1 : 2), all = rows * own.Hkv;
  const int W = shares <= 12 || all > 16 * CA_SMS ? 1 : shares <= 32 || all > 1024 ? 2 : 8, per = PC_THREADS / 32 / W;
  const dim3 grid(static_cast<unsigned>((rows * own.Hkv + per - 1) / per));
  auto run = [&](auto d) {
    constexpr int D = decltype(d)::value;
    return W == 1 ? launch_dependent(prefix_combine_kernel<D, 1>, grid, PC_THREADS, 0, st, a)
         : W == 2 ? launch_dependent(prefix_combine_kernel<D, 2>, grid, PC_THREADS, 0, st, a)
                  : launch_dependent(prefix_combine_kernel<D, 8>, grid, PC_THREADS, 0, st, a);
  };
  return l.d == 128 ? run(std::integral_constant<int, 128>()) : run(std::integral_constant<int, 64>());
}

}  // namespace sparge
