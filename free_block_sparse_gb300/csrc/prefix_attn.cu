// Attention of a whole batch over a prefix that its sequences share, from the paged 4-bit cache, on tcgen05 tensor cores.
#include <climits>
#include <cmath>

#include <cuda_fp16.h>

#include "cache4.cuh"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"
#include "rowsplit.cuh"

namespace sparge {
namespace {

// Warps: softmax (4 per stream, a row a thread), widening (two groups of 4 that take turns), products (one per stream), loads.
constexpr int PF_SOFT = 8, PF_WIDE = 8, PF_PROD = PF_SOFT + PF_WIDE, PF_LOAD = PF_PROD + 2;
constexpr int PF_THREADS = (PF_LOAD + 1) * 32;
constexpr int PF_ROWS = 256;             // rows of a slot: two streams of 128
constexpr float PF_RESCALE = 8.f;
constexpr float PF_TOP = 15.f;           // P' stays below 2^15, within f16

struct PrefixArgs {
  const __nv_bfloat16 *q;
  int64_t q_sb, q_sh, q_sn;
  const uint8_t *pool;
  const int32_t *pages;
  int64_t n_pages;
  int rec_shift, recs, tiles;       // records of a page (1 << rec_shift), of the prefix; 64-token tiles
  int Hkv, G, Nq, rows, groups;     // rows of a KV head: B G Nq; groups of them: items of a KV head
  float scale_log2;
  float *part_o, *part_ml;          // [CTA + item][256][D], [CTA + item][256] (reference, sum)
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
  static constexpr uint32_t K = 0, V = K + NS * TILE, Q = V + NS * TILE, RING = Q + (QSMEM ? 2 * 128 * D * 2 : 0);
  static constexpr uint32_t TABK = RING + RS * RAW, TABV = TABK + 4 * 64 * 16, CTRL = TABV + 4 * 512;
  static constexpr uint32_t SMEM = CTRL + 1024;
  // TMEM columns
  static constexpr uint32_t O = 0, S = 2 * D, P = S + 128, QC = P + 64, QCOLS = D / 2;
  static_assert(QC + (QSMEM ? 0 : R) * QCOLS <= 512, "TMEM");
  static_assert(SMEM <= 227 * 1024, "shared memory");
};
struct PfInfo {  // of a widened tile: K = K' k_unit, V = V' 2^g; bit r of missing: record r is not there
  float k_unit;
  int g;
  uint32_t missing;
};
struct PfCtrl {
  uint64_t raw_full[8], raw_free[8], k_full[4], k_free[4], v_full[4], v_free[4];
  uint64_t q_full[2], q_free, s_full[2], s_free[2], p_full[2], pv_done[2], drained[2];
  PfInfo info[8];  // (tile % 8: K's stage is free again before the softmax has read what goes with it)
  int need[4][4];  // of a tile (tile % 4): K by warps 0 and 1 of its group, V by 2 and 3
  uint8_t bad[8][4];
  uint32_t tmem;
  int abort, no_abort;
};
static_assert(sizeof(PfCtrl) <= 1024, "control block");

__device__ __forceinline__ void pf_bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ float pf_pow2(int e) { return __int_as_float((e + 127) << 23); }  // e in -126..127
__device__ __forceinline__ int pf_exponent(float x) { return static_cast<int>((__float_as_uint(x) >> 23) & 0xFFu) - 127; }
__device__ __forceinline__ uint32_t pf_half2(float lo, float hi) {  // an infinity or a NaN stays one
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
__device__ __forceinline__ void pf_ld_wait_for(uint32_t (&r)[32], float &m) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+f"(m)
               :
               : "memory");
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
  if (threadIdx.x == 0) {
    for (int s = 0; s < RS; ++s) {
      mbar_init(&cs.raw_full[s], 4);
      mbar_init(&cs.raw_free[s], 4);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&cs.k_full[s], 4);
      mbar_init(&cs.k_free[s], R);
      mbar_init(&cs.v_full[s], 4);
      mbar_init(&cs.v_free[s], R);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&cs.q_full[t], 4);
      mbar_init(&cs.s_full[t], 1);
      mbar_init(&cs.s_free[t], 4);
      mbar_init(&cs.p_full[t], 4);
      mbar_init(&cs.pv_done[t], 1);
    }
    mbar_init(&cs.drained[0], 1);
    mbar_init(&cs.drained[1], 1);
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
    uint32_t done = 0, piece = 0;  // jobs of this stream so far, pieces
    bool ok = true;
    for (; ok && share.next(a, item, tile0, n); ++piece) {
      // ---- the row's queries: f16, times a power of two that takes its maximum to [2^14, 2^15) ----
      const int kvh = item / a.groups, r = (item % a.groups) * (128 * R) + (R == 2 ? t * 128 : 0) + row;
      float rm = 0.f;  // 2^(e - 14) scale: what a product of the scaled row counts
      {
        const int b = r / (a.G * a.Nq), rr = r % (a.G * a.Nq);
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + b * a.q_sb + (kvh * a.G + rr / a.Nq) * a.q_sh +
                                                           static_cast<int64_t>(rr % a.Nq) * a.q_sn);
        float mx = 0.f;
#pragma unroll 1
        for (int i = 0; i < D / 8; i += 4) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = r < a.rows ? src[i + k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int x = 0; x < 4; ++x) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(u[x])), fabsf(bf16hi(u[x]))));
          }
        }
        const int e = min(max(pf_exponent(mx), -100), 116);
        const float f = pf_pow2(14 - e);
        rm = a.scale_log2 * pf_pow2(e - 14);
        // in each 8 channels the order 0 4 1 5 2 6 3 7, in which the codes' words give them
        if (R == 2 || t == 0) {
          // the other stream's products with the rows before these have been made (this one's have: its O is complete)
          if (R == 1 && piece > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&cs.q_free, (piece - 1) & 1, abort, a.status));
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll 1
          for (int i = 0; i < D / 8; i += 4) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = r < a.rows ? src[i + k] : make_uint4(0u, 0u, 0u, 0u);
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint4 u = v[k];
              w[4 * k] = pf_half2(bf16lo(u.x) * f, bf16lo(u.z) * f);
              w[4 * k + 1] = pf_half2(bf16hi(u.x) * f, bf16hi(u.z) * f);
              w[4 * k + 2] = pf_half2(bf16lo(u.y) * f, bf16lo(u.w) * f);
              w[4 * k + 3] = pf_half2(bf16hi(u.y) * f, bf16hi(u.w) * f);
            }
            if (C::QSMEM) {
              const uint32_t at = smem_u32(smem) + C::Q + t * (128 * D * 2) + (i / 8) * 16384 + row * 128;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pf_sts128(at + ((((i & 7) + k) ^ (row & 7)) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            } else {
              tmem_st16(tl + C::QC + (R == 2 ? t * C::QCOLS : 0) + 4 * i, w);
            }
          }
          tmem_st_wait();
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&cs.q_full[t]);
        }
      }
      float m_ref = -INFINITY, l = 0.f;
      int G = 0;  // O counts 2^G
      const bool live = r - lane < a.rows;  // a warp past the last row takes part in the waits alone
      // columns 8 c + 4 r + i of a half are tokens of its record r: those that are not there are hidden; the others' maximum
      auto hide = [](uint32_t (&x)[32], uint32_t gone) {
        float m = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          if ((gone >> ((k >> 2) & 1)) & 1u) x[k] = 0xFF800000u;
          m = fmaxf(m, __uint_as_float(x[k]));
        }
        return m;
      };
      const int jobs = R == 2 ? n : (n - t + 1) / 2;
      for (int j = 0; j < jobs; ++j, ++done) {
        const uint32_t tile = tc + (R == 2 ? j : 2 * j + t), st = tile % NS;
        ok = mbar_wait(&cs.v_full[st], (tile / NS) & 1, abort, a.status) && mbar_wait(&cs.s_full[t], done & 1, abort, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        // 32 columns are held at a time; the others are read for their maximum now and once more for their turn
        uint32_t v[32];
        float mx = -INFINITY, m1;
        const float mult = rm * cs.info[tile & 7].k_unit;
        const int g = cs.info[tile & 7].g;
        const uint32_t missing = cs.info[tile & 7].missing;
        if (live) {
          tmem_ld32_max(sc + 32, v, m1);
          pf_ld_wait_for(v, m1);
          if (missing) m1 = hide(v, missing >> 2);
          tmem_ld32_max(sc, v, mx);
          pf_ld_wait_for(v, mx);
          if (missing) mx = hide(v, missing);
          mx = fmaxf(mx, m1) * mult;
        }
        if (j > 0) {  // the product before this one has read its P and added to O
          ok = __all_sync(0xffffffffu, mbar_wait(&cs.pv_done[t], (done - 1) & 1, abort, a.status));
          if (!ok) break;
          tc_fence_after();
        }
        if (live) {
          if (m_ref == -INFINITY) G = g;
          const bool resc = mx > m_ref + PF_RESCALE || mx - m_ref + static_cast<float>(g - G) > PF_TOP;
          if (__any_sync(0xffffffffu, resc)) {
            float f = 1.f;
            if (resc) {
              const float to = fmaxf(m_ref, mx), al = fast_exp2(m_ref - to);
              // O's unit follows: this tile's, or what the sums before need
              const int Gn = m_ref == -INFINITY ? g : max(g, __float2int_ru(fmaxf(static_cast<float>(G) + (m_ref - to), -1000.f)));
              f = al * pf_pow2(min(max(G - Gn, -126), 127));
              l *= al;
              m_ref = to;
              G = Gn;
            }
            if (j > 0) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_ld16(oc + 16 * q, o);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tmem_st16(oc + 16 * q, o);
              }
            }
          }
          // P' = 2^(x - m_ref + g - G); a row whose reference is still -inf has only hidden columns (or NaN)
          const int up = G - g;
          const float nref = m_ref == -INFINITY ? 0.f : -m_ref;
          const bool tiny = __any_sync(0xffffffffu, up > 60);  // V of this tile beside what O holds: the sum of P goes by itself
          const float2 m2 = make_float2(mult, mult), nr2 = make_float2(nref - static_cast<float>(up), nref - static_cast<float>(up));
          float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (h == 1) {
              tmem_ld32_max(sc + 32, v, m1);
              pf_ld_wait_for(v, m1);
              if (missing) hide(v, missing >> 2);
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&cs.s_free[t]);
            }
            if (tiny) {
              float sum = 0.f;
#pragma unroll
              for (int k = 0; k < 32; ++k) sum += fast_exp2(fmaf(__uint_as_float(v[k]), mult, nref));
              l += sum;
            }
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float2 e2 = ffma2(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), m2, nr2);
              const float2 p2 = make_float2(fast_exp2(e2.x), fast_exp2(e2.y));
              rs[k & 1] = fadd2(rs[k & 1], p2);
              pk[k] = pack_f16x2(p2.x, p2.y);
            }
            tmem_st16(pc + 16 * h, pk);
          }
          const float2 sum = fadd2(rs[0], rs[1]);
          if (!tiny) l = fmaf(sum.x + sum.y, pf_pow2(max(up, -126)), l);
          tmem_st_wait();
        } else if (lane == 0) {
          mbar_arrive(&cs.s_free[t]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cs.p_full[t]);
      }
      if (!ok) break;
      // ---- the piece's end: O (times 2^G), the reference and the sum ----
      if (jobs > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&cs.pv_done[t], (done - 1) & 1, abort, a.status));
        if (!ok) break;
        tc_fence_after();
      }
      const int64_t at = (static_cast<int64_t>(blockIdx.x) + item) * PF_ROWS + t * 128 + row;
      if (r < a.rows) *reinterpret_cast<float2 *>(a.part_ml + 2 * at) = make_float2(m_ref, l);
      if (jobs > 0 && live) {
        const float back = pf_pow2(min(max(G, -126), 127));
        float *to = a.part_o + at * D;
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t o[16];
          tmem_ld16(oc + 16 * q, o);
          tmem_ld_wait();
          if (r < a.rows) {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<float4 *>(to + 16 * q + k) =
                  make_float4(__uint_as_float(o[k]) * back, __uint_as_float(o[k + 1]) * back, __uint_as_float(o[k + 2]) * back,
                              __uint_as_float(o[k + 3]) * back);
          }
        }
        tc_fence_before();
      }
      tc += n;
    }
  } else if (warp < PF_PROD) {
    // ------------------------------------ widening: codes to f16 tiles ------------------------------------
    // A tile's power of two for K and the one for V follow from the words of all its tokens.  The words of the group's next tiles are
    // looked at, and the next table is made, around the widening of the one in front, so that one barrier a tile is enough.
    const int w4 = warp & 3, tid = w4 * 32 + lane, group = (warp - PF_SOFT) >> 2;
    const int side = tid >> 6, rec = (tid >> 4) & 3, tk = tid & 15;  // this thread's token and side in words and tables
    const uint32_t base = smem_u32(smem);
    float s[NG], m[NG];  // its words of the tile behind
    bool ok = true;
    auto words = [&](uint32_t tile) {
      const uint32_t rs = tile % RS;
      // (a warp whose wait gives up goes on to the next barrier, where all four leave together)
      ok = __all_sync(0xffffffffu, mbar_wait(&cs.raw_full[rs], (tile / RS) & 1, abort, a.status)) && ok;
      const bool gone = cs.bad[rs][rec] != 0;
      const uint8_t *at = smem + C::RING + rs * C::RAW + rec * C::PITCH + (side ? Rec::VW : Rec::KW) + tk * NG * 4;
      int need = -200;  // f <= -need: code * 2^-24 s 2^(f + 24) is within f16, and so is the value
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t word = *reinterpret_cast<const uint32_t *>(at + 4 * g);
        s[g] = gone ? 0.f : bf16lo(word);
        m[g] = gone ? 0.f : bf16hi(word);
        if (fabsf(s[g]) < INFINITY && fabsf(m[g]) < INFINITY)
          need = max(need, max(pf_exponent(s[g]) + 9, max(pf_exponent(m[g]), pf_exponent(fmaf(15.f, s[g], m[g]))) - 14));
      }
      need = __reduce_max_sync(0xffffffffu, need);
      if (lane == 0) cs.need[tile & 3][w4] = need;
    };
    int fk = 0, fv = 0;
    auto table = [&](uint32_t tile) {
      const int *need = cs.need[tile & 3];
      fk = min(max(-max(need[0], need[1]), -126), 100);
      fv = min(max(-max(need[2], need[3]), -126), 100);
      const int f = side ? fv : fk;
      const float fs = pf_pow2(f + 24), fm = pf_pow2(f);
      const int pos = 32 * (rec >> 1) + 8 * ((tk & 7) >> 1) + 4 * (rec & 1) + 2 * (tk >> 3) + (tk & 1);
      uint8_t *tk_ = smem + C::TABK + (tile & 3) * 1024, *tv = smem + C::TABV + (tile & 3) * 512;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t ss = pf_half2(s[g] * fs, s[g] * fs), mm = pf_half2(m[g] * fm, m[g] * fm);
        if (side) {
          *reinterpret_cast<uint16_t *>(tv + (g * 64 + pos) * 2) = static_cast<uint16_t>(ss);
          *reinterpret_cast<uint16_t *>(tv + 256 + (g * 64 + pos) * 2) = static_cast<uint16_t>(mm);
        } else {
          *reinterpret_cast<uint2 *>(tk_ + pos * 16 + g * 8) = make_uint2(ss, mm);
        }
      }
    };
    auto all_ok = [&]() { return ok = !bar_red_or(1 + group, 128, !ok); };
    const uint32_t total = static_cast<uint32_t>(share.end - share.at);  // tiles of all the CTA's pieces
    const uint32_t tile0 = group;  // the group takes every second tile
    if (tile0 < total) {
      words(tile0);
      if (all_ok()) {
        table(tile0);
        if (tile0 + 2 < total) words(tile0 + 2);
      }
    }
    for (uint32_t tile = tile0; tile < total; tile += 2) {
      {
        const uint32_t rs = tile % RS, st = tile % NS;
        if (tile >= NS) ok = __all_sync(0xffffffffu, mbar_wait(&cs.k_free[st], (tile / NS - 1) & 1, abort, a.status)) && ok;
        const int k_is = fk, v_is = fv;
        if (!all_ok()) break;  // this tile's table and the next one's powers are there
        const uint8_t *raw = smem + C::RING + rs * C::RAW;
        const uint8_t *tabk = smem + C::TABK + (tile & 3) * 1024, *tabv = smem + C::TABV + (tile & 3) * 512;
        if (tid == 0) {
          PfInfo &i = cs.info[tile & 7];
          i.k_unit = pf_pow2(-k_is);
          i.g = -v_is;
          i.missing = cs.bad[rs][0] | (cs.bad[rs][1] << 1) | (cs.bad[rs][2] << 2) | (cs.bad[rs][3] << 3);
        }
        if (tile + 2 < total) table(tile + 2);
        // ---- K: a lane takes the codes of 8-channel piece c of every 32 channels of a token ----
        {
          const int c = lane & 3, r = (lane >> 2) & 1;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int task = w4 + 4 * k, pr = task & 1, t = (task >> 1) * 4 + (lane >> 3);
            const int pos = 32 * pr + 8 * ((t & 7) >> 1) + 4 * r + 2 * (t >> 3) + (t & 1);
            const uint8_t *src = raw + (2 * pr + r) * C::PITCH + Rec::K + t * (D / 2) + c * (D / 8);
            uint32_t code[2 * NG];
            uint2 sm[NG];
            if constexpr (D == 128) {
              const uint4 u = *reinterpret_cast<const uint4 *>(src), x = *reinterpret_cast<const uint4 *>(tabk + pos * 16);
              code[0] = u.x; code[1] = u.y; code[2] = u.z; code[3] = u.w;
              sm[0] = make_uint2(x.x, x.y);
              sm[1] = make_uint2(x.z, x.w);
            } else {
              const uint2 u = *reinterpret_cast<const uint2 *>(src);
              code[0] = u.x; code[1] = u.y;
              sm[0] = *reinterpret_cast<const uint2 *>(tabk + pos * 16);
            }
            const uint32_t to = base + C::K + st * C::TILE + pos * 128;
#pragma unroll
            for (int w = 0; w < 2 * NG; ++w) {
              const uint32_t lo = sm[w / 2].x, hi = pf_sixteenth2(lo), mm = sm[w / 2].y, u = code[w], u8 = u >> 8;
              pf_sts128(to + (w >> 1) * 8192 + (((4 * (w & 1) + c) ^ (pos & 7)) << 4), pf_hfma2(u & 0x000F000Fu, lo, mm),
                        pf_hfma2(u & 0x00F000F0u, hi, mm), pf_hfma2(u8 & 0x000F000Fu, lo, mm), pf_hfma2(u8 & 0x00F000F0u, hi, mm));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cs.k_full[st]);
        // (a warp whose wait gives up leaves its V as it is and goes on to the next barrier)
        if (tile >= NS) ok = __all_sync(0xffffffffu, mbar_wait(&cs.v_free[st], (tile / NS - 1) & 1, abort, a.status)) && ok;
        // ---- V, transposed: lane 4 g + c holds channels g and g + 8 of every 16 for tokens 2c, 2c + 1, 2c + 8, 2c + 9 of two records ----
        {
          const int g = lane >> 2, c = lane & 3;
          constexpr int NU = 2 * NG;  // words of a warp: d = 128: a half of the channels and a pair of records; d = 64: a quarter
          const int part = D == 128 ? w4 >> 1 : 0, u0 = D == 128 ? 0 : 2 * (w4 >> 1), pr = (w4 & 1) ^ (g & 1);
          const uint4 s4 = *reinterpret_cast<const uint4 *>(tabv + (part * 64 + 32 * pr + 8 * c) * 2);
          const uint4 m4 = *reinterpret_cast<const uint4 *>(tabv + 256 + (part * 64 + 32 * pr + 8 * c) * 2);
          const uint32_t ss[4] = {s4.x, s4.y, s4.z, s4.w}, mm[4] = {m4.x, m4.y, m4.z, m4.w};
          uint32_t sh[4], code[2][NU];
#pragma unroll
          for (int k = 0; k < 4; ++k) sh[k] = pf_sixteenth2(ss[k]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint8_t *src = raw + (2 * pr + r) * C::PITCH + Rec::V + part * 512 + 16 * lane + 4 * u0;
            if constexpr (NU == 4) {
              const uint4 u = *reinterpret_cast<const uint4 *>(src);
              code[r][0] = u.x; code[r][1] = u.y; code[r][2] = u.z; code[r][3] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2 *>(src);
              code[r][0] = u.x; code[r][1] = u.y;
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
          mbar_arrive(&cs.v_full[st]);
          mbar_arrive(&cs.raw_free[rs]);
        }
        if (tile + 4 < total) words(tile + 4);
      }
    }
  } else if (warp < PF_LOAD) {
    // ------------------------------------ products of one stream ------------------------------------
    // (a thread for each stream: waits, fences and issue of a job take it about as long as the tensor unit takes the products)
    const int t = warp - PF_PROD;
    if (lane == 0) {
      const uint64_t dk = smem_desc_sw128(smem_u32(smem + C::K), 16, 1024), dv = smem_desc_sw128(smem_u32(smem + C::V), 16, 1024);
      const uint64_t dq = smem_desc_sw128(smem_u32(smem + C::Q) + (C::QSMEM ? t * 128 * D * 2 : 0), 16, 1024);
      const uint32_t sc = tmem + C::S + t * 64, oc = tmem + C::O + t * D, pc = tmem + C::P + t * 32;
      const uint32_t qc = tmem + C::QC + (R == 2 ? t * C::QCOLS : 0);
      uint32_t done = 0, piece = 0;  // jobs so far, pieces
      bool ok = true;
      for (; ok && share.next(a, item, tile0, n); ++piece) {
        const int jobs = R == 2 ? n : (n - t + 1) / 2;
        ok = mbar_wait(&cs.q_full[R == 2 ? t : 0], piece & 1, abort, a.status);
        for (int j = 0; ok && j <= jobs; ++j) {
          if (j < jobs) {  // scores of job j, once the softmax has read those before
            const uint32_t tile = tc + (R == 2 ? j : 2 * j + t), st = tile % NS;
            ok = mbar_wait(&cs.k_full[st], (tile / NS) & 1, abort, a.status) &&
                 (done == 0 || mbar_wait(&cs.s_free[t], (done - 1) & 1, abort, a.status));
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = dk + st * (C::TILE >> 4);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              if (C::QSMEM)
                mma_bf16_ss(sc, dq + (s >> 2) * (16384 >> 4) + (s & 3) * 2, b + (s >> 2) * (8192 >> 4) + (s & 3) * 2, IDESC_S, s > 0 ? 1u : 0u);
              else
                mma_bf16_ts(sc, qc + s * 8, b + (s >> 2) * (8192 >> 4) + (s & 3) * 2, IDESC_S, s > 0 ? 1u : 0u);
            }
            mma_commit(&cs.s_full[t]);
            mma_commit(&cs.k_free[st]);
            if (R == 1 && t == 1 && j == jobs - 1) mma_commit(&cs.q_free);
            ++done;
          }
          if (j > 0) {  // P V of job j - 1
            const uint32_t tile = tc + (R == 2 ? j - 1 : 2 * (j - 1) + t), st = tile % NS, nth = done - (j < jobs ? 2 : 1);
            ok = mbar_wait(&cs.v_full[st], (tile / NS) & 1, abort, a.status) && mbar_wait(&cs.p_full[t], nth & 1, abort, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint64_t b = dv + st * (C::TILE >> 4);
#pragma unroll
            for (int s = 0; s < 4; ++s) mma_bf16_ts(oc, pc + s * 8, b + s * 2, IDESC_PV, s > 0 || j > 1 ? 1u : 0u);
            mma_commit(&cs.pv_done[t]);
            mma_commit(&cs.v_free[st]);
          }
        }
        if (R == 1 && t == 1 && jobs == 0) mma_commit(&cs.q_free);
        tc += n;
      }
      if (!ok) {  // products in flight end before the CTA gives its TMEM back
        mma_commit(&cs.drained[t]);
        mbar_wait(&cs.drained[t], 0, &cs.no_abort, a.status);
      }
    }
    __syncwarp();
  } else {
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
        if (tile >= RS) ok = mbar_wait(&cs.raw_free[rs], (tile / RS - 1) & 1, abort, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane / 4 == j - j0) {
          uint64_t *bar = &cs.raw_full[rs];
          cs.bad[rs][lane & 3] = src == nullptr;
          if (src != nullptr) {
            mbar_arrive_expect_tx(bar, Rec::BYTES);
            pf_bulk_load(smem + C::RING + rs * C::RAW + (lane & 3) * C::PITCH, src, Rec::BYTES, bar);
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == PF_PROD) tmem_dealloc(tmem, 512);
}

// --------------------------------------------------------------------------------------------
// Every row's shares - of the prefix from each CTA that held some of it, of the sequence's own tokens from those of the
// cache attention - weighted by 2^(m - M) and divided by the weighted sum.  A warp per row, eight shares loaded at a time.
// --------------------------------------------------------------------------------------------
struct PfCombineArgs {
  SplitArgs own;
  const float *part_o, *part_ml;
  const int32_t *lens;
  int64_t total;  // tiles of all items
  int tiles, ctas, groups, R, rt, width, rec_shift, prefix;
};

constexpr int PC_THREADS = 128, PC_FEW = 8;
template <int D>
__global__ void __launch_bounds__(PC_THREADS) prefix_combine_kernel(const PfCombineArgs a) {
  constexpr int NL = D / 4;
  start_after_earlier();
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (PC_THREADS / 32) + (threadIdx.x >> 5);
  const int rows = a.own.rows;                      // of a sequence and KV head
  const int64_t per = static_cast<int64_t>(a.own.B) * rows;
  const int kvh = static_cast<int>(i / per);
  if (kvh >= a.own.Hkv) return;
  const int r = static_cast<int>(i - kvh * per), b = r / rows, rr = r % rows;
  const int64_t cap = static_cast<int64_t>(a.width) << (a.rec_shift + 4);
  const int len = max(a.lens[b] > cap ? static_cast<int>(cap) : a.lens[b], 0);
  __nv_bfloat16 *out = a.own.row(b, kvh, rr) + 4 * lane;
  if (len == 0) {
    if (lane < NL) put_row(out, make_float4(0.f, 0.f, 0.f, 0.f), 0.f);
    return;
  }
  const int tile = 8 * a.rt, oitem = (b * a.own.Hkv + kvh) * a.own.ntile + rr / tile;
  const int2 ends = a.own.ends[oitem];
  const int n_own = ends.y - ends.x + 1;
  const int64_t own0 = (static_cast<int64_t>(ends.x) + oitem) * tile + rr % tile;
  int n = n_own;
  int64_t pre0 = 0;
  if (len - a.own.Nq >= a.prefix) {
    const int prow = 128 * a.R, item = kvh * a.groups + r / prow;
    // CTA c holds tiles total c / ctas .. total (c + 1) / ctas - 1
    const int64_t t0 = static_cast<int64_t>(item) * a.tiles, t1 = t0 + a.tiles - 1;
    const int c0 = static_cast<int>(((t0 + 1) * a.ctas - 1) / a.total), c1 = static_cast<int>(((t1 + 1) * a.ctas - 1) / a.total);
    pre0 = (static_cast<int64_t>(c0) + item) * PF_ROWS + r % prow;
    n += (c1 - c0 + 1) * (a.R == 2 ? 1 : 2);
  }
  const int64_t pstep = a.R == 2 ? PF_ROWS : 128;
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int w = 0; w < n; w += PC_FEW) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < PC_FEW && w + lane < n) {
      const int k = w + lane;
      ml = k < n_own ? *reinterpret_cast<const float2 *>(a.own.part_ml + 2 * (own0 + static_cast<int64_t>(k) * tile))
                     : *reinterpret_cast<const float2 *>(a.part_ml + 2 * (pre0 + (k - n_own) * pstep));
    }
    float4 v[PC_FEW];
#pragma unroll
    for (int u = 0; u < PC_FEW; ++u) {
      const int k = w + u;
      if (k < n && lane < NL)
        v[u] = k < n_own ? *reinterpret_cast<const float4 *>(a.own.part_o + (own0 + static_cast<int64_t>(k) * tile) * D + 4 * lane)
                         : *reinterpret_cast<const float4 *>(a.part_o + (pre0 + (k - n_own) * pstep) * D + 4 * lane);
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
  if (lane < NL) put_row(out, o, L == 0.f ? 0.f : 1.f / L);
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
  const dim3 grid(static_cast<unsigned>((rows * own.Hkv + PC_THREADS / 32 - 1) / (PC_THREADS / 32)));
  return l.d == 128 ? launch_dependent(prefix_combine_kernel<128>, grid, PC_THREADS, 0, st, a)
                    : launch_dependent(prefix_combine_kernel<64>, grid, PC_THREADS, 0, st, a);
}

}  // namespace sparge
