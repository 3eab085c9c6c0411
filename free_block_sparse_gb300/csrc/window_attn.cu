// Causal attention over a sliding window and a few first tokens, for chunks of queries, on tcgen05 tensor
// cores: query row at position p sees key c <= p when c > p - window or c < sinks.
//
// One CTA computes 128 rows against the 64-key blocks that they see (the first tokens', then the window's), one after
// another.  The rows are P = 128 / heads queries of as many heads of a KV head as its group allows (a power of two up to 16):
// P queries see window + P - 1 keys between them, so fewer of them mean fewer blocks and fewer hidden scores for the
// same rows.  Warp roles (160 threads):
//   warps 0-3  softmax + epilogue; one query row per thread (TMEM lane).
//   warp 4     one thread: TMA loads of Q, then of each block's K and V (an f16 copy), and the products: the next
//              block's S = Q K^T as soon as the softmax has read this one's, then O += P V of this one.
// A short window leaves a CTA few blocks between its start and its end, and at d = 64 a block's softmax takes longer than
// its products, so what pays is CTAs side by side whose chains of score, softmax and product cover one another:
// P has TMEM columns of its own, so one score buffer is enough and at d = 64 three CTAs share an SM (2 at d = 128,
// where O takes 128 columns); five warps, so 128 registers hold a row's 64 scores; every load stage and buffer is freed by a
// barrier that is waited for anyway.
//
// Softmax in the log2 domain.  The exponent reference moves only when a score passes it by more than 8 (P <= 2^8):
// then O and the row sum are scaled down.  Columns are masked 32 by a warp's 32 rows: hidden from all, seen by all, or a
// bit mask per row.  P and V enter the second product as f16, which keeps 3 more bits of P than bf16 would.
//
// Measured (f16 copy of V included; beside it the block-sparse kernel under the same mask, two score buffers per CTA):
// d = 64, 32 + 8 heads of 16K, window 4096: 534 us (668), 46% of the tensor peak; 2 x 15K of 64 + 8 heads, window 461: 409 us
// (792; 454 with tiles of 128 queries of one head); d = 128, 32 + 8 heads of 16K: window 256 162 us (209), 1280 365 (367),
// 1536 415 (405), 4096 859 (767): at d = 128 the products alone fill the tensor unit, which two score buffers
// feed better over a long window.
// At d = 64 under the long window a block takes 680 cycles of an SM: 1510 instructions (380 per scheduler) and the chain's waits; the
// products 340.
#include <cfloat>

#include <cuda_fp16.h>

#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace sparge {
namespace {

constexpr int WA_THREADS = 160;
constexpr float WA_RESCALE = 8.f;

struct WindowAttnArgs {
  __nv_bfloat16 *o;
  const float *v_unit;
  int64_t o_sb, o_sh, o_sn;
  int Hkv, G, Nq, Nk, ntile, nkb, off, window, sinks;  // off = Nk - Nq
  int shift;                                           // P = 1 << shift queries of a tile, of 128 / P heads
  float scale_log2;
  int *status;
};

template <int D>
struct WaCfg {
  static constexpr int CTAS = D == 64 ? 3 : 2;                 // per SM
  static constexpr uint32_t CHUNK = KBLK * 128, CH = D / 64;   // 64 rows of 64 channels
  static constexpr uint32_t TILE = CH * CHUNK;
  static constexpr uint32_t Q = 0, K = 2 * TILE, V = K + 2 * TILE, CTRL = V + 2 * TILE;
  // at least 58 KB (d = 128: 77) of shared memory keeps a further CTA, for which there is no TMEM, off the SM
  static constexpr uint32_t MIN = (D == 64 ? 58u : 77u) * 1024u;
  static constexpr uint32_t SMEM = CTRL + 512 > MIN ? CTRL + 512 : MIN;
  // TMEM columns: O, then S, then P.  Allocations are powers of two: 128 and 32 (three CTAs: 480 of 512), or 256.  The two
  // are made before the CTA gives up its permit to allocate; three CTAs never hold all columns, so each gets its second.
  static constexpr uint32_t TMEM = 2 * D, SCOL = D, PCOLS = 32;
};
struct WaCtrl {
  uint64_t q_full, s_full, s_free, p_full, pv_done, drained;
  uint64_t k_full[2], v_full[2];
  uint32_t tmem_base, tmem_p;
  int abort, no_abort;  // no_abort: for waits that an abort does not end
};
static_assert(sizeof(WaCtrl) <= 512, "control block");

// The key blocks of the P queries from position p0 on: `ns` of the first tokens, then from `lo` on, n in all.
struct WaBlocks {
  int ns, lo, n;
  __device__ __forceinline__ WaBlocks(const WindowAttnArgs &a, int p0) {
    const int first = p0 - a.window + 1;
    lo = first > 0 ? first / KBLK : 0;
    ns = min(lo, a.sinks / KBLK + (a.sinks % KBLK != 0 ? 1 : 0));
    n = ns + min(a.nkb, (p0 + (1 << a.shift) - 1) / KBLK + 1) - lo;
  }
  __device__ __forceinline__ int at(int t) const { return t < ns ? t : lo + t - ns; }
};

// tcgen05.wait::ld that the loaded registers pass through, so nothing that uses them moves in front of it.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32], float &m) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+f"(m)
               :
               : "memory");
}

// bits 0 .. k (none below 0, all from 31 on)
__device__ __forceinline__ uint32_t upto(int k) { return k < 0 ? 0u : k >= 31 ? 0xffffffffu : (2u << k) - 1u; }

template <int D>
__global__ void __launch_bounds__(WA_THREADS, WaCfg<D>::CTAS)
    window_attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const WindowAttnArgs a) {
  using C = WaCfg<D>;
  constexpr uint32_t IDESC_S = idesc_f32acc(128, KBLK, FMT_BF16, false);
  constexpr uint32_t IDESC_PV = idesc_f32acc(128, D, FMT_F16, true);
  extern __shared__ __align__(1024) uint8_t smem[];
  // the 128-byte swizzle of TMA and of the MMA descriptors assumes 1024-byte aligned tiles
  if (smem_u32(smem) & 1023u) {
    wait_for_earlier();
    if (threadIdx.x == 0) record_status(a.status, -4 /* SPARGE_ERR_CUDA */);
    return;
  }
  WaCtrl &cs = *reinterpret_cast<WaCtrl *>(smem + C::CTRL);
  volatile int *abort = &cs.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // work item: (b, kvh) outermost so that CTAs of the same time share K and V in L2, a tile's groups of heads adjacent
  const int heads = 128 >> a.shift, groups = a.G / heads, per_bk = a.ntile * groups;
  const int bk = blockIdx.x / per_bk, rem = blockIdx.x % per_bk;
  const int b = bk / a.Hkv, kvh = bk % a.Hkv, h0 = kvh * a.G + rem % groups * heads;
  const int q0 = (a.ntile - 1 - rem / groups) << a.shift;  // the tile's first query
  const WaBlocks wb(a, a.off + q0);

  if (threadIdx.x == 0) {
    mbar_init(&cs.q_full, 1);
    mbar_init(&cs.s_full, 1);
    mbar_init(&cs.drained, 1);
    mbar_init(&cs.s_free, 4);
    mbar_init(&cs.p_full, 4);
    mbar_init(&cs.pv_done, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&cs.k_full[s], 1);
      mbar_init(&cs.v_full[s], 1);
    }
    cs.abort = 0;
    cs.no_abort = 0;
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&cs.tmem_base, C::TMEM);
    if (D == 64) tmem_alloc(&cs.tmem_p, C::PCOLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  let_dependents_start();
  wait_for_earlier();
  const uint32_t tmem = cs.tmem_base, tmem_p = D == 64 ? cs.tmem_p : tmem + C::SCOL + KBLK;

  // block t of K or V into its stage, t % 2
  auto load = [&](uint32_t ring, const CUtensorMap *map, uint64_t *bar, int t) {
    const int st = t % 2;
    mbar_arrive_expect_tx(bar + st, C::TILE);
    for (uint32_t c = 0; c < C::CH; ++c)
      tma_load_4d(smem + ring + st * C::TILE + c * C::CHUNK, map, bar + st, 64 * c, KBLK * wb.at(t), kvh, b);
  };
  if (warp == 4) {
    // ------------------------------------ loads and products ------------------------------------
    if (lane == 0) {
      mbar_arrive_expect_tx(&cs.q_full, 2 * C::TILE);
      for (uint32_t c = 0; c < C::CH; ++c)
        tma_load_4d(smem + C::Q + c * 2 * C::CHUNK, &tq, &cs.q_full, 64 * c, q0, h0, b);
      load(C::K, &tk, cs.k_full, 0);
      load(C::V, &tv, cs.v_full, 0);
      if (wb.n > 1) load(C::K, &tk, cs.k_full, 1);
      const uint64_t dq = smem_desc_sw128(smem_u32(smem + C::Q), 16, 1024);
      const uint64_t dk = smem_desc_sw128(smem_u32(smem + C::K), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_u32(smem + C::V), C::CHUNK, 1024);
      auto scores = [&](int t) {
        tc_fence_after();
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_bf16_ss(tmem + C::SCOL, dq + (s >> 2) * (2 * C::CHUNK >> 4) + (s & 3) * 2,
                      dk + (t % 2) * (C::TILE >> 4) + (s >> 2) * (C::CHUNK >> 4) + (s & 3) * 2, IDESC_S, s > 0 ? 1u : 0u);
        mma_commit(&cs.s_full);
      };
      auto landed = [&](uint64_t *bar, int t) { return mbar_wait(bar + t % 2, (t / 2) & 1, abort, a.status); };
      bool ok = mbar_wait(&cs.q_full, 0, abort, a.status) && landed(cs.k_full, 0);
      if (ok) scores(0);
      for (int t = 0; ok && t < wb.n; ++t) {
        if (t + 1 < wb.n) {  // the next scores, once the softmax has read these
          if (!(ok = landed(cs.k_full, t + 1) && mbar_wait(&cs.s_free, t & 1, abort, a.status))) break;
          scores(t + 1);
          if (t + 2 < wb.n) load(C::K, &tk, cs.k_full, t + 2);  // over block t, whose scores have been read
        }
        if (!(ok = landed(cs.v_full, t) && mbar_wait(&cs.p_full, t & 1, abort, a.status))) break;
        tc_fence_after();
#pragma unroll
        for (int s = 0; s < KBLK / 16; ++s)
          mma_bf16_ts(tmem, tmem_p + s * 8, dv + (t % 2) * (C::TILE >> 4) + s * (2048 >> 4), IDESC_PV, t > 0 || s > 0 ? 1u : 0u);
        mma_commit(&cs.pv_done);
        // over block t - 1, whose product was done before this P was written
        if (t + 1 < wb.n) load(C::V, &tv, cs.v_full, t + 1);
      }
      if (!ok) {  // products in flight end before the CTA gives its TMEM back, copies before it exits
        mma_commit(&cs.drained);
        mbar_wait(&cs.drained, 0, &cs.no_abort, a.status);
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 1000000ull) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------ softmax warps ------------------------------------
    // (rows past the last query: zeros from TMA, computed and dropped)
    const int r = warp * 32 + lane, qi = q0 + (r & ((1 << a.shift) - 1)), pos = a.off + qi;
    // the positions of the warp's rows lie in pos0 .. pos1
    const int pos0 = a.off + q0 + ((warp * 32) & ((1 << a.shift) - 1)), pos1 = pos0 + min(32, 1 << a.shift) - 1;
    const bool row_ok = qi < a.Nq;
    const uint32_t tl = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    const uint32_t sc = tl + C::SCOL, pc = tmem_p + (static_cast<uint32_t>(warp * 32) << 16);
    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
    for (int t = 0; t < wb.n; ++t) {
      const int j = wb.at(t);
      ok = __all_sync(0xffffffffu, mbar_wait(&cs.s_full, t & 1, abort, a.status));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[2][32];
      float mh[2];
      tmem_ld32_max(sc, v[0], mh[0]);
      tmem_ld32_max(sc + 32, v[1], mh[1]);
      tmem_ld_wait_for(v[0], mh[0]);
      tmem_ld_wait_for(v[1], mh[1]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&cs.s_free);
      // 32 columns by this warp's 32 rows: hidden from all, seen by all (most), or mixed
      bool hidden[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int key0 = KBLK * j + 32 * c;
        hidden[c] = key0 > pos1 || (key0 + 31 <= pos0 - a.window && key0 >= a.sinks);
        if (hidden[c]) {
          mh[c] = -INFINITY;
        } else if (key0 + 31 > pos0 || (key0 <= pos1 - a.window && key0 + 31 >= a.sinks)) {
          // bit k: this row sees column k (up to its position, and in its window or among the first tokens)
          const int lim = pos - key0, low = lim - a.window, open = a.sinks - key0;
          const uint32_t seen = upto(lim) & (~upto(low) | upto(open - 1));
          mh[c] = -INFINITY;
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            if (!((seen >> k) & 1u)) v[c][k] = 0xFF800000u;  // -inf
            mh[c] = fmaxf(mh[c], __uint_as_float(v[c][k]));
          }
        }
      }
      const float m = fmaxf(mh[0], mh[1]) * a.scale_log2;
      // the product of block t - 1 has read its P and added to O
      if (t > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&cs.pv_done, (t - 1) & 1, abort, a.status));
        if (!ok) break;
        tc_fence_after();
      }
      const bool resc = m > m_ref + WA_RESCALE;
      if (__any_sync(0xffffffffu, resc)) {
        const float alpha = resc ? fast_exp2(m_ref - m) : 1.f;
        if (resc) m_ref = m;
        l *= alpha;
        if (t > 0) {
#pragma unroll 1
          for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            tmem_ld16(tl + 16 * q, o);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
            tmem_st16(tl + 16 * q, o);
          }
        }
      }
      // P = 2^(x * scale_log2 - m_ref); a row whose reference is still -inf has only hidden columns
      const float nref = m_ref == -INFINITY ? 0.f : -m_ref;
      const float2 nr2 = make_float2(nref, nref);
      float2 rs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) pk[k] = 0u;
        if (!hidden[c]) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 e2 = ffma2(make_float2(__uint_as_float(v[c][2 * k]), __uint_as_float(v[c][2 * k + 1])), sc2, nr2);
            const float2 p2 = make_float2(fast_exp2(e2.x), fast_exp2(e2.y));
            rs[k & 1] = fadd2(rs[k & 1], p2);
            pk[k] = pack_f16x2(p2.x, p2.y);
          }
        }
        tmem_st16(pc + 16 * c, pk);
      }
      const float2 sum = fadd2(rs[0], rs[1]);
      l += sum.x + sum.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&cs.p_full);
    }
    // ------------------------------------ epilogue ------------------------------------
    if (ok) ok = mbar_wait(&cs.pv_done, (wb.n - 1) & 1, abort, a.status);  // every product has completed
    __syncwarp();
    tc_fence_after();
    const bool all_ok = __all_sync(0xffffffffu, ok);
    const float inv_l = l > 0.f ? a.v_unit[bk] / l : 0.f;  // (bk: this (batch, KV head))
    __nv_bfloat16 *orow = a.o + b * a.o_sb + (h0 + (r >> a.shift)) * a.o_sh + static_cast<int64_t>(qi) * a.o_sn;
#pragma unroll 1
    for (int q = 0; q < (all_ok ? D / 16 : 0); ++q) {
      uint32_t o[16];
      tmem_ld16(tl + 16 * q, o);
      tmem_ld_wait();
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        w[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv_l, __uint_as_float(o[2 * k + 1]) * inv_l);
      if (row_ok) {
        *reinterpret_cast<uint4 *>(orow + 16 * q) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(orow + 16 * q + 8) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) {
    tmem_dealloc(tmem, C::TMEM);
    if (D == 64) tmem_dealloc(tmem_p, C::PCOLS);
  }
}

template <int D>
cudaError_t launch_t(const WindowAttn &l, const WindowAttnArgs &a, cudaStream_t st) {
  static std::atomic<unsigned long long> smem_set{0};
  if (cudaError_t e = set_smem_limit_once(window_attn_kernel<D>, static_cast<int>(WaCfg<D>::SMEM), smem_set); e != cudaSuccess)
    return e;
  const int64_t grid = static_cast<int64_t>(l.B) * a.Hkv * (a.G / (128 >> a.shift)) * a.ntile;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  // Set up while the copy of V runs (4 x 16 heads of 323 queries 13.0 us, else 14.3), but for few CTAs of many blocks: those
  // would crowd on the SMs that the copy leaves (210 CTAs of 65 blocks 65 us, else 62).
  if (grid < 152 * WaCfg<D>::CTAS && a.window > 24 * KBLK) {
    window_attn_kernel<D><<<static_cast<unsigned>(grid), WA_THREADS, WaCfg<D>::SMEM, st>>>(l.tq, l.tk, l.tv, a);
    return cudaGetLastError();
  }
  return launch_dependent(window_attn_kernel<D>, dim3(static_cast<unsigned>(grid)), WA_THREADS, WaCfg<D>::SMEM, st, l.tq, l.tk,
                          l.tv, a);
}

}  // namespace

cudaError_t launch_window_attn(const WindowAttn &l, cudaStream_t st) {
  WindowAttnArgs a;
  a.o = static_cast<__nv_bfloat16 *>(l.o);
  a.v_unit = l.v_unit;
  a.o_sb = l.o_sb; a.o_sh = l.o_sh; a.o_sn = l.o_sn;
  a.Hkv = l.Hkv; a.G = l.G;
  a.Nq = l.Nq; a.Nk = l.Nk; a.off = l.Nk - l.Nq;
  const int P = window_attn_queries(l.G);
  a.shift = 0;
  while ((1 << a.shift) < P) ++a.shift;
  a.ntile = (l.Nq + P - 1) / P;
  a.nkb = (l.Nk + KBLK - 1) / KBLK;
  a.window = l.window;
  a.sinks = l.sinks;
  a.scale_log2 = l.scale * 1.4426950408889634f;
  a.status = l.status;
  if (l.window < 1) return cudaErrorInvalidValue;
  return l.d == 128 ? launch_t<128>(l, a, st) : launch_t<64>(l, a, st);
}

}  // namespace sparge
