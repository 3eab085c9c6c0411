// Decoding steps and short chunks under a sliding window with a few first tokens: up to WINDOW_DECODE_ROWS query
// rows per KV head (the Nq queries of its G heads), in tiles of 8 or 16, against contiguous bf16 keys and values.
//
// Bound by memory: a tile reads every visible key and value once, 4 d bytes per token and KV head (the tiles of
// one KV head side by side, from L2).  A 128-row
// tensor-core tile would be almost empty here and its softmax would still be done for all its rows, so the
// rows are the narrow side of mma.sync products (n = 8):
//   S^T = K Q^T: A = 16 tokens x 16 channels by ldmatrix, B = Q^T held in registers;
//   O^T = V^T P^T: A = 16 channels x 16 tokens by ldmatrix.trans, B = P^T transposed in registers.
// P enters as the sum of two bf16 (its value and what that leaves: 16 bits), so V is read in place as
// bf16 without losing P's precision; the second product costs nothing here.
// Each warp takes every fourth 16-token record of its CTA's share through a ring of TMA copies of its own
// (128-byte swizzle, conflict-free for ldmatrix; 3 records of 8 KB in flight per warp at d = 128, 8 warps per
// SM).  The line of tiles, the merge of the warps and the combining kernel are rowsplit.cuh's.
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/sparge.h"
#include "common.cuh"
#include "kernels.h"
#include "rowsplit.cuh"

namespace sparge {
namespace {

constexpr int WD_CTAS = 2 * CA_SMS;

struct WindowArgs : SplitArgs {
  const __nv_bfloat16 *q;
  int64_t q_sb, q_sh, q_sn;
  int Nk, window, sinks, ns, lo, recs;  // records: ns of the first tokens, then lo, lo + 1, ...
  float scale_log2;
  int *status;
  __device__ __forceinline__ bool empty(int) const { return false; }
};

template <int D, int RT>
struct WdSmem {
  static constexpr int BOX = 16 * 128;            // 16 tokens x 64 channels
  static constexpr int REC = 2 * (D / 64) * BOX;  // K boxes, then V boxes
  static constexpr int ST = D == 64 ? 6 : 3;
  static constexpr int WRING = ST * REC;
  static constexpr int OROW = D + 4;
  static_assert(8 * RT * OROW * 4 <= WRING, "a warp's sums fit its ring");
  static constexpr int OFF_ML = CA_WARPS * WRING, OFF_CTRL = OFF_ML + CA_WARPS * 8 * RT * 8;
  static constexpr int TOTAL = OFF_CTRL + 512;
};
struct WdCtrl {
  uint64_t full[CA_WARPS][6];
  int abort;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int RT>
__global__ void __launch_bounds__(CA_WARPS * 32, 2)
    window_decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const WindowArgs a) {
  using S = WdSmem<D, RT>;
  constexpr int MT = D / 16, ST = S::ST;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzle assumes it
    wait_for_earlier();
    if (threadIdx.x == 0) record_status(a.status, -4 /* SPARGE_ERR_CUDA */);
    return;
  }
  WdCtrl &cs = *reinterpret_cast<WdCtrl *>(smem + S::OFF_CTRL);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t *ring = smem + warp * S::WRING;
  if (threadIdx.x == 0) {
    cs.abort = 0;
    for (int w = 0; w < CA_WARPS; ++w)
      for (int s = 0; s < ST; ++s) mbar_init(&cs.full[w][s], 1);
    fence_barrier_init();
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  __syncthreads();
  let_dependents_start();
  wait_for_earlier();

  const int tiles = (a.recs + 3) >> 2;  // of an item, 64 tokens each; the grid has at most as many CTAs as there are tiles
  const int64_t total = static_cast<int64_t>(tiles) * a.B * a.Hkv * a.ntile;
  int64_t at = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  uint32_t used = 0;
  // addresses inside a record: this lane's row and half of the ldmatrix blocks of K and of V
  const int krow = (lane & 7) + 8 * ((lane >> 3) & 1), khalf = lane >> 4;
  const int vrow = (lane & 7) + 8 * (lane >> 4), vhalf = (lane >> 3) & 1;

  while (at < end) {
    const int item = static_cast<int>(at / tiles), tile0 = static_cast<int>(at % tiles);
    const int nt = static_cast<int>(end - at < tiles - tile0 ? end - at : tiles - tile0);
    const int rt = item % a.ntile, kvh = item / a.ntile % a.Hkv, b = item / a.ntile / a.Hkv;
    const int row0 = rt * 8 * RT;
    const int k0 = tile0 * 4 + warp, kend = min(a.recs, (tile0 + nt) * 4);
    const int nrec = kend > k0 ? (kend - k0 + 3) >> 2 : 0;
    auto token_of = [&](int k) { return 16 * (k < a.ns ? k : a.lo + k - a.ns); };
    auto issue = [&](int i) {  // one lane
      const uint32_t st = (used + i) % ST;
      const int tok = token_of(k0 + 4 * i);
      uint8_t *dst = ring + st * S::REC;
      mbar_arrive_expect_tx(&cs.full[warp][st], S::REC);
#pragma unroll
      for (int u = 0; u < D / 64; ++u) tma_load_4d(dst + u * S::BOX, &tk, &cs.full[warp][st], 64 * u, tok, kvh, b);
#pragma unroll
      for (int u = 0; u < D / 64; ++u) tma_load_4d(dst + (D / 64 + u) * S::BOX, &tv, &cs.full[warp][st], 64 * u, tok, kvh, b);
    };
    if (lane == 0)
      for (int i = 0; i < min(nrec, ST); ++i) issue(i);

    // ---- Q: B operands, and the positions of this lane's rows 2c and 2c + 1 of each row tile ----
    uint32_t qf[RT][MT][2];
    int pos[RT][2];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int r = row0 + 8 * j + g;
      const bool ok = r < a.rows;
      const int h = kvh * a.G + (ok ? r / a.Nq : 0), qi = ok ? r % a.Nq : 0;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q + b * a.q_sb + h * a.q_sh + static_cast<int64_t>(qi) * a.q_sn);
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        qf[j][u][0] = ok ? src[8 * u + c] : 0u;
        qf[j][u][1] = ok ? src[8 * u + 4 + c] : 0u;
      }
      const int p = a.Nk - a.Nq + qi;  // rows past the last are computed and dropped
      pos[j][0] = __shfl_sync(0xffffffffu, p, 8 * c);
      pos[j][1] = __shfl_sync(0xffffffffu, p, 8 * c + 4);
    }

    float acc[MT][RT][4];  // O^T: channels 16 u + g and + 8, rows 2c and 2c + 1
    float2 l[RT], nref[RT], thr[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      l[j] = both(0.f);
      nref[j] = both(0.f);
      thr[j] = both(-INFINITY);
    }
#pragma unroll
    for (int u = 0; u < MT; ++u)
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[u][j][k] = 0.f;

    auto record = [&](auto edge_tag, uint32_t p, int tok) {
      constexpr bool EDGE = decltype(edge_tag)::value;
      float sc[RT][4];
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[j][k] = 0.f;
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        uint32_t ka[4];
        ldsm4(p + (u / 4) * S::BOX + krow * 128 + (((2 * (u % 4) + khalf) ^ (krow & 7)) << 4), ka);
#pragma unroll
        for (int j = 0; j < RT; ++j) mma_bf16(sc[j], ka, qf[j][u][0], qf[j][u][1]);
      }
      // tokens g (x0) and g + 8 (x1), rows 2c and 2c + 1
      float2 x0[RT], x1[RT];
      bool move = false;
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        x0[j] = fmul2(make_float2(sc[j][0], sc[j][1]), both(a.scale_log2));
        x1[j] = fmul2(make_float2(sc[j][2], sc[j][3]), both(a.scale_log2));
        if constexpr (EDGE) {
          auto hide = [&](float &x, int t, int q) {
            if (!(t <= q && (t < a.sinks || q - t < a.window))) x = -INFINITY;
          };
          hide(x0[j].x, tok + g, pos[j][0]);
          hide(x0[j].y, tok + g, pos[j][1]);
          hide(x1[j].x, tok + g + 8, pos[j][0]);
          hide(x1[j].y, tok + g + 8, pos[j][1]);
        }
        move = move || fmaxf(x0[j].x, x1[j].x) > thr[j].x || fmaxf(x0[j].y, x1[j].y) > thr[j].y;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          float2 al;
          al.x = follow(thr[j].x, nref[j].x, fmaxf(x0[j].x, x1[j].x));
          al.y = follow(thr[j].y, nref[j].y, fmaxf(x0[j].y, x1[j].y));
          l[j] = fmul2(l[j], al);
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            acc[u][j][0] *= al.x;
            acc[u][j][1] *= al.y;
            acc[u][j][2] *= al.x;
            acc[u][j][3] *= al.y;
          }
        }
      }
      uint32_t pb[RT][2][2];  // P^T: value and rest, tokens 0-7 and 8-15
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const float2 y0 = fadd2(x0[j], nref[j]), y1 = fadd2(x1[j], nref[j]);
        const float2 p0 = make_float2(fast_exp2(y0.x), fast_exp2(y0.y)), p1 = make_float2(fast_exp2(y1.x), fast_exp2(y1.y));
        l[j] = fadd2(l[j], fadd2(p0, p1));
        const uint32_t h0 = pack_bf16x2(p0.x, p0.y), h1 = pack_bf16x2(p1.x, p1.y);
        pb[j][0][0] = transpose8x8(h0);
        pb[j][0][1] = transpose8x8(h1);
        pb[j][1][0] = transpose8x8(pack_bf16x2(p0.x - bf16lo(h0), p0.y - bf16hi(h0)));
        pb[j][1][1] = transpose8x8(pack_bf16x2(p1.x - bf16lo(h1), p1.y - bf16hi(h1)));
      }
      // EDGE: values of tokens that no query sees are taken as zero, whatever they hold (this lane's operand
      // words hold tokens 2c, 2c + 1 and 2c + 8, 2c + 9)
      uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
      if constexpr (EDGE) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t m = 0u;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int t = tok + 2 * c + 8 * k + e;  // seen by some query: positions Nk - Nq .. Nk - 1
            if (t < a.Nk && (t < a.sinks || t > a.Nk - a.Nq - a.window)) m |= 0xFFFFu << (16 * e);
          }
          keep[k] = m;
        }
      }
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        uint32_t va[4];
        ldsm4_trans(p + (D / 64 + u / 4) * S::BOX + vrow * 128 + (((2 * (u % 4) + vhalf) ^ (vrow & 7)) << 4), va);
        if constexpr (EDGE) {
          va[0] &= keep[0];
          va[1] &= keep[0];
          va[2] &= keep[1];
          va[3] &= keep[1];
        }
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          mma_bf16(acc[u][j], va, pb[j][0][0], pb[j][0][1]);
          mma_bf16(acc[u][j], va, pb[j][1][0], pb[j][1][1]);
        }
      }
    };

    for (int i = 0; i < nrec; ++i) {
      const uint32_t n = used + i, st = n % ST;
      const bool landed = mbar_wait(&cs.full[warp][st], (n / ST) & 1, &cs.abort, a.status);
      if (!__all_sync(0xffffffffu, landed)) break;
      const int tok = token_of(k0 + 4 * i);
      const uint32_t p = smem_u32(ring + st * S::REC);
      // whole for every query: not past the first query, and in the last query's window or among the first tokens
      if (tok + 15 <= a.Nk - a.Nq && (tok >= a.Nk - a.window || tok + 15 < a.sinks))
        record(std::false_type{}, p, tok);
      else
        record(std::true_type{}, p, tok);
      __syncwarp();  // every lane has read the stage
      if (lane == 0 && i + ST < nrec) issue(i + ST);
    }
    used += nrec;

    // ---- the item's (or its share's) end ----
    float *mo = reinterpret_cast<float *>(ring);  // every copy of the item has landed and been read
    float2 *ml = reinterpret_cast<float2 *>(smem + S::OFF_ML);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = 8 * j + 2 * c + k;
        float ls = k ? l[j].y : l[j].x;
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        if (g == 0)
          ml[warp * 8 * RT + row] =
              make_float2((k ? thr[j].y : thr[j].x) == -INFINITY ? -INFINITY : -(k ? nref[j].y : nref[j].x), ls);
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          mo[row * S::OROW + 16 * u + g] = acc[u][j][k];
          mo[row * S::OROW + 16 * u + 8 + g] = acc[u][j][2 + k];
        }
      }
    end_item<D, RT>(a, smem, S::WRING, S::OROW, ml, item, b, kvh, row0, tile0 == 0, tile0 + nt == tiles);
    if (*reinterpret_cast<volatile int *>(&cs.abort)) break;
    at += nt;
  }
  if (*reinterpret_cast<volatile int *>(&cs.abort)) {  // let copies already in flight land before the CTA exits
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000ull) {
    }
  }
}

template <int D, int RT>
cudaError_t launch_t(const WindowDecode &l, const WindowArgs &a, int64_t ctas, cudaStream_t st) {
  using S = WdSmem<D, RT>;
  static std::atomic<unsigned long long> smem_set{0};
  if (cudaError_t e = set_smem_limit_once(window_decode_kernel<D, RT>, S::TOTAL, smem_set); e != cudaSuccess) return e;
  if (cudaError_t e = launch_dependent(window_decode_kernel<D, RT>, dim3(static_cast<unsigned>(ctas)), CA_WARPS * 32, S::TOTAL, st,
                                       l.tk, l.tv, a);
      e != cudaSuccess)
    return e;
  return launch_split_combine<D, RT>(a, ctas, st);
}

}  // namespace

size_t window_decode_ws_bytes(int64_t B, int64_t Hkv, int64_t d) {
  return split_ws(B * Hkv * (WINDOW_DECODE_ROWS / 16), WD_CTAS, 2, d).total;
}

cudaError_t launch_window_decode(const WindowDecode &l, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(l.G) * l.Nq;
  if (rows > WINDOW_DECODE_ROWS || l.window < 1) return cudaErrorInvalidValue;
  const int rt = row_tile(rows);
  WindowArgs a;
  a.o = static_cast<__nv_bfloat16 *>(l.o);
  a.o_sb = l.o_sb; a.o_sh = l.o_sh; a.o_sn = l.o_sn;
  a.B = l.B; a.Hkv = l.Hkv; a.G = l.G; a.Nq = l.Nq;
  a.rows = static_cast<int>(rows);
  a.ntile = static_cast<int>((rows + 8 * rt - 1) / (8 * rt));
  const int64_t items = static_cast<int64_t>(l.B) * l.Hkv * a.ntile;
  if (items > INT_MAX) return cudaErrorInvalidValue;
  const SplitWs w = split_ws(items, WD_CTAS, rt, l.d);
  uint8_t *ws = static_cast<uint8_t *>(l.ws);
  a.part_o = reinterpret_cast<float *>(ws + w.o);
  a.part_ml = reinterpret_cast<float *>(ws + w.ml);
  a.ends = reinterpret_cast<int2 *>(ws + w.ends);
  a.q = static_cast<const __nv_bfloat16 *>(l.q);
  a.q_sb = l.q_sb; a.q_sh = l.q_sh; a.q_sn = l.q_sn;
  a.Nk = l.Nk; a.window = l.window; a.sinks = l.sinks;
  const int first = l.Nk - l.Nq - l.window + 1;  // the first key of the first query's window
  a.lo = first > 0 ? first / 16 : 0;
  a.ns = l.sinks / 16 + (l.sinks % 16 != 0);
  if (a.ns > a.lo) a.ns = a.lo;
  a.recs = a.ns + (l.Nk + 15) / 16 - a.lo;
  a.scale_log2 = l.scale * 1.4426950408889634f;
  a.status = l.status;
  const int64_t total = (a.recs + 3) / 4 * items, ctas = total < WD_CTAS ? total : WD_CTAS;
  if (l.d == 128) return rt == 1 ? launch_t<128, 1>(l, a, ctas, st) : launch_t<128, 2>(l, a, ctas, st);
  return rt == 1 ? launch_t<64, 1>(l, a, ctas, st) : launch_t<64, 2>(l, a, ctas, st);
}

}  // namespace sparge
