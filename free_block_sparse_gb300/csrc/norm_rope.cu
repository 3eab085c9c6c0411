// Norm of queries and keys for each head and rotation by position, in one pass (the step that comes
// before the attention of a model whose heads are normalised).
//
//   y = x / sqrt(mean(x^2) + eps) * w          per token and head, over the d channels
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t)   for the rot/2 pairs of the first rot channels,
//                                                t = position * inv_freq[pair]
//
// Bound by memory: q and k are read once and written once; fp32 arithmetic, one rounding to bf16.
// Measured at 32K tokens of 32 + 8 heads, d = 128: 104 us for 671 MB, 96% of the measured copy rate.
// D / 16 threads share a row, 16 channels each as two 16-byte pieces chosen so that both channels of
// every pair are in one thread.  A thread keeps its place in the row for all heads of a token, so
// the angles of its 8 pairs are computed once per token and serve every head of its share, and with
// the weights folded into them an element costs two packed products.
// Angles: the frequency is held as a fraction of a turn in 64-bit fixed point, so position times
// frequency modulo one turn is one integer product, exact to position * 2^-64 turns at any
// position; its top 32 bits give an angle in [-pi, pi), where the hardware's sine and cosine are within
// 2^-21 (a thousandth of the output's rounding).
#include <cmath>

#include "../../include/sparge.h"
#include "common.cuh"
#include "dependent.cuh"
#include "kernels.h"

namespace sparge {
namespace {

struct NormRopeArgs {
  const __nv_bfloat16 *x[2];  // q, k
  __nv_bfloat16 *y[2];
  int64_t xsb[2], xsh[2], xsn[2], ysb[2], ysh[2], ysn[2];
  const float *w[2];
  int H[2];
  const int32_t *pos;
  const double *inv_freq;
  int64_t start;
  int64_t tokens;  // B N
  int N, rot, per;  // per: heads of one CTA
  float eps;
};

constexpr int NR_THREADS = 128;
// Heads whose rows a thread has in flight while it computes as many (32K tokens of 32 + 8 heads: 104 us;
// with 2 heads 109, with 1 127).
constexpr int NR_U = 4;
constexpr int NR_PER = 20;  // most heads of a CTA

// inv_freq (radians per token) as turns per token in units of 2^-64, modulo one turn.  The double is
// M 2^e with a 53-bit M; M 2^11 times 2^66 / (2 pi) (its high word) is M 2^13 / (2 pi), and a shift
// by e + 51 brings it to units of 2^-64 turns.  Infinities and NaN have no angle: 0.
__device__ __forceinline__ uint64_t turns64(double f) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((b >> 52) & 0x7FFu);
  if (ex == 0 || ex == 0x7FF) return 0ull;
  const uint64_t m = ((b & 0xFFFFFFFFFFFFFull) | 0x10000000000000ull) << 11;
  const uint64_t hi = __umul64hi(m, 0xA2F9836E4E44152Aull);  // 2^66 / (2 pi) = 2^65 / pi
  const int sh = ex - 1075 + 51;
  uint64_t t = sh >= 0 ? (sh < 64 ? hi << sh : 0ull) : (sh > -64 ? hi >> -sh : 0ull);
  return (b >> 63) ? 0ull - t : t;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(NR_THREADS) norm_rope_kernel(const NormRopeArgs a) {
  constexpr int TR = D / 16;                 // threads of a row
  constexpr int TOK = NR_THREADS / TR;       // tokens of a CTA
  let_dependents_start();
  const int t = threadIdx.x % TR;
  const int64_t m = static_cast<int64_t>(blockIdx.x) * TOK + threadIdx.x / TR;
  const bool live = m < a.tokens;
  const int64_t mm = live ? m : a.tokens - 1;
  const int b = static_cast<int>(mm / a.N), n = static_cast<int>(mm % a.N);
  // the thread's two pieces of 8 channels: neighbouring pairs lie in adjacent pieces; pairs
  // (i, i + rot/2) in pieces rot/16 apart, the channels behind rot two by two
  const int rc = a.rot / 16;
  int p0, p1;
  if (INTER || t >= rc) {
    p0 = 2 * t;
    p1 = 2 * t + 1;
  } else {
    p0 = t;
    p1 = t + rc;
  }
  // heads h0 .. h1 - 1 of q's, then k's; a group of up to NR_U heads of one side is loaded while the one
  // before it is computed, the first while the angles are
  int h = blockIdx.y * a.per;
  const int h1 = min(h + a.per, a.H[0] + a.H[1]);
  auto row = [&](int head, int s) {
    return a.x[s] + b * a.xsb[s] + static_cast<int64_t>(n) * a.xsn[s] + (s ? head - a.H[0] : head) * a.xsh[s];
  };
  uint4 v[NR_U][2];
  auto load = [&](int head) {  // the group that starts at `head`; returns its size
    const int s = head >= a.H[0] ? 1 : 0, cnt = min(NR_U, (s ? h1 : min(h1, a.H[0])) - head);
    const __nv_bfloat16 *x = row(head, s);
#pragma unroll
    for (int u = 0; u < NR_U; ++u)
      if (u < cnt) {
        v[u][0] = *reinterpret_cast<const uint4 *>(x + u * a.xsh[s] + 8 * p0);
        v[u][1] = *reinterpret_cast<const uint4 *>(x + u * a.xsh[s] + 8 * p1);
      }
    return cnt;
  };
  wait_for_earlier();
  int cnt = load(h);
  __shared__ uint64_t turns[D / 2];
  for (int j = threadIdx.x; j < a.rot / 2; j += NR_THREADS) turns[j] = turns64(a.inv_freq[j]);
  __syncthreads();
  float cs[8], sn[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = 1.f;
    sn[j] = 0.f;
  }
  if (t < rc) {
    const int64_t pos = a.pos ? static_cast<int64_t>(a.pos[mm]) : a.start + n;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t ph = static_cast<uint64_t>(pos) * turns[8 * t + j];
      const float angle = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 1.4629180792671596e-9f;  // pi 2^-31
      sn[j] = __sinf(angle);
      cs[j] = __cosf(angle);
    }
  }
  int side = -1;
  float2 own[8], other[8];
  while (cnt > 0) {
    const int s = h >= a.H[0] ? 1 : 0;
    // The weights go into the rotation: pair number j of the thread is channels (ia, ib) of its 16, and
    // y_a = r (x_a w_a cos - x_b w_b sin), y_b = r (x_b w_b cos + x_a w_a sin); own[i] multiplies channel
    // i itself, other[i] its partner.
    if (s != side) {
      side = s;
      float w[16], o[16], p[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = a.w[s] ? a.w[s][8 * (j < 8 ? p0 : p1) + (j & 7)] : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int ia = INTER ? 2 * j : j, ib = INTER ? 2 * j + 1 : 8 + j;
        o[ia] = w[ia] * cs[j];
        o[ib] = w[ib] * cs[j];
        p[ia] = -(w[ib] * sn[j]);
        p[ib] = w[ia] * sn[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        own[j] = make_float2(o[2 * j], o[2 * j + 1]);
        other[j] = make_float2(p[2 * j], p[2 * j + 1]);
      }
    }
    __nv_bfloat16 *y = a.y[s] + b * a.ysb[s] + static_cast<int64_t>(n) * a.ysn[s] + (s ? h - a.H[0] : h) * a.ysh[s];
    const int now = cnt;
    uint4 cur[NR_U][2];
#pragma unroll
    for (int u = 0; u < NR_U; ++u) {
      cur[u][0] = v[u][0];
      cur[u][1] = v[u][1];
    }
    h += now;
    cnt = h < h1 ? load(h) : 0;
#pragma unroll
    for (int u = 0; u < NR_U; ++u) {
      if (u >= now) break;  // the same for the whole CTA
      float2 f[8];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t q[4] = {cur[u][k].x, cur[u][k].y, cur[u][k].z, cur[u][k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) f[4 * k + j] = make_float2(bf16lo(q[j]), bf16hi(q[j]));
      }
      float2 s2 = fmul2(f[0], f[0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) s2 = ffma2(f[j], f[j], s2);
      float ss = s2.x + s2.y;
#pragma unroll
      for (int off = TR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
      const float2 r2 = make_float2(r, r);
      uint32_t o[8];
      // x r first: x w may leave fp32's range where the norm would have brought it back
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmul2(f[j], r2);
      if (t < rc) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 partner = INTER ? make_float2(f[j].y, f[j].x) : f[(j + 4) % 8];
          const float2 g = ffma2(f[j], own[j], fmul2(partner, other[j]));
          o[j] = pack_bf16x2(g.x, g.y);
        }
      } else {  // channels that do not turn have no partner: an infinity or a NaN stays in its own
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 g = fmul2(f[j], own[j]);
          o[j] = pack_bf16x2(g.x, g.y);
        }
      }
      if (live) {
        *reinterpret_cast<uint4 *>(y + u * a.ysh[s] + 8 * p0) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(y + u * a.ysh[s] + 8 * p1) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace
}  // namespace sparge

using namespace sparge;

extern "C" int sparge_qk_norm_rope(const sparge_tensor *q, const sparge_tensor *k, const int32_t *positions,
                                   int64_t start, const double *inv_freq, int rot_dim, int interleaved,
                                   const float *q_weight, const float *k_weight, float eps, sparge_tensor *q_out,
                                   sparge_tensor *k_out, sparge_stream_t stream) {
  clear_error();
  View v[4];
  int rc;
  if ((rc = check_tensor(q, "q", &v[0])) || (rc = check_tensor(k, "k", &v[1])) ||
      (rc = check_tensor(q_out, "q_out", &v[2])) || (rc = check_tensor(k_out, "k_out", &v[3])))
    return rc;
  if (v[0].B != v[1].B || v[0].N != v[1].N || v[0].d != v[1].d)
    return fail(SPARGE_ERR_INVALID_ARG, "q and k disagree in B, N or d");
  for (int s = 0; s < 2; ++s) {
    const View &x = v[s], &y = v[2 + s];
    if (x.B != y.B || x.H != y.H || x.N != y.N || x.d != y.d)
      return fail(SPARGE_ERR_INVALID_ARG, "%s_out has another shape than %s", s ? "k" : "q", s ? "k" : "q");
    if (x.B * x.N != 0 && x.data == y.data && (x.sb != y.sb || x.sh != y.sh || x.sn != y.sn))
      return fail(SPARGE_ERR_INVALID_ARG, "in place, %s_out needs the strides of %s", s ? "k" : "q", s ? "k" : "q");
  }
  if (rot_dim < 0 || rot_dim > v[0].d || rot_dim % 16)
    return fail(SPARGE_ERR_INVALID_ARG, "rot_dim=%d must be a multiple of 16 in 0..%lld", rot_dim, (long long)v[0].d);
  if (rot_dim > 0 && !inv_freq) return fail(SPARGE_ERR_INVALID_ARG, "inv_freq is NULL");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(SPARGE_ERR_INVALID_ARG, "eps=%g must be finite and >= 0", (double)eps);
  if (v[0].B * v[0].N == 0) return SPARGE_OK;
  NormRopeArgs a;
  for (int s = 0; s < 2; ++s) {
    a.x[s] = static_cast<const __nv_bfloat16 *>(v[s].data);
    a.y[s] = static_cast<__nv_bfloat16 *>(const_cast<void *>(v[2 + s].data));
    a.xsb[s] = v[s].sb; a.xsh[s] = v[s].sh; a.xsn[s] = v[s].sn;
    a.ysb[s] = v[2 + s].sb; a.ysh[s] = v[2 + s].sh; a.ysn[s] = v[2 + s].sn;
    a.H[s] = static_cast<int>(v[s].H);
  }
  a.w[0] = q_weight;
  a.w[1] = k_weight;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.start = start;
  a.tokens = v[0].B * v[0].N;
  a.N = static_cast<int>(v[0].N);
  a.rot = rot_dim;
  a.eps = eps;
  const int d = static_cast<int>(v[0].d), tok = NR_THREADS / (d / 16), heads = a.H[0] + a.H[1];
  const int64_t tiles = (a.tokens + tok - 1) / tok;
  if (tiles > 0x7fffffffLL) return fail(SPARGE_ERR_UNSUPPORTED, "too many tokens");
  // Heads of a CTA: the angles serve them all (at 32K tokens of 40 heads 1 head takes 319 us, 4 134,
  // 20 104), but few tokens want CTAs for every SM (64 tokens: 1 head 2.9 us, 8 4.3), so as many as
  // leave 4 CTAs for each of the 152 SMs, in equal groups.
  int64_t per = tiles * heads / (4 * 152);
  per = per < 1 ? 1 : (per > NR_PER ? NR_PER : per);
  const int64_t groups = (heads + per - 1) / per;
  per = (heads + groups - 1) / groups;
  if ((heads + per - 1) / per > 65535) per = (heads + 65534) / 65535;  // 65535 heads each
  a.per = static_cast<int>(per);
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>((heads + per - 1) / per));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      launch_dependent(d == 128 ? (interleaved ? norm_rope_kernel<128, true> : norm_rope_kernel<128, false>)
                                : (interleaved ? norm_rope_kernel<64, true> : norm_rope_kernel<64, false>),
                       grid, NR_THREADS, 0, s, a);
  return e == cudaSuccess ? SPARGE_OK : cuda_fail(e, "norm and rotation launch");
}
