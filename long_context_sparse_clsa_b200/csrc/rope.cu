// Rotary positions of queries and keys, one launch (rotary embedding: Su et al. 2021,
// "RoFormer"; by-parts frequencies: Peng et al. 2023, "YaRN", the ramp over turns).
//
//   pair i of a head's first rot elements, position pos:  a = pos f_i
//   (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
//
// The kernel moves every element in and out once: HBM is the bound (671 MB for 32768
// tokens of 32 + 8 heads, d = 128, bf16: 101.3 us, 6.6 TB/s; 537 MB for 131072 tokens of 8 heads: 87 us, 6.2 TB/s).  The
// angles need care: pos f_i reaches 10^5 and more radians.  f_i / 2 pi comes from the host as a 64-bit
// fraction of a turn, so that its product with pos, cut to 64 bits, is the angle reduced to one
// turn; its upper 32 bits go to fp32 and into sine and cosine.  The fraction comes from a double, off by about
// 2^-55 turns a token for the fastest pair, as fp64 angles are (2^-38 turns at 131072 tokens; the fp32 angle is
// off by 2^-26): what the fixed point saves is time.  One table per
// token serves all its heads (rot/2 entries in shared memory); a CTA issues its first loads before it
// computes the table.  With few heads a token the table is the larger part: with fp64 products, and the
// fractions read from the parameters by index (32 addresses a warp, one after the other), the 537 MB
// took 134 us.
// A unit of work is what one thread can turn alone: 16 bytes of the first half and 16 of
// the second ("half"), or 16 bytes ("interleaved"); so outputs may overwrite their inputs.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace clsa {

namespace {

constexpr int kMaxPairs = 64;      // d <= 128
constexpr int kMaxTokRope = 16;    // tokens per CTA
constexpr int kMaxThreadsRope = 256;
constexpr int kMaxHeads = 5;       // heads of a thread in flight (timed for 8, 10 and 40 heads a token)

struct RopeParams {
  const void* q;
  const void* k;
  const int32_t* pos;
  void* q_out;
  void* k_out;
  int n_pos, jq, jk;   // rows n + j n_pos, j < jq (queries) and j < jk (keys), share position n
  int Hq, Hk, d, rot;
  int tpc;             // tokens per CTA
  float mscale, sign;  // sign: -1 for the transpose
  uint64_t turns[kMaxPairs];  // of a token, in 2^-64 turns
};

template <typename T> struct Vec16;
template <> struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[8]) {
    unpack_bf16x2(v.x, x[0], x[1]);
    unpack_bf16x2(v.y, x[2], x[3]);
    unpack_bf16x2(v.z, x[4], x[5]);
    unpack_bf16x2(v.w, x[6], x[7]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  }
};
template <> struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

// A thread owns one vector (c, threadIdx.x) of the heads of one token (threadIdx.z): its cosines and
// sines stay in registers while it walks the heads threadIdx.y, + blockDim.y, ..., kHeads of
// them in flight (2, 4 or 5: what a thread does not need costs registers and instructions).  (With a flat index and a table look-up per vector the kernel was bound by its
// own instructions: 127 us for the 671 MB.)
template <typename T, bool HALF, int kHeads>
__global__ void __launch_bounds__(kMaxThreadsRope) rope_kernel(const __grid_constant__ RopeParams p) {
  pdl_enter();
  constexpr int N = Vec16<T>::N, NC = HALF ? N : N / 2;  // elements, pairs of a vector
  __shared__ __align__(16) float2 tab[kMaxTokRope][kMaxPairs];
  const int half = p.rot / 2;
  const int rv = HALF ? half / N : p.rot / N;   // vectors of a head that are turned
  const int tok = threadIdx.z, c = threadIdx.x, n = blockIdx.x * p.tpc + tok;
  const bool live = n < p.n_pos, rot = c < rv;
  const int nq = p.jq * p.Hq, nh = nq + p.jk * p.Hk;  // the position's heads: rows n, n + n_pos, ... of q, then of k
  // a pass-through vector c >= rv lies rv further on in "half"
  const int v = rot ? c : c + (HALF ? rv : 0);
  auto at = [&](int hh) {                       // element offset of the vector in q (hh < nq) or k
    const bool isq = hh < nq;
    if (!isq) hh -= nq;
    const int H = isq ? p.Hq : p.Hk, J = isq ? p.jq : p.jk;
    const int j = J == 1 ? 0 : hh / H;
    return (((size_t)j * p.n_pos + n) * H + (hh - j * H)) * p.d + (size_t)(v * N);
  };
  uint4 a[kHeads], b[kHeads];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int hh = h0 + k * blockDim.y;
      if (!live || hh >= nh) continue;
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const T*>(hh < nq ? p.q : p.k) + at(hh));
      a[k] = __ldcs(s);
      if (HALF && rot) b[k] = __ldcs(s + rv);
    }
  };
  int h0 = threadIdx.y;
  fetch(h0);
  const int nt = blockDim.x * blockDim.y * blockDim.z, me = threadIdx.x + blockDim.x * (threadIdx.y + blockDim.y * threadIdx.z);
  const int ntok = min(p.tpc, p.n_pos - (int)blockIdx.x * p.tpc);
  for (int i = me; i < ntok * half; i += nt) {
    const int t = i / half, f = i - t * half;
    uint64_t turns;                            // a load by address: the lanes' entries lie side by side
    asm("ld.u64 %0, [%1];" : "=l"(turns) : "l"(p.turns + f));
    const uint64_t x = (uint64_t)(int64_t)p.pos[blockIdx.x * p.tpc + t] * turns;
    const int h = (int)((x + 0x80000000u) >> 32);  // in 2^-32 turns, from -1/2 to 1/2
    float sn, cs;
    sincospif((float)h * 0x1p-31f, &sn, &cs);
    tab[t][f] = make_float2(cs * p.mscale, sn * p.mscale * p.sign);
  }
  __syncthreads();
  if (!live) return;
  float2 cs[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) cs[i] = rot ? tab[tok][c * NC + i] : make_float2(1.f, 0.f);
  while (h0 < nh) {
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
      const int hh = h0 + k * blockDim.y;
      if (hh >= nh) continue;
      uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(hh < nq ? p.q_out : p.k_out) + at(hh));
      if (!rot) {  // behind the rotated part: as it is
        __stcs(d, a[k]);
        continue;
      }
      float x[N];
      Vec16<T>::unpack(a[k], x);
      if constexpr (HALF) {
        float y[N];
        Vec16<T>::unpack(b[k], y);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float x1 = x[i], x2 = y[i];
          x[i] = x1 * cs[i].x - x2 * cs[i].y;
          y[i] = x2 * cs[i].x + x1 * cs[i].y;
        }
        __stcs(d, Vec16<T>::pack(x));
        __stcs(d + rv, Vec16<T>::pack(y));
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const float x1 = x[2 * i], x2 = x[2 * i + 1];
          x[2 * i] = x1 * cs[i].x - x2 * cs[i].y;
          x[2 * i + 1] = x2 * cs[i].x + x1 * cs[i].y;
        }
        __stcs(d, Vec16<T>::pack(x));
      }
    }
    h0 += kHeads * blockDim.y;
    fetch(h0);
  }
}

// turns per token of each pair, f_i / 2 pi, without the whole ones (under 1 us of the host for 64 pairs);
// false: a frequency is so large that a double holds no part of a turn
bool rope_turns(const clsa_rope_args* a, uint64_t* turns) {
  const double two_pi = 6.283185307179586476925286766559;
  double theta = a->theta;
  if (a->scaling == CLSA_ROPE_BASE) theta *= std::pow(a->factor, (double)a->rot / (a->rot - 2));
  for (int i = 0; i < a->rot / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / a->rot);
    if (a->scaling == CLSA_ROPE_LINEAR) f /= a->factor;
    if (a->scaling == CLSA_ROPE_BY_PARTS) {
      const double r = a->orig_len * f / two_pi;
      const double g = std::min(1.0, std::max(0.0, (r - a->beta_slow) / (a->beta_fast - a->beta_slow)));
      f = g * f + (1.0 - g) * f / a->factor;
    }
    const double x = f / two_pi, part = x - std::floor(x);
    if (!(x < 0x1p52)) return false;
    turns[i] = (uint64_t)std::ldexp(part, 63) << 1;  // part < 1 of 53 bits: no bit is lost above 2^-63
  }
  return true;
}

}  // namespace

cudaError_t launch_rope(const clsa_rope_args* a, cudaStream_t s) {
  RopeParams p{};
  if (!rope_turns(a, p.turns)) return cudaErrorInvalidValue;
  p.q = a->q;
  p.k = a->k;
  p.pos = a->pos;
  p.q_out = a->q_out;
  p.k_out = a->k_out;
  p.n_pos = a->n_pos;
  p.jq = a->q ? a->Nq / a->n_pos : 0;
  p.jk = a->k ? a->Nk / a->n_pos : 0;
  p.Hq = a->Hq;
  p.Hk = a->Hk;
  p.d = a->d;
  p.rot = a->rot;
  p.mscale = a->mscale > 0 ? (float)a->mscale : 1.f;
  p.sign = a->inverse ? -1.f : 1.f;
  const int n = a->dtype == CLSA_BF16 ? 8 : 4;
  const bool half = a->layout == CLSA_ROPE_HALF;
  const int uph = (half ? a->rot / 2 : a->rot) / n + (a->d - a->rot) / n;  // vectors (or pairs of them) of a head: 4 to 32
  const int nh = p.jq * p.Hq + p.jk * p.Hk;
  // Many positions: up to kMaxHeads heads a thread, CTAs of 64 threads (101.3 us for 32768 x 40 heads; 105 with
  // two heads a thread; 87 for 131072 x 8 heads, 90 with 128 threads).  Few: more threads, two heads each
  // (2.3 us for 16 x 40 heads; 3.1 with five).
  const bool many = a->n_pos >= 4 * device_info().sm_count;
  int hy = 1;
  if (!many) hy = (nh + 1) / 2;
  else while (hy * kMaxHeads < nh) hy *= 2;
  hy = std::max(1, std::min(hy, kMaxThreadsRope / uph));
  const int heads = (nh + hy - 1) / hy;           // of a thread
  const int spread = std::max(1, a->n_pos / (4 * std::max(1, device_info().sm_count)));
  p.tpc = std::max(1, std::min({kMaxTokRope, 64 / (uph * hy), spread}));
  const dim3 threads(uph, hy, p.tpc);
  const dim3 grid((a->n_pos + p.tpc - 1) / p.tpc);
  const auto go = [&](auto kh) {
    constexpr int KH = decltype(kh)::value;
    if (a->dtype == CLSA_BF16)
      return half ? launch_pdl(rope_kernel<__nv_bfloat16, true, KH>, grid, threads, 0, s, p)
                  : launch_pdl(rope_kernel<__nv_bfloat16, false, KH>, grid, threads, 0, s, p);
    return half ? launch_pdl(rope_kernel<float, true, KH>, grid, threads, 0, s, p)
                : launch_pdl(rope_kernel<float, false, KH>, grid, threads, 0, s, p);
  };
  const cudaError_t e = heads <= 2   ? go(std::integral_constant<int, 2>{})
                        : heads == 4 ? go(std::integral_constant<int, 4>{})
                                     : go(std::integral_constant<int, 5>{});
  launches_add(1, s);
  return e;
}

}  // namespace clsa
