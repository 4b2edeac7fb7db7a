// Rotary positions of queries and keys, one launch (rotary embedding: Su et al. 2021,
// "RoFormer"; by-parts frequencies: Peng et al. 2023, "YaRN", the ramp over turns).
//
//   pair i of a head's first rot elements, position pos:  a = pos f_i
//   (x1, x2) -> m (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
//
// The kernel moves every element in and out once: HBM is the bound (671 MB for 32768
// tokens of 32 + 8 heads, d = 128, bf16).  The angles need care and cost little: pos f_i
// reaches 10^5 and more radians, so f_i / 2 pi comes as fp64 from the host, the product and
// its reduction to half a turn are fp64, and sine and cosine of the reduced angle fp32.
// One table per token serves all its heads (rot/2 entries in shared memory); a CTA issues
// its first loads before it computes the table, so the fp64 work hides behind them.
// A unit of work is what one thread can turn alone: 16 bytes of the first half and 16 of
// the second ("half"), or 16 bytes ("interleaved"); so outputs may overwrite their inputs.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "kernels.h"

namespace clsa {

namespace {

constexpr int kMaxPairs = 64;      // d <= 128
constexpr int kMaxTokRope = 16;    // tokens per CTA
constexpr int kMaxThreadsRope = 256;

struct RopeParams {
  const void* q;
  const void* k;
  const int32_t* pos;
  void* q_out;
  void* k_out;
  int n_pos, jq, jk;   // rows n + j n_pos, j < jq (queries) and j < jk (keys), share position n
  int Hq, Hk, d, rot;
  int tpc;             // tokens per CTA
  int uph, upt;        // units per head, per token
  float mscale, sign;  // sign: -1 for the transpose
  double turns[kMaxPairs];
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

// one unit: where it lies, what kind it is, and its data
struct RopeUnit {
  const uint4* src = nullptr;  // null: no unit
  uint4* dst = nullptr;
  int tok = 0, c = 0;          // token of the CTA; vector of the head (of the first half, for "half")
  uint4 a, b;
};

template <typename T, bool HALF>
__global__ void __launch_bounds__(kMaxThreadsRope) rope_kernel(const RopeParams p) {
  pdl_enter();
  constexpr int N = Vec16<T>::N;
  __shared__ float2 tab[kMaxTokRope][kMaxPairs];
  const int n0 = blockIdx.x * p.tpc;
  const int ntok = min(p.tpc, p.n_pos - n0);
  const int half = p.rot / 2;
  const int total = ntok * p.upt;
  const int nt = blockDim.x;
  const int rv = HALF ? half / N : p.rot / N;   // units of a head that are turned

  auto locate = [&](int u) {
    RopeUnit r;
    if (u >= total) return r;
    r.tok = u / p.upt;
    const int w = u - r.tok * p.upt;
    int hh = w / p.uph;
    r.c = w - hh * p.uph;
    const bool isq = hh < p.jq * p.Hq;
    if (!isq) hh -= p.jq * p.Hq;
    const int H = isq ? p.Hq : p.Hk;
    const int j = hh / H, h = hh - j * H;
    const size_t row = (size_t)j * p.n_pos + n0 + r.tok;
    // the vector of the head: a pass-through unit c >= rv lies rv further on in "half"
    const int v = r.c < rv ? r.c : r.c + (HALF ? rv : 0);
    const size_t off = (row * H + h) * p.d + (size_t)v * N;
    r.src = reinterpret_cast<const uint4*>(static_cast<const T*>(isq ? p.q : p.k) + off);
    r.dst = reinterpret_cast<uint4*>(static_cast<T*>(isq ? p.q_out : p.k_out) + off);
    r.a = __ldcs(r.src);
    if (HALF && r.c < rv) r.b = __ldcs(r.src + rv);
    return r;
  };
  auto turn = [&](const RopeUnit& r) {
    if (!r.src) return;
    if (r.c >= rv) {  // behind the rotated part: as it is
      __stcs(r.dst, r.a);
      return;
    }
    float x[N], y[N];
    if (HALF) {
      Vec16<T>::unpack(r.a, x);
      Vec16<T>::unpack(r.b, y);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 cs = tab[r.tok][r.c * N + i];
        const float x1 = x[i], x2 = y[i];
        x[i] = x1 * cs.x - x2 * cs.y;
        y[i] = x2 * cs.x + x1 * cs.y;
      }
      __stcs(r.dst, Vec16<T>::pack(x));
      __stcs(r.dst + rv, Vec16<T>::pack(y));
    } else {
      Vec16<T>::unpack(r.a, x);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 cs = tab[r.tok][(r.c * N + i) / 2];
        const float x1 = x[i], x2 = x[i + 1];
        x[i] = x1 * cs.x - x2 * cs.y;
        x[i + 1] = x2 * cs.x + x1 * cs.y;
      }
      __stcs(r.dst, Vec16<T>::pack(x));
    }
  };

  int u = threadIdx.x;
  RopeUnit r0 = locate(u), r1 = locate(u + nt);
  for (int i = threadIdx.x; i < ntok * half; i += nt) {
    const int t = i / half, f = i - t * half;
    double a = (double)p.pos[n0 + t] * p.turns[f];
    a -= rint(a);                              // turns, in [-1/2, 1/2]
    float s, c;
    sincospif((float)(2.0 * a), &s, &c);
    tab[t][f] = make_float2(c * p.mscale, s * p.mscale * p.sign);
  }
  __syncthreads();
  while (r0.src) {
    turn(r0);
    turn(r1);
    u += 2 * nt;
    r0 = locate(u);
    r1 = locate(u + nt);
  }
}

// turns per token of each pair: f_i / 2 pi
void rope_turns(const clsa_rope_args* a, double* turns) {
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
    turns[i] = f / two_pi;
  }
}

}  // namespace

cudaError_t launch_rope(const clsa_rope_args* a, cudaStream_t s) {
  RopeParams p{};
  // the table of the last parameters this host thread used (64 powers cost more than a launch)
  static thread_local struct {
    bool set = false;
    int rot, scaling, orig_len;
    double v[4];
    double turns[kMaxPairs];
  } memo;
  const double v[4] = {a->theta, a->factor, a->beta_fast, a->beta_slow};
  if (!memo.set || memo.rot != a->rot || memo.scaling != a->scaling || memo.orig_len != a->orig_len ||
      std::memcmp(memo.v, v, sizeof v) != 0) {
    rope_turns(a, memo.turns);
    memo.rot = a->rot;
    memo.scaling = a->scaling;
    memo.orig_len = a->orig_len;
    std::memcpy(memo.v, v, sizeof v);
    memo.set = true;
  }
  std::memcpy(p.turns, memo.turns, sizeof p.turns);
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
  p.uph = (half ? a->rot / 2 : a->rot) / n + (a->d - a->rot) / n;
  p.upt = (p.jq * p.Hq + p.jk * p.Hk) * p.uph;
  // a CTA takes about 512 units (two a thread), more than one token where a token has few,
  // but no more than spread n_pos over the SMs
  const int spread = std::max(1, (a->n_pos + device_info().sm_count - 1) / std::max(1, device_info().sm_count));
  p.tpc = std::max(1, std::min({kMaxTokRope, 512 / std::max(1, p.upt), spread}));
  const int per = std::min(p.tpc * (long long)p.upt, 2LL * kMaxThreadsRope);
  const int threads = std::min(kMaxThreadsRope, std::max(64, ((per + 1) / 2 + 31) / 32 * 32));
  const dim3 grid((a->n_pos + p.tpc - 1) / p.tpc);
  cudaError_t e;
  if (a->dtype == CLSA_BF16)
    e = half ? launch_pdl(rope_kernel<__nv_bfloat16, true>, grid, dim3(threads), 0, s, p)
             : launch_pdl(rope_kernel<__nv_bfloat16, false>, grid, dim3(threads), 0, s, p);
  else
    e = half ? launch_pdl(rope_kernel<float, true>, grid, dim3(threads), 0, s, p)
             : launch_pdl(rope_kernel<float, false>, grid, dim3(threads), 0, s, p);
  launches_add(1, s);
  return e;
}

}  // namespace clsa
