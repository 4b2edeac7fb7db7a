// Streaming attention of few query rows over many cached tokens, shared by the 8-bit cache's
// attention and by window attention's decode form (bf16 cache):
//   O[r] = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(q_r . k_j * scale),  j over the tokens r sees.
//
// What bounds it is moving K and V: with G query heads per KV head a byte of the cache feeds 2 G
// multiplies.  So every warp is a stream of its own, with no barrier in its loop: it takes tiles of
// 16 tokens, multiplies them on the tensor core (mma.sync m16n8k16; a 128-row tcgen05 tile would be
// empty for G = 4) and keeps a running maximum, sum and output for its rows.  Consecutive tokens
// come by TMA through a ring of the warp's own in shared memory (three tiles ahead: 147 KB in flight
// on an SM at d = 128); an index list's by plain loads into the registers that feed the tensor
// core, one tile ahead (through a ring of asynchronous copies 24 layers over 2048 tokens took
// 17.4 us, by loads 16.3).
// Measured (32 heads on 8, d = 128; inputs in turn that L2 does not hold): 131072 tokens of the 8-bit cache 50.7
// us, 5.3 TB/s, of which the loop takes 42, at about the rate of a plain copy, and 8 go to the launch, the plan and the
// merge (fp32 queries 65); 16 sequences of 16K to 128K tokens, 1.0 M in all, 320 us, 6.4 TB/s; 1028 bf16 tokens
// of 16 sequences 17.5 us (fp32 37); 24 layers over 2048 selected tokens 18.3 us, a chain of latencies (plan 1.5,
// indices and first rows 3 to 6, loop 6, merge 4).  Prompt rows over one cache are not its strength: each streams
// the cache by itself, through L2 (512 rows over 16384 tokens 2.6 ms, over 131072 21 ms).
//
// Fragments.  Both products are computed transposed, so that 16 is the token axis and 8 the row
// axis (R <= 8 rows waste nothing):
//   S^T (16 tokens x 8 rows) = K (16 x d) Q^T (d x 8)       A = K, B = Q^T
//   O^T (16 of d x 8 rows)  += V^T (16 x 16 tokens) P^T     A = V^T, B = P^T
// The order of a contraction is free, so the d axis of the first product is permuted to let a
// lane read 16 contiguous bytes of its two tokens, and the d rows of the second to let it
// read contiguous bytes of its four tokens; pairs of tokens are merged by byte permutes.
// P comes out of the first product transposed for the second: two movmatrix.
//
// 8-bit cache.  e4m3 codes become halves exactly.  A key block's scale multiplies the score.
// Q is brought to half range by a power of two per row (exact but for elements 2^-28 of the
// row's largest).  The value blocks' scales 2^e go into the exponent: the output is
// accumulated from 2^(s_j + e_j - n) with a reference n of its own, so halves never lose a
// block of small scale.  e is whole for the powers of two that the cache's own write makes; of any other scale
// it has a fraction (bf16 rows), or what is left of it multiplies the weight (fp32 rows).  With fp32 queries Q
// and P are split into two halves each: 22 bits, but no finer than 2^-38 of the row's largest element of Q and 2^-32 of
// its largest weight, where the second half is subnormal (a weight 2^-16 of the largest keeps 16 bits).
// bf16 rows.  P is rounded to the type of V's operand, since a product's factors have one type: to halves (off by up
// to 2^-11 of a weight) or bf16 (2^-8); the row's sum takes it as it was.  Against 64 bits the result over the 8-bit cache
// is then off by 1.01 times what weights in fp32 leave, that over bf16 rows by 1.3 to 1.4 times (0.0022 of the
// result for 0.0016, the output's own rounding).
// fp32 rows.  The tensor core cuts its sums off instead of rounding them, always towards zero; over many
// tiles that adds up (6e-6 of the result over 700 tokens, 4e-7 as it is).  So a tile's products are added to the
// output, and 16 of d to the score, by fp32 additions.
// fp32 cache.  Every factor is the exact sum of three bf16 parts; six of the nine products
// of parts are formed.  K's and V's parts are rounded, so that the others, 2^-22.4 of a product at most and 2^-26 as a
// rule, are of either sign (parts that are all cut off lose 2^-24.7 on the average, always towards zero).  The
// parts of K and V cost more than the products, so rows beyond 8 go 16 to a unit (T = 2048, W = 1024, 32 heads on 8:
// 1390 us; 13 % less than with 8).
//
// The reference (of sums and of outputs) moves only when a score exceeds it by 2^8; then the
// sums are rescaled.  A row's largest p is at least 2^0, at most 2^8: no overflow.  Where p becomes
// halves it is 2^7 larger still (halves end at 2^16), so that the halves' smallest step, 2^-24,
// is 2^-31 of the largest.
//
// Work split.  A unit is a (sequence, row group, KV head); the heads of the same tokens go to CTAs side by
// side.  Few units of like length get whole CTAs each; else all units' tiles form one line that the
// CTAs share equally, so ragged lengths balance.  A unit that several CTAs share is merged by the one
// that arrives last, in CTA order (the result does not depend on who that is).  Many units go to a
// warp each, which shares nothing with the others (fp32, T = 742, W = 6, 32 heads on 8: 31 us, against
// 102 with CTAs).
#pragma once

#include <cuda.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fp8.cuh"
#include "kernels.h"
#include "tma.h"

namespace clsa {
namespace stream {

constexpr int kTile = 16;                   // tokens of a tile
constexpr int kMinTiles = 12;               // fewest tiles worth a CTA (one a warp)
constexpr float kNone = -3e38f;             // reference of a row that has seen nothing
constexpr float kTau = 8.f;
constexpr float kLift = 7.f;                // 8-bit cache: the largest p of a row lies in [2^7, 2^15] of half range
constexpr float kLn2 = 0.6931471805599453f;
enum Cache { kE4m3 = 0, kBf16 = 1, kFp32 = 2 };

struct Params {
  const void* Q;            // row r of sequence b: (r / G) * q_sl + b * q_sb + (g G + r % G) D
  const void* K;            // [seqs][n_max][Hkv][D]
  const void* V;
  const float* ks;          // 8-bit cache: [seqs][nblk][Hkv]
  const float* vs;
  const int32_t* idx;       // [B][k] or null
  const int32_t* count;     // [B] tokens (or selected tokens)
  void* O;                  // as Q
  float* lse;               // as Q without D, or null
  float* part;              // [2 P][rows (D + 3)]
  uint32_t* counter;        // [B nrg Hkv], zero between calls
  void* ws_header;
  long long q_sl, q_sb;
  int B, nrg, R, Hkv, G, n_max, k, nblk, bshift, seqs;
  int HG, nh, PG;           // heads side by side, Hkv / HG, groups of HG CTAs
  int T, window, sinks;     // T > 0: row r is the token count - T + r / G and sees a window and the sinks
  float scale_log2;
};
struct Maps {
  CUtensorMap k, v;         // [seqs * n_max][Hkv * D] bytes, boxes of 16 tokens (ring only)
};

// a (sequence, row group): which tokens its rows see between them
struct Item {
  int b, rg, npos;          // npos positions; position i < keepP is token i (none from keep on), the others i + shift
  int keep, keepP, shift;   // keepP: keep rounded up to a tile, so that a tile's tokens are consecutive
  int p0;                   // position of row 0 (window form)
};

__device__ __forceinline__ Item item_of(const Params& p, int s, int rows) {
  Item it;
  it.b = p.nrg == 1 ? s : s / p.nrg;
  it.rg = s - it.b * p.nrg;
  const int cnt = p.count[it.b];
  it.p0 = 0;
  if (p.T == 0) {
    it.npos = max(0, min(cnt, p.idx ? p.k : p.n_max));
    it.keep = it.keepP = it.shift = 0;
    return it;
  }
  const int len = max(0, min(cnt, p.n_max));
  const int r0 = it.rg * rows, r1 = min(r0 + rows, p.R) - 1;
  it.p0 = len - p.T;
  const int first = it.p0 + r0 / p.G, last = it.p0 + r1 / p.G;
  if (last < 0) {
    it.npos = it.keep = it.keepP = it.shift = 0;
    return it;
  }
  const int lo = max(0, first - p.window + 1);
  it.keep = min(p.sinks, lo);
  it.keepP = (it.keep + kTile - 1) / kTile * kTile;
  it.shift = lo - it.keepP;
  it.npos = it.keepP + last + 1 - lo;
  return it;
}
__device__ __forceinline__ Item item_from(const Item& x, int lane) {  // a lane's item, to all
  Item it;
  it.b = __shfl_sync(0xffffffffu, x.b, lane), it.rg = __shfl_sync(0xffffffffu, x.rg, lane);
  it.npos = __shfl_sync(0xffffffffu, x.npos, lane), it.p0 = __shfl_sync(0xffffffffu, x.p0, lane);
  it.keep = __shfl_sync(0xffffffffu, x.keep, lane), it.keepP = __shfl_sync(0xffffffffu, x.keepP, lane);
  it.shift = __shfl_sync(0xffffffffu, x.shift, lane);
  return it;
}
__device__ __forceinline__ int token_of(const Item& it, int i) {  // token of position i, or -1
  return i >= it.npos ? -1 : i >= it.keepP ? i + it.shift : i < it.keep ? i : -1;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// what the halves of `h` leave of (lo, hi)
__device__ __forceinline__ uint32_t rest_f16x2(uint32_t h, float lo, float hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_f16x2(lo - f.x, hi - f.y);
}

// (x, y) = the sum of three bf16 pairs, exactly (8 bits each, cut off); an infinity stays in the first
__device__ __forceinline__ void split3(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const float hx = __uint_as_float(__float_as_uint(x) & 0xffff0000u), hy = __uint_as_float(__float_as_uint(y) & 0xffff0000u);
  const float rx = fabsf(x) == INFINITY ? 0.f : x - hx, ry = fabsf(y) == INFINITY ? 0.f : y - hy;
  const float mx = __uint_as_float(__float_as_uint(rx) & 0xffff0000u), my = __uint_as_float(__float_as_uint(ry) & 0xffff0000u);
  hi = __byte_perm(__float_as_uint(hx), __float_as_uint(hy), 0x7632u);
  mid = __byte_perm(__float_as_uint(mx), __float_as_uint(my), 0x7632u);
  lo = __byte_perm(__float_as_uint(rx - mx), __float_as_uint(ry - my), 0x7632u);
}
// as split3, the first two parts rounded to nearest: the parts are smaller (2^-8 and 2^-17 of the number, not 2^-7 and
// 2^-15) and of either sign.  The largest numbers stay finite, and an infinity goes into the last part.
__device__ __forceinline__ void split3_near(float x, float y, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const auto near = [](float a, float b) {
    uint32_t r;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  };
  float a, b;
  hi = near(x, y);
  unpack_bf16x2(hi, a, b);
  x -= a, y -= b;
  mid = near(x, y);
  unpack_bf16x2(mid, a, b);
  lo = __byte_perm(__float_as_uint(x - a), __float_as_uint(y - b), 0x7632u);
}
__device__ __forceinline__ void add4(float (&a)[4], const float (&b)[4]) {
  a[0] += b[0], a[1] += b[1], a[2] += b[2], a[3] += b[3];
}
// the products of parts that are formed, small ones first
__device__ constexpr int kTermA[6] = {2, 0, 1, 1, 0, 0};
__device__ constexpr int kTermB[6] = {0, 2, 1, 0, 1, 0};

__device__ __forceinline__ int warp_scan_int(int v, int lane) {  // sum over the lanes up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}
__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

// 2^x, subnormal results kept: the scales of all the values that a row sees may be near 2^-100
__device__ __forceinline__ float exp2_gradual(float x) {
  const bool low = x < -64.f;
  return fast_exp2(low ? x + 64.f : x) * (low ? 0x1p-64f : 1.f);
}
// log2 by the hardware approximation: exact for powers of two (test_gpu_kv8_scales.py), -inf for 0 and subnormals
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, int NT>
constexpr int slot_floats() { return NT * 8 * (D + 3); }

// A variant: the kind of cache, fp32 rows, consecutive tokens through the ring (or loads into registers), head
// dimension, row tiles; a unit per warp.
template <int CACHE_, bool F32_, bool RING_, int D_, int NT_, bool SOLO_ = false>
struct Cfg {
  using Solo = Cfg<CACHE_, F32_, RING_, D_, NT_, true>;
  static constexpr bool SOLO = SOLO_;
  static constexpr int CACHE = CACHE_, D = D_, NT = NT_;
  static constexpr bool F32 = F32_, RING = RING_;
  static constexpr int ROWS = NT * 8;
  static constexpr int ES = CACHE == kE4m3 ? 1 : CACHE == kBf16 ? 2 : 4;  // bytes of a cache element
  static constexpr int RB = D * ES;                                       // bytes of a token's row
  static constexpr int STAGE = 2 * kTile * RB;                            // K and V of a tile
  // warps of a CTA (one CTA per SM): what the registers allow (fp32 at d = 128: what leaves room for two
  // ring tiles a warp).  One large CTA rather than three small: a unit that all SMs share has a third
  // of the partials to merge.
  static constexpr int W = CACHE == kFp32 && D == 128 ? 6 : NT == 2 || CACHE == kFp32 ? 8 : 12;
  // ring tiles of a warp: three (50.8 us over 128K tokens; 53.0 with four, 51.0 with two), or what there is room for
  static constexpr int ROOM = 192 * 1024 / (W * STAGE);
  static constexpr int NST = RING ? (ROOM < 3 ? ROOM : 3) : 1;
  // dynamic shared memory: the ring; over it the warps' outputs, or the weights of P parts and their outputs'
  // sums
  static size_t smem(int P) {
    return std::max({(size_t)W * NST * STAGE, (size_t)W * ROWS * D * 4, (size_t)P * ROWS * 4 + W * 32 * 16}) + 1024;
  }
};

template <typename C>
__device__ void kernel_body(const Maps& maps, const Params& p) {
  constexpr int CACHE = C::CACHE, D = C::D, NT = C::NT, ROWS = C::ROWS, ES = C::ES, RB = C::RB, NST = C::NST;
  constexpr bool F32 = C::F32, RING = C::RING, FP8 = CACHE == kE4m3, IDX = FP8 && !RING;
  static_assert(F32 ? CACHE != kBf16 : CACHE != kFp32, "bf16 cache: bf16 rows; fp32 cache: fp32 rows");
  static_assert(!RING || NST >= 2, "a ring of two tiles at least");
  static_assert(RING || FP8, "index lists: the 8-bit cache");
  constexpr int kWarps = C::W, kThreads = kWarps * 32;
  constexpr int KC = D * ES / 64;              // 16-byte chunks of a token's row that a lane takes
  constexpr int KS = D / 16;                   // k steps of S, d tiles of O
  constexpr int NQ = CACHE == kFp32 ? 3 : F32 ? 2 : 1;  // parts of a Q or P value
  constexpr int VB = D * ES / 8;               // V bytes of a token that a lane takes: 8 to 64
  using VecV = typename std::conditional<VB == 8, uint2, uint4>::type;
  constexpr int VC = VB <= 16 ? 1 : VB / 16;
  using TQ = typename std::conditional<F32, float, __nv_bfloat16>::type;

  extern __shared__ __align__(1024) unsigned char sm_raw[];
  unsigned char* const sm_base = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
  float* const sm_o = reinterpret_cast<float*>(sm_base);
  __shared__ uint64_t sm_full[RING ? kWarps : 1][NST];
  __shared__ float sm_m[3][kWarps][ROWS];
  __shared__ float sm_f[ROWS];
  __shared__ long long sm_off[ROWS];           // where the unit's rows lie in Q and O
  __shared__ int sm_scan[kWarps];
  __shared__ int sm_unit[2];
  __shared__ int sm_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int nS = p.B * p.nrg, c = blockIdx.x;
  if (RING && lane == 0) {                     // the warp's own barriers
    if (warp == 0) {
      prefetch_tensormap(&maps.k);
      prefetch_tensormap(&maps.v);
    }
#pragma unroll
    for (int i = 0; i < NST; ++i) mbar_init(&sm_full[warp][i], 1);
    fence_mbar_init();
  }
  unsigned char* const ring = sm_base + (size_t)warp * NST * C::STAGE;
  int issued = 0, used = 0;                    // tiles of the ring
  bool dead = false;                           // a wait ran out

  // ---- the units' tiles, and how the CTAs share them ------------------------------------------
  auto tiles_of = [&](int npos) { return (npos + kTile - 1) / kTile; };
  auto out_at = [&](int b, int g, int row) { return (long long)(row / p.G) * p.q_sl + b * p.q_sb + (long long)(g * p.G + row % p.G) * D; };
  auto store4 = [&](long long at, float4 x) {
    TQ* o = static_cast<TQ*>(p.O) + at;
    if constexpr (F32) *reinterpret_cast<float4*>(o) = x;
    else *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  };
  // rows that see nothing: O = 0, lse = -inf
  for (int s = c; s < nS; s += gridDim.x) {
    const Item it = item_of(p, s, ROWS);
    if (it.npos > 0) continue;
    const int nr = min(ROWS, p.R - it.rg * ROWS);
#pragma unroll 1
    for (int i = tid; i < p.Hkv * nr * (D / 4); i += kThreads) {
      const int g = i / (nr * (D / 4)), j = i % (nr * (D / 4));
      const long long at = out_at(it.b, g, it.rg * ROWS + j / (D / 4));
      store4(at + (j % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
      if (p.lse && j % (D / 4) == 0) p.lse[at / D] = -INFINITY;
    }
  }

  // CTAs c, c + 1, ... take the HG heads of the same tokens; nh heads are in the line
  const int HG = p.HG, nh = p.nh, PG = p.PG, cg = HG == 1 ? c : c / HG, gsub = c - cg * HG;
  const bool folded = nh == 1;
  const int nU = nS * nh;
  if (cg >= PG) return;
  // Two ways to share.  Whole CTAs per unit (a unit of x of all N tiles takes x PG / N of them): no CTA
  // works on two units one behind the other, and where a unit has one CTA there is nothing to
  // merge.  Taken for few units, where it leaves no CTA more than an eighth (and two rounds of
  // its warps) above N / PG; else the line of all units' tiles is cut into equal stretches.
  bool whole = false;
  int s, base = 0, r0 = 0, r1 = 1;               // item; its first tile in the line; this CTA's stretch
  int u_g = 0, u_c0 = 0, u_n = 0;                // whole: the unit's head in the line, first CTA, CTAs
  int N, P, q, rem;                              // CTA cc takes tiles [bnd(cc), bnd(cc + 1)) of N
  // no fewer tiles a CTA than worth it, but a unit does not wait for another while CTAs are idle
  auto ctas = [&]() { return min(PG, max((N + kMinTiles - 1) / kMinTiles, min(N, nU))); };
  auto bnd = [&](int cc) { return cc * q + min(cc, rem); };
  auto owner = [&](int t) { return t < rem * (q + 1) ? t / (q + 1) : rem + (t - rem * (q + 1)) / q; };
  Item it;
  constexpr bool solo = C::SOLO;
  constexpr int stride = solo ? 1 : kWarps;         // tiles from one of a warp's to its next
  if constexpr (solo) {                          // units r0, r0 + PG warps, ...
    r0 = cg * kWarps + warp;
    r1 = nU;
  } else if (nU <= 32) {                         // every warp for itself, a lane per unit
    it.npos = 0;
    if (lane < nU) it = item_of(p, folded ? lane : lane / nh, ROWS);
    const int mine = tiles_of(it.npos);
    N = warp_sum_int(mine);
    if (N == 0) return;
    // floor(mine PG / N): a quotient of floats is off by one at most
    int fair = (int)__fdividef((float)mine * PG, (float)N);
    const long long off = (long long)mine * PG - (long long)fair * N;
    fair += off < 0 ? -1 : off >= N ? 1 : 0;
    const int want = mine > 0 ? max(1, min(fair, (mine + kMinTiles - 1) / kMinTiles)) : 0;
    const int most = (int)__reduce_max_sync(0xffffffffu, want > 0 ? (unsigned)ceilf(__fdividef((float)mine, (float)want)) : 0u);
    const int pref = warp_scan_int(want, lane) - want, used = __shfl_sync(0xffffffffu, pref + want, 31);
    const float share = __fdividef((float)N, (float)PG);
    whole = used <= PG && most <= (int)(share * 1.125f) + 2 * kWarps;
    int u;
    if (whole) {
      const unsigned here = __ballot_sync(0xffffffffu, pref <= cg && cg < pref + want);
      if (here == 0) return;                     // more CTAs than wanted
      u = __ffs(here) - 1;
      s = folded ? u : u / nh;
      u_g = u - s * nh;
      u_c0 = __shfl_sync(0xffffffffu, pref, u);
      u_n = __shfl_sync(0xffffffffu, want, u);
    } else {
      P = ctas();
      q = N / P;
      rem = N - q * P;
      if (cg >= P) return;
      r0 = bnd(cg);
      r1 = bnd(cg + 1);
      const int before = warp_scan_int(mine, lane) - mine;
      u = __ffs(__ballot_sync(0xffffffffu, before <= r0 && r0 < before + mine)) - 1;
      s = u / nh;
      base = __shfl_sync(0xffffffffu, before, s * nh);
    }
    it = item_from(it, u);
  } else {                                       // a run of items per thread
    const int per = (nS + kThreads - 1) / kThreads;
    int mine = 0;
#pragma unroll 1
    for (int x = tid * per; x < min(nS, (tid + 1) * per); ++x) mine += tiles_of(item_of(p, x, ROWS).npos) * nh;
    const int scan = warp_scan_int(mine, lane);
    if (lane == 31) sm_scan[warp] = scan;
    __syncthreads();
    N = 0;
    int before = scan - mine;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm_scan[w];
      N += sm_scan[w];
    }
    if (N == 0) return;
    P = ctas();
    q = N / P;
    rem = N - q * P;
    if (cg >= P) return;
    r0 = bnd(cg);
    r1 = bnd(cg + 1);
    if (mine > 0 && before <= r0 && r0 < before + mine) {  // one thread: tile r0 is among its own
      int x = tid * per;
#pragma unroll 1
      for (;; ++x) {
        const int t = tiles_of(item_of(p, x, ROWS).npos) * nh;
        if (r0 < before + t) break;
        before += t;
      }
      sm_unit[0] = x;
      sm_unit[1] = before;
    }
    __syncthreads();
    s = sm_unit[0];
    base = sm_unit[1];
    it = item_of(p, s, ROWS);
  }

  while (r0 < r1) {
    // ---- the next unit (it, g): its tiles [t_beg, t_end); CTA groups c0 .. c0 + n - 1 share it -------
    if (solo) {
      s = folded ? r0 : r0 / nh;
      it = item_of(p, s, ROWS);
    }
    int nt_item = tiles_of(it.npos);
    int g, t_beg, t_end, c0, n;
    if (solo) {
      g = folded ? gsub : r0 - s * nh;
      c0 = t_beg = 0;
      t_end = nt_item;
      n = 1;
      r0 += PG * kWarps;
      if (nt_item == 0) continue;
    } else if (whole) {
      g = folded ? gsub : u_g;
      c0 = u_c0;
      n = u_n;
      const int qq = nt_item / n, rr = nt_item - qq * n, i = cg - c0;
      t_beg = i * qq + min(i, rr);
      t_end = t_beg + qq + (i < rr ? 1 : 0);
      r0 = r1;
    } else {
      while (r0 >= base + nt_item * nh) {
        base += nt_item * nh;
        it = item_of(p, ++s, ROWS);
        nt_item = tiles_of(it.npos);
      }
      const int x = (r0 - base) / nt_item;
      g = folded ? gsub : x;
      const int ts = base + x * nt_item, te = ts + nt_item;
      t_beg = r0 - ts;
      t_end = min(r1, te) - ts;
      c0 = owner(ts);
      n = owner(te - 1) - c0 + 1;
      r0 = min(r1, te);
    }
    const int b = it.b, row0 = it.rg * ROWS, nr = min(ROWS, p.R - row0);

    float o[NT][KS][4], l[NT][2], m[NT][2], mv[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < KS; ++j) o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
      m[nt][0] = m[nt][1] = mv[nt][0] = mv[nt][1] = kNone;
    }

    int prow[NT][2];                             // window form: positions of rows 2 tig, 2 tig + 1
    if (!FP8) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        prow[nt][0] = it.p0 + (row0 + nt * 8 + 2 * tig) / p.G;
        prow[nt][1] = it.p0 + (row0 + nt * 8 + 2 * tig + 1) / p.G;
      }
    }

    // ---- the stream: tile t of the unit into registers -------------------------------------
    const size_t seq = (size_t)(b % p.seqs);
    const size_t rstr = (size_t)p.Hkv * D * ES;
    const uint8_t* kb = static_cast<const uint8_t*>(p.K) + (seq * p.n_max * p.Hkv + g) * D * ES;
    const uint8_t* vb = static_cast<const uint8_t*>(p.V) + (seq * p.n_max * p.Hkv + g) * D * ES;
    const float* scp = FP8 ? (lane < 16 ? p.ks : p.vs) + seq * p.nblk * p.Hkv + g : nullptr;
    // token of position 16 t + lane % 16, or -1
    auto token = [&](int t) {
      const int i = t * kTile + (lane & 15);
      if (t >= t_end || i >= it.npos) return -1;
      if (IDX) {
        const int tk = __ldg(p.idx + (size_t)b * p.k + i);
        if ((unsigned)tk < (unsigned)p.n_max) return tk;
        if (lane < 16) record_error(p.ws_header, CLSA_ERR_BAD_INDEX, ((long long)b << 32) | (unsigned)i);
        return -1;
      }
      return FP8 ? i : token_of(it, i);
    };
    // byte offset of 16-byte chunk ch of token r's row in a stage (ch counts through the row)
    auto chunk = [&](int r, int ch) {
      if constexpr (RB == 64) return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
      else return (ch >> 3) * 2048 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
    };
    // the ring: tile t by TMA, 128 bytes of 16 tokens a box, swizzled by the TMA unit
    auto issue = [&](int t) {
      if (t >= t_end || dead) return;
      if (lane == 0) {
        const int slot = issued % NST;
        uint64_t* bar = &sm_full[warp][slot];
        unsigned char* dst = ring + slot * C::STAGE;
        const int i = t * kTile, row = (int)seq * p.n_max + (FP8 || i < it.keepP ? i : i + it.shift);
        mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll
        for (int x = 0; x < (RB + 127) / 128; ++x) {
          tma_load_2d(dst + 2048 * x, &maps.k, g * RB + 128 * x, row, bar);
          tma_load_2d(dst + kTile * RB + 2048 * x, &maps.v, g * RB + 128 * x, row, bar);
        }
      }
      ++issued;
    };
    uint4 kr[2][KC];                             // K: tokens gid, gid + 8
    VecV vr[4][VC];                              // V: tokens 2 tig, 2 tig + 1, + 8, + 9
    auto load_k = [&](int tok) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tk = __shfl_sync(0xffffffffu, tok, gid + 8 * h);
#pragma unroll
        for (int i = 0; i < KC; ++i)
          kr[h][i] = tk >= 0 ? ld_stream_v4(kb + (size_t)tk * rstr + 64 * i + 16 * tig) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    auto load_v = [&](int tok) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int tk = __shfl_sync(0xffffffffu, tok, 2 * tig + (h & 1) + 8 * (h >> 1));
#pragma unroll
        for (int i = 0; i < VC; ++i) {
          const uint8_t* a = vb + (size_t)max(tk, 0) * rstr + (VC == 1 ? VB * gid : 128 * i + 16 * gid);
          if constexpr (VB == 8) {
            vr[h][i] = tk >= 0 ? __ldg(reinterpret_cast<const uint2*>(a)) : make_uint2(0u, 0u);
          } else {
            vr[h][i] = tk >= 0 ? ld_stream_v4(a) : make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
    };
    auto load_scale = [&](int tok) { return FP8 && tok >= 0 ? __ldg(scp + (size_t)(tok >> p.bshift) * p.Hkv) : 1.f; };

    // ---- Q^T fragments: row gid of each row tile, the d order of the K fragments -----------
    uint32_t qb[NQ][NT][KS][2];
    float qs[NT][2];                             // score factor of rows 2 tig, 2 tig + 1
    auto load_q = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = row0 + nt * 8 + gid;
        const bool in = row < p.R;
        const TQ* q = static_cast<const TQ*>(p.Q) + (in ? out_at(b, g, row) : 0);
        if constexpr (FP8) {
          float x[KS][4];
          float mx = 0.f;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const int d0 = 64 * (ks >> 2) + 16 * tig + 4 * (ks & 3);
            if (!in) {
              x[ks][0] = x[ks][1] = x[ks][2] = x[ks][3] = 0.f;
            } else if constexpr (F32) {
              const float4 v = *reinterpret_cast<const float4*>(q + d0);
              x[ks][0] = v.x, x[ks][1] = v.y, x[ks][2] = v.z, x[ks][3] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(q + d0);
              unpack_bf16x2(v.x, x[ks][0], x[ks][1]);
              unpack_bf16x2(v.y, x[ks][2], x[ks][3]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(x[ks][e]));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          // the row's largest element to [2^13, 2^14): e its exponent (not finite: no shift)
          const int e = mx < INFINITY ? max((int)(__float_as_uint(mx) >> 23) - 127 - 13, -126) : 0;
          const float s1 = exp2_int(-e);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float lo = x[ks][2 * i] * s1, hi = x[ks][2 * i + 1] * s1;
              qb[0][nt][ks][i] = pack_f16x2(lo, hi);
              if constexpr (F32) qb[1][nt][ks][i] = rest_f16x2(qb[0][nt][ks][i], lo, hi);
            }
          }
          const float f = p.scale_log2 * exp2_int(e);
          qs[nt][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
          qs[nt][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
        } else if constexpr (CACHE == kFp32) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const float4 v = in ? *reinterpret_cast<const float4*>(q + 16 * ks + 4 * tig) : make_float4(0.f, 0.f, 0.f, 0.f);
            split3(v.x, v.y, qb[0][nt][ks][0], qb[1][nt][ks][0], qb[2][nt][ks][0]);
            split3(v.z, v.w, qb[0][nt][ks][1], qb[1][nt][ks][1], qb[2][nt][ks][1]);
          }
          qs[nt][0] = qs[nt][1] = p.scale_log2;
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint2 v = in ? *reinterpret_cast<const uint2*>(q + 32 * (ks >> 1) + 8 * tig + 4 * (ks & 1)) : make_uint2(0u, 0u);
            qb[0][nt][ks][0] = v.x;
            qb[0][nt][ks][1] = v.y;
          }
          qs[nt][0] = qs[nt][1] = p.scale_log2;
        }
      }
    };

    if constexpr (!FP8) load_q();                // before the loads: there the registers are scarce
    const int nw = solo ? kWarps : min(kWarps, t_end - t_beg);  // warps that have a tile
    int t = solo ? 0 : t_beg + warp, tok = -1, tok_n = -1;
    float sc;
    if constexpr (RING) {
#pragma unroll
      for (int x = 0; x < NST; ++x) issue(t + x * stride);
      tok = token(t);
      sc = load_scale(tok);
    } else {
      tok = token(t);
      tok_n = token(t + stride);
      if constexpr (IDX) {                       // while the indices are on their way
        if (warp < nw) load_q();
      }
      sc = load_scale(tok);
      load_k(tok);
      load_v(tok);
    }
    if constexpr (RING && FP8) {
      if (warp < nw) load_q();
    }
    if (!solo && tid < nr) sm_off[tid] = out_at(b, g, row0 + tid);
    for (; t < t_end; t += stride) {
      int tok_nn = -1;
      unsigned char* stage = nullptr;
      if constexpr (RING) {
        const int slot = used % NST;
        if (!dead && !mbar_wait_warp(&sm_full[warp][slot], (uint32_t)(used / NST) & 1u)) {
          if (lane == 0) record_error(p.ws_header, CLSA_ERR_TIMEOUT, 70);
          dead = true;
        }
        ++used;
        stage = ring + slot * C::STAGE;
        tok_n = token(t + stride);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < KC; ++i)
            kr[h][i] = *reinterpret_cast<const uint4*>(stage + chunk(gid + 8 * h, 4 * i + tig));
      } else {
        tok_nn = token(t + 2 * stride);
      }
      // S^T (fp32 rows: the first parts' products of 16 of d by themselves, added up in fp32; the others, which
      // are small, in the tensor core)
      float sa[NT][4], rest[F32 ? NT : 1][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sa[nt][0] = sa[nt][1] = sa[nt][2] = sa[nt][3] = 0.f;
        if constexpr (F32) rest[nt][0] = rest[nt][1] = rest[nt][2] = rest[nt][3] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < KC; ++i) {
        const uint32_t w0[4] = {kr[0][i].x, kr[0][i].y, kr[0][i].z, kr[0][i].w};
        const uint32_t w1[4] = {kr[1][i].x, kr[1][i].y, kr[1][i].z, kr[1][i].w};
        if constexpr (FP8) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a[4];
            e4m3x4_to_f16x4(w0[w], a[0], a[2]);
            e4m3x4_to_f16x4(w1[w], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (F32) {
                mma_f16_16816(rest[nt], a, qb[1][nt][4 * i + w][0], qb[1][nt][4 * i + w][1]);
                float t[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16_16816(t, a, qb[0][nt][4 * i + w][0], qb[0][nt][4 * i + w][1]);
                add4(sa[nt], t);
              } else {
                mma_f16_16816(sa[nt], a, qb[0][nt][4 * i + w][0], qb[0][nt][4 * i + w][1]);
              }
            }
          }
        } else if constexpr (CACHE == kFp32) {
          uint32_t a[3][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            split3_near(__uint_as_float(w0[2 * e]), __uint_as_float(w0[2 * e + 1]), a[0][2 * e], a[1][2 * e], a[2][2 * e]);
            split3_near(__uint_as_float(w1[2 * e]), __uint_as_float(w1[2 * e + 1]), a[0][2 * e + 1], a[1][2 * e + 1], a[2][2 * e + 1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 5; ++x) mma_bf16_16816(rest[nt], a[kTermA[x]], qb[kTermB[x]][nt][i][0], qb[kTermB[x]][nt][i][1]);
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma_bf16_16816(t, a[0], qb[0][nt][i][0], qb[0][nt][i][1]);
            add4(sa[nt], t);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {w0[2 * j], w1[2 * j], w0[2 * j + 1], w1[2 * j + 1]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(sa[nt], a, qb[0][nt][2 * i + j][0], qb[0][nt][2 * i + j][1]);
          }
        }
      }
      if constexpr (RING) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int r = 2 * tig + (h & 1) + 8 * (h >> 1);
#pragma unroll
          for (int i = 0; i < VC; ++i) {
            if constexpr (VB == 8) vr[h][i] = *reinterpret_cast<const uint2*>(stage + kTile * RB + chunk(r, gid >> 1) + 8 * (gid & 1));
            else vr[h][i] = *reinterpret_cast<const uint4*>(stage + kTile * RB + chunk(r, 8 * i + gid));
          }
        }
        // a tile with places that hold no token of the unit: whatever lies there, V = 0
        if (!__all_sync(0xffffffffu, tok >= 0)) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int tk = __shfl_sync(0xffffffffu, tok, 2 * tig + (h & 1) + 8 * (h >> 1));
#pragma unroll
            for (int i = 0; i < VC; ++i)
              if (tk < 0) vr[h][i] = VecV{};
          }
        }
      } else {
        load_k(tok_n);
      }
      if constexpr (F32) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) add4(sa[nt], rest[nt]);
      }
      // scores of tokens gid, gid + 8 (h) and rows 2 tig, 2 tig + 1 (x): sa[nt][2 h + x]
      const int tk[2] = {__shfl_sync(0xffffffffu, tok, gid), __shfl_sync(0xffffffffu, tok, gid + 8)};
      float kf[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f}, vf[2] = {1.f, 1.f};
      if constexpr (FP8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          kf[h] = __shfl_sync(0xffffffffu, sc, gid + 8 * h);
          const float sv = __shfl_sync(0xffffffffu, sc, 16 + gid + 8 * h);
          if constexpr (F32) {
            // vf 2^ev, 2^ev the next power of two: vf is 1 for a power of two, else in (1/2, 1), or 0 for 0
            const int e = min(max((int)(((__float_as_uint(sv) & 0x7fffffffu) + 0x7fffffu) >> 23) - 127, -126), 126);
            ev[h] = (float)e;
            vf[h] = sv * exp2_int(-e);
          } else {
            // its logarithm: whole for a power of two, else off by some 2^-21, far below a half's rounding
            ev[h] = fast_log2(sv);
          }
        }
        sc = load_scale(tok_n);
      }
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1, x = e & 1;
          float v = sa[nt][e] * (FP8 ? kf[h] * qs[nt][x] : qs[nt][x]);
          bool see = tk[h] >= 0;
          if (!FP8 && p.T > 1) {
            const int pr = prow[nt][x];
            see = see && tk[h] <= pr && (tk[h] > pr - p.window || tk[h] < p.sinks);
          }
          v = see ? v : -INFINITY;
          sa[nt][e] = v;
          up |= v > m[nt][x] + kTau;
          if (FP8) up |= v + ev[h] > mv[nt][x] + (kTau + kLift);
        }
      }
      if (__any_sync(0xffffffffu, up)) {         // some row's reference moves
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float a = fmaxf(sa[nt][x], sa[nt][2 + x]);
            float w = FP8 ? fmaxf(sa[nt][x] + ev[0], sa[nt][2 + x] + ev[1]) : a;
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
              if (FP8) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, d));
            }
            a = fmaxf(m[nt][x], a);
            l[nt][x] *= fast_exp2(m[nt][x] - a);
            m[nt][x] = a;
            w = FP8 ? fmaxf(mv[nt][x], w - kLift) : a;
            const float f = fast_exp2(mv[nt][x] - w);
            mv[nt][x] = w;
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              o[nt][j][x] *= f;
              o[nt][j][2 + x] *= f;
            }
          }
        }
      }
      // P^T, its sum, and O^T
      uint32_t pb[NQ][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float w[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float v = sa[nt][2 * h + x];
            const float e = fast_exp2(v - m[nt][x]);
            l[nt][x] += e;
            w[x] = FP8 ? fast_exp2(v + ev[h] - mv[nt][x]) : e;
            if constexpr (FP8 && F32) w[x] *= vf[h];
          }
          if constexpr (CACHE == kFp32) {
            uint32_t f[3];
            split3(w[0], w[1], f[0], f[1], f[2]);
#pragma unroll
            for (int x = 0; x < 3; ++x) pb[x][nt][h] = transpose_8x8(f[x]);
          } else {
            const uint32_t f = FP8 ? pack_f16x2(w[0], w[1]) : pack_bf16x2(w[0], w[1]);
            pb[0][nt][h] = transpose_8x8(f);
            if constexpr (F32) pb[1][nt][h] = transpose_8x8(rest_f16x2(f, w[0], w[1]));
          }
        }
      }
      auto pv = [&](int j, const uint32_t (&a)[4]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (F32) {                   // a tile by itself, small parts first
            float t[4] = {0.f, 0.f, 0.f, 0.f};
            mma_f16_16816(t, a, pb[1][nt][0], pb[1][nt][1]);
            mma_f16_16816(t, a, pb[0][nt][0], pb[0][nt][1]);
            add4(o[nt][j], t);
          } else if constexpr (FP8) {
            mma_f16_16816(o[nt][j], a, pb[0][nt][0], pb[0][nt][1]);
          } else {
            mma_bf16_16816(o[nt][j], a, pb[0][nt][0], pb[0][nt][1]);
          }
        }
      };
#pragma unroll
      for (int i = 0; i < VC; ++i) {
        const uint32_t* va = reinterpret_cast<const uint32_t*>(&vr[0][i]);
        const uint32_t* vb2 = reinterpret_cast<const uint32_t*>(&vr[1][i]);
        const uint32_t* vc = reinterpret_cast<const uint32_t*>(&vr[2][i]);
        const uint32_t* vd = reinterpret_cast<const uint32_t*>(&vr[3][i]);
        if constexpr (CACHE == kFp32) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t a[3][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              split3_near(__uint_as_float(va[2 * w + e]), __uint_as_float(vb2[2 * w + e]), a[0][e], a[1][e], a[2][e]);
              split3_near(__uint_as_float(vc[2 * w + e]), __uint_as_float(vd[2 * w + e]), a[0][2 + e], a[1][2 + e], a[2][2 + e]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int x = 0; x < 6; ++x) mma_bf16_16816(t, a[kTermA[x]], pb[kTermB[x]][nt][0], pb[kTermB[x]][nt][1]);
              add4(o[nt][2 * i + w], t);
            }
          }
        } else
#pragma unroll
        for (int w = 0; w < (int)sizeof(VecV) / 4; ++w) {
          uint32_t a[4];
          if constexpr (FP8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t sel = h ? 0x7362u : 0x5140u;
              e4m3x4_to_f16x4(__byte_perm(va[w], vb2[w], sel), a[0], a[1]);
              e4m3x4_to_f16x4(__byte_perm(vc[w], vd[w], sel), a[2], a[3]);
              pv(2 * w + h, a);
            }
          } else {
            a[0] = __byte_perm(va[w], vb2[w], 0x5410u);
            a[1] = __byte_perm(va[w], vb2[w], 0x7632u);
            a[2] = __byte_perm(vc[w], vd[w], 0x5410u);
            a[3] = __byte_perm(vc[w], vd[w], 0x7632u);
            pv(4 * i + w, a);
          }
        }
      }
      if constexpr (RING) {
        __syncwarp();                            // the stage has been used: the next tile may overwrite it
        issue(t + NST * stride);
      } else {
        load_v(tok_n);
      }
      tok = tok_n;
      tok_n = tok_nn;
    }
    if (RING && dead) {                          // loads in flight land before their memory has another use
      for (; used < issued; ++used) mbar_wait_warp(&sm_full[warp][used % NST], (uint32_t)(used / NST) & 1u);
    }
    // float4 of a row that holds a lane's d tiles j, j + 1
    auto chunk_of = [&](int j) { return FP8 ? gid * (D / 32) + j / 2 : CACHE == kBf16 ? 16 * (j >> 2) + 2 * gid + ((j & 3) >> 1) : 8 * (j >> 1) + gid; };
    // a row's outputs over its sum: x times over_sum(); -1 where it saw nothing, and then 0, not 0 * x: x is NaN
    // beside a value of another row that is not finite
    auto over_sum = [&](float M, float Mv, float L) { return L == 0.f ? -1.f : (FP8 ? exp2_gradual(Mv - M) : 1.f) / L; };
    auto times = [](float4 x, float f) {
      return f < 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    };
    auto put_lse = [&](long long at, float M, float L) {
      if (p.lse) p.lse[at / D] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    };
    if constexpr (solo) {                        // the warp has the whole unit
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], d);
          const int row = nt * 8 + 2 * tig + x;
          if (row >= nr) continue;
          const long long at = out_at(b, g, row0 + row);
          const float f = over_sum(m[nt][x], mv[nt][x], l[nt][x]);
#pragma unroll
          for (int j = 0; j < KS; j += 2)
            store4(at + chunk_of(j) * 4, times(make_float4(o[nt][j][x], o[nt][j][2 + x], o[nt][j + 1][x], o[nt][j + 1][2 + x]), f));
          if (gid == 0) put_lse(at, m[nt][x], l[nt][x]);
        }
      }
      __syncwarp();
    } else {
    if (RING) __syncthreads();                   // the warps' outputs go over the ring

    // ---- the warps' results to one -----------------------------------------------------------
    // float4 `ch` of a warp's row, placed so that neither its writers nor its readers collide
    auto so = [&](int w, int row, int ch) { return reinterpret_cast<float4*>(sm_o) + (w * ROWS + row) * (D / 4) + (ch ^ ((row >> 1) & 3)); };
    if (warp < nw) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], d);
          if (gid == 0) {
            sm_m[0][warp][nt * 8 + 2 * tig + x] = m[nt][x];
            sm_m[1][warp][nt * 8 + 2 * tig + x] = mv[nt][x];
            sm_m[2][warp][nt * 8 + 2 * tig + x] = l[nt][x];
          }
        }
#pragma unroll
        for (int j = 0; j < KS; j += 2) {          // two d tiles: 4 elements of d in a row
          const int ch = chunk_of(j);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            *so(warp, nt * 8 + 2 * tig + x, ch) = make_float4(o[nt][j][x], o[nt][j][2 + x], o[nt][j + 1][x], o[nt][j + 1][2 + x]);
        }
      }
    }
    __syncthreads();
    // float4 i of the unit's rows over the warps, with its row's references and sum
    auto warps_sum = [&](int i, float& M, float& Mv, float& L) {
      const int row = i / (D / 4);
      M = Mv = kNone;
#pragma unroll 4
      for (int w = 0; w < nw; ++w) {
        M = fmaxf(M, sm_m[0][w][row]);
        Mv = fmaxf(Mv, sm_m[1][w][row]);
      }
      L = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int w = 0; w < nw; ++w) {
        const float4 y = *so(w, row, i % (D / 4));
        const float f = fast_exp2(sm_m[1][w][row] - Mv);
        L += sm_m[2][w][row] * (FP8 ? fast_exp2(sm_m[0][w][row] - M) : f);
        x.x = fmaf(f, y.x, x.x);
        x.y = fmaf(f, y.y, x.y);
        x.z = fmaf(f, y.z, x.z);
        x.w = fmaf(f, y.w, x.w);
      }
      return x;
    };
    auto lse_of = [&](int row, float M, float L) { put_lse(sm_off[row], M, L); };
    const int tasks = nr * (D / 4);              // float4s of the unit's rows
    if (n == 1) {
#pragma unroll 1
      for (int i = tid; i < tasks; i += kThreads) {
        float M, Mv, L;
        const float4 x = warps_sum(i, M, Mv, L);
        store4(sm_off[i / (D / 4)] + (i % (D / 4)) * 4, times(x, over_sum(M, Mv, L)));
        if (i % (D / 4) == 0) lse_of(i / (D / 4), M, L);
      }
      if (RING) fence_proxy_async_smem();        // before the next unit's TMA writes
      __syncthreads();                           // shared memory is free again
      continue;
    }
    // slot 1 of a CTA: the unit that begins in its stretch and goes on behind it (at most one);
    // slot 0: the unit that began before it
    float* const part0 = p.part + (size_t)(2 * (c0 * HG + gsub)) * slot_floats<D, NT>();
    const int step = 2 * HG * slot_floats<D, NT>();
    const auto slot = [&](int i) { return part0 + (i * step + (i == 0 ? slot_floats<D, NT>() : 0)); };
    float* my = slot(cg - c0);
#pragma unroll 1
    for (int i = tid; i < tasks; i += kThreads) {
      float M, Mv, L;
      __stcg(reinterpret_cast<float4*>(my) + i, warps_sum(i, M, Mv, L));
      if (i % (D / 4) == 0) {
        float* x = my + ROWS * D + i / (D / 4);
        __stcg(x, M);
        __stcg(x + ROWS, Mv);
        __stcg(x + 2 * ROWS, L);
      }
    }
    // the merge: S threads per float4, each for every S-th part, kB loads in flight
    constexpr int kB = 8;
    const int S = tasks < kThreads ? min(kThreads / tasks, n) : 1, sl = S > 1 ? tid / tasks : 0, i0 = tid - sl * tasks;
    uint32_t* ctr = p.counter + (size_t)s * p.Hkv + g;
    __syncthreads();  // every thread's part is stored before the arrival, which releases them
    if (tid == 0) sm_last = atom_add_acq_rel_gpu(ctr, 1u) == (uint32_t)(n - 1);
    __syncthreads();
    if (sm_last) {      // the others' parts, released before their arrivals
      float* const wt = sm_o;                    // [n][ROWS]: the parts' weights
      float4* const sums = reinterpret_cast<float4*>(sm_o + (n * ROWS + 3) / 4 * 4);
      float4 y[kB];
      auto fetch = [&](int i, int j0) {
#pragma unroll
        for (int j = 0; j < kB; ++j) y[j] = __ldcg(reinterpret_cast<const float4*>(slot(min(j0 + j * S, n - 1))) + i);
      };
      if (sl < S && i0 < tasks) fetch(i0, sl);
      // a warp's rows (two at most), a lane per part
      constexpr int RW = (ROWS + kWarps - 1) / kWarps;
      float M[RW], Mv[RW], L[RW];
#pragma unroll
      for (int x = 0; x < RW; ++x) {
        M[x] = Mv[x] = kNone;
        L[x] = 0.f;
      }
#pragma unroll 1
      for (int i = lane; i < n; i += 32) {
        float mi[RW], vi[RW], li[RW];
#pragma unroll
        for (int x = 0; x < RW; ++x) {
          const float* v = slot(i) + ROWS * D + min(warp + x * kWarps, nr - 1);
          mi[x] = __ldcg(v), vi[x] = __ldcg(v + ROWS), li[x] = __ldcg(v + 2 * ROWS);
        }
#pragma unroll
        for (int x = 0; x < RW; ++x) {
          const float top = fmaxf(M[x], mi[x]);
          L[x] = L[x] * fast_exp2(M[x] - top) + li[x] * fast_exp2(mi[x] - top);
          M[x] = top;
          Mv[x] = fmaxf(Mv[x], vi[x]);
          if (warp + x * kWarps < nr) wt[i * ROWS + warp + x * kWarps] = vi[x];
        }
      }
      float top[RW];
#pragma unroll
      for (int x = 0; x < RW; ++x) top[x] = warp_max(M[x]);
#pragma unroll
      for (int x = 0; x < RW; ++x) Mv[x] = warp_max(Mv[x]);
#pragma unroll
      for (int x = 0; x < RW; ++x) L[x] = warp_sum(L[x] * fast_exp2(M[x] - top[x]));
#pragma unroll
      for (int x = 0; x < RW; ++x) {
        const int row = warp + x * kWarps;
        if (row < nr) {
          for (int i = lane; i < n; i += 32) wt[i * ROWS + row] = fast_exp2(wt[i * ROWS + row] - Mv[x]);
          if (lane == 0) {
            sm_f[row] = over_sum(top[x], Mv[x], L[x]);
            lse_of(row, top[x], L[x]);
          }
        }
      }
      __syncthreads();
      if (sl < S) {
#pragma unroll 1
        for (int i = i0; i < tasks; i += kThreads) {
          const int row = i / (D / 4);
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int j0 = sl; j0 < n; j0 += kB * S) {
            if (i != i0 || j0 != sl) fetch(i, j0);
#pragma unroll
            for (int j = 0; j < kB; ++j) {
              if (j0 + j * S < n) {
                const float w = wt[(j0 + j * S) * ROWS + row];
                x.x = fmaf(w, y[j].x, x.x);
                x.y = fmaf(w, y[j].y, x.y);
                x.z = fmaf(w, y[j].z, x.z);
                x.w = fmaf(w, y[j].w, x.w);
              }
            }
          }
          x = times(x, sm_f[row]);
          if (S > 1) sums[sl * tasks + i] = x;
          else store4(sm_off[row] + (i % (D / 4)) * 4, x);
        }
      }
      if (S > 1) {
        __syncthreads();
        if (tid < tasks) {
          float4 x = sums[tid];
          for (int j = 1; j < S; ++j) {
            const float4 z = sums[j * tasks + tid];
            x.x += z.x, x.y += z.y, x.z += z.z, x.w += z.w;
          }
          store4(sm_off[tid / (D / 4)] + (tid % (D / 4)) * 4, x);
        }
      }
      if (tid == 0) *ctr = 0u;  // clean for the next call
    }
    if (RING) fence_proxy_async_smem();
    __syncthreads();
    }
  }
}

template <typename C>
__global__ void __launch_bounds__(C::W * 32, 1) stream_attn_kernel(const __grid_constant__ Maps maps, const Params p) {
  pdl_enter();
  kernel_body<C>(maps, p);
}

inline size_t counter_bytes(const Params& p) { return align_up((size_t)p.B * p.nrg * p.Hkv * 4, 256); }

// the most tiles that a unit can have
inline int most_tiles(const Params& p, int rows) {
  long long seen = p.idx ? p.k : p.n_max;
  if (p.T > 0) seen = std::min<long long>(seen, (long long)p.window + p.sinks + (rows - 1) / p.G + kTile);
  return (int)((seen + kTile - 1) / kTile);
}

// the row groups of R rows: one or two row tiles
inline int row_tiles(int R, bool f32) { return R <= 8 || f32 ? 1 : 2; }

// 2-D map of bytes [rows][row_bytes], boxes of 16 rows and up to 128 bytes
inline bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t row_bytes, uint32_t box_bytes) {
  const TmapEncodeFn fn = tmap_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {row_bytes, rows}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_bytes, kTile}, es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            box_bytes == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename C>
size_t ws_bytes(const Params& p) {
  const int P = std::max(1, device_info().sm_count);
  return counter_bytes(p) + (size_t)2 * P * slot_floats<C::D, C::NT>() * 4;
}

template <typename C>
cudaError_t launch_as(Params& p, cudaStream_t s) {
  const int P = std::max(1, device_info().sm_count);
  Maps maps{};
  if (C::RING) {
    const uint64_t rows = (uint64_t)p.seqs * p.n_max, bytes = (uint64_t)p.Hkv * C::RB;
    if (!make_map(&maps.k, p.K, rows, bytes, std::min(C::RB, 128)) || !make_map(&maps.v, p.V, rows, bytes, std::min(C::RB, 128)))
      return cudaErrorInvalidValue;
  }
  const size_t smem = C::smem(P);
  cudaError_t e = cudaFuncSetAttribute(stream_attn_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch_pdl(stream_attn_kernel<C>, dim3(P), dim3(C::W * 32), smem, s, maps, p);
  launches_add(1, s);
  return e;
}

template <typename C>
cudaError_t launch(Params p, void* ws_body, cudaStream_t s) {
  const int P = std::max(1, device_info().sm_count);
  p.counter = static_cast<uint32_t*>(ws_body);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws_body) + counter_bytes(p));
  // Heads side by side, so that the cache's rows, which hold all heads, are read whole at about the same
  // time.  Only where few CTAs stay idle for it.
  p.HG = p.Hkv <= P && (P % p.Hkv) * 16 <= P ? p.Hkv : 1;
  p.nh = p.Hkv / p.HG;
  p.PG = P / p.HG;
  // More units than CTAs: a unit per warp, unless its rounds fit the warps badly.  Besides its tiles, a
  // warp's share of HBM each, a unit is taken to cost a CTA 6.5 us and a warp 3 (fitted; a CTA's lie between 3.6, short
  // units, and 6).  A unit per warp and per CTA, us, 32 heads on 8, d = 128: 8-bit cache, 900 sequences of 512 tokens
  // 180 and 330; 900 of 64 42 and 183; 200 of 1000 72 and 119; 40 of 1000 68 and 36; 64 of 4096 258 and 108; bf16
  // windows of 300, T = 4, 200 sequences 68 and 106; fp32 windows, T = 2048, W = 1024 1390 and 1592, W = 64 158 and 334,
  // 8 heads on 2 (1.7 rounds) 559 and 403.  All chosen right; not so 40 sequences of 200 tokens: 18 and 25, by CTAs.
  const double units = (double)p.B * p.nrg * p.nh, rounds = units / ((double)p.PG * C::W);
  const double tiles_us = most_tiles(p, C::ROWS) * (C::STAGE * C::W / 44e3);
  const bool solo = units > p.PG && std::ceil(rounds) * (3 + tiles_us) < rounds * (6.5 * C::W + tiles_us);
  return solo ? launch_as<typename C::Solo>(p, s) : launch_as<C>(p, s);
}

}  // namespace stream
}  // namespace clsa
