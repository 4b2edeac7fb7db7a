// Streaming attention of few query rows over many cached tokens, shared by the 8-bit cache's
// attention and by window attention's decode form (bf16 cache):
//   O[r] = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(q_r . k_j * scale),  j over the tokens r sees.
//
// What bounds it is moving K and V: with G query heads per KV head a byte of the cache feeds 2 G
// multiplies.  So every warp is a stream of its own, with no barrier in its loop: it takes
// tiles of 16 tokens, loads K and V straight into the registers that feed the tensor core
// (mma.sync m16n8k16; a 128-row tcgen05 tile would be empty for G = 4), keeps a running
// maximum, sum and output for its rows, and issues the next tile's loads as soon as the
// registers are free.  Nothing of the cache passes through shared memory.
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
// block of small scale.  With fp32 queries Q and P are split into two halves each (22 bits).
// fp32 cache.  Every factor is the exact sum of three bf16 parts; six of the nine products
// of parts are formed (the others are below 2^-24).
//
// The reference (of sums and of outputs) moves only when a score exceeds it by 2^8; then the
// sums are rescaled.  A row's largest p is at least 2^0, at most 2^8: no overflow.  Where p becomes
// halves it is 2^7 larger still (halves end at 2^16), so that the halves' smallest step, 2^-24,
// is 2^-31 of the largest.
//
// Work split.  A unit is a (sequence, row group, KV head).  Few units of like length get whole CTAs
// each; else all units' tiles form one line that the CTAs share equally, so ragged lengths
// balance.  A unit that several CTAs share is merged by the one that arrives last, in CTA
// order (the result does not depend on who that is).
#pragma once

#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"

namespace clsa {
namespace stream {

constexpr int kTile = 16;                   // tokens of a tile
constexpr int kMinTiles = 4;                // fewest tiles worth a CTA
constexpr int kAhead = 4;                   // tiles of a warp between its L2 prefetch and its loads
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
  int T, window, sinks;     // T > 0: row r is the token count - T + r / G and sees a window and the sinks
  float scale_log2;
};

// a (sequence, row group): which tokens its rows see between them
struct Item {
  int b, rg, npos;          // npos positions; position i is token i (i < keep) or i + shift
  int keep, shift, p0;      // p0: position of row 0 (window form)
};

__device__ __forceinline__ Item item_of(const Params& p, int s, int rows) {
  Item it;
  it.b = s / p.nrg;
  it.rg = s - it.b * p.nrg;
  const int cnt = p.count[it.b];
  it.p0 = 0;
  if (p.T == 0) {
    it.npos = max(0, min(cnt, p.idx ? p.k : p.n_max));
    it.keep = it.npos;
    it.shift = 0;
    return it;
  }
  const int len = max(0, min(cnt, p.n_max));
  const int r0 = it.rg * rows, r1 = min(r0 + rows, p.R) - 1;
  it.p0 = len - p.T;
  const int first = it.p0 + r0 / p.G, last = it.p0 + r1 / p.G;
  if (last < 0) {
    it.npos = it.keep = it.shift = 0;
    return it;
  }
  const int lo = max(0, first - p.window + 1);
  it.keep = min(p.sinks, lo);
  it.shift = lo - it.keep;
  it.npos = it.keep + last + 1 - lo;
  return it;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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
// the products of parts that reach 2^-24 of the whole, small ones first
__device__ constexpr int kTermA[6] = {2, 0, 1, 1, 0, 0};
__device__ constexpr int kTermB[6] = {0, 2, 1, 0, 1, 0};

template <int D, int NT>
constexpr int slot_floats() { return NT * 8 * (D + 3); }

// warps of a CTA (one CTA per SM): what the registers allow, 168 or 255 a thread.  One large CTA
// rather than three small: a unit that all SMs share has a third of the partials to merge.
template <int CACHE, int NT>
__host__ __device__ constexpr int warps_of() { return NT == 1 && CACHE != kFp32 ? 12 : 8; }

// shared memory: the warps' outputs, or the weights of up to P contributors
template <int CACHE, int D, int NT>
__host__ __device__ constexpr size_t smem_bytes(int P) {
  const size_t o = (size_t)warps_of<CACHE, NT>() * NT * 8 * D * 4, w = (size_t)P * NT * 8 * 4;
  return o > w ? o : w;
}

template <int CACHE, bool F32, int D, int NT>
__device__ void kernel_body(const Params& p) {
  static_assert(F32 ? CACHE != kBf16 : CACHE != kFp32, "bf16 cache: bf16 rows; fp32 cache: fp32 rows");
  constexpr bool FP8 = CACHE == kE4m3;
  constexpr int kWarps = warps_of<CACHE, NT>(), kThreads = kWarps * 32;
  constexpr int ROWS = NT * 8;
  constexpr int ES = FP8 ? 1 : CACHE == kBf16 ? 2 : 4;  // bytes of a cache element
  constexpr int KC = D * ES / 64;              // 16-byte chunks of a token's row that a lane takes
  constexpr int KS = D / 16;                   // k steps of S, d tiles of O
  constexpr int NQ = CACHE == kFp32 ? 3 : F32 ? 2 : 1;  // parts of a Q or P value
  constexpr int VB = D * ES / 8;               // V bytes of a token that a lane takes: 8 to 64
  using VecV = typename std::conditional<VB == 8, uint2, uint4>::type;
  constexpr int VC = VB <= 16 ? 1 : VB / 16;
  using TQ = typename std::conditional<F32, float, __nv_bfloat16>::type;

  extern __shared__ __align__(16) float sm_o[];
  __shared__ float sm_m[3][kWarps][ROWS];
  __shared__ float sm_f[ROWS];
  __shared__ long long sm_off[ROWS];           // where the unit's rows lie in Q and O
  __shared__ int sm_scan[2][kWarps];
  __shared__ int sm_top[kWarps];
  __shared__ int sm_unit[4];
  __shared__ int sm_last;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int nS = p.B * p.nrg, c = blockIdx.x;

  // ---- the units' tiles, and how the CTAs share them ------------------------------------------
  auto tiles_of = [&](int npos) { return (npos + kTile - 1) / kTile; };
  // sum of x over the threads, and over those before this one (two in turn: sm_scan has two rows)
  auto block_scan = [&](int row, int x, int& before) {
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    if (lane == 31) sm_scan[row][warp] = v;
    __syncthreads();
    int sum = 0;
    before = v - x;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sm_scan[row][w];
      sum += sm_scan[row][w];
    }
    return sum;
  };
  const int nU = nS * p.Hkv;
  const bool few = nU <= (int)gridDim.x && nU <= kThreads;  // a thread per unit; else a run of items per thread
  const int per = (nS + kThreads - 1) / kThreads;
  int mine = 0, before;
  if (few) {
    if (tid < nU) mine = tiles_of(item_of(p, tid / p.Hkv, ROWS).npos);
  } else {
    for (int s = tid * per; s < min(nS, (tid + 1) * per); ++s) mine += tiles_of(item_of(p, s, ROWS).npos) * p.Hkv;
  }
  const int N = block_scan(0, mine, before);

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
    for (int i = tid; i < p.Hkv * nr * (D / 4); i += kThreads) {
      const int g = i / (nr * (D / 4)), j = i % (nr * (D / 4));
      const long long at = out_at(it.b, g, it.rg * ROWS + j / (D / 4));
      store4(at + (j % (D / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
      if (p.lse && j % (D / 4) == 0) p.lse[at / D] = -INFINITY;
    }
  }
  if (N == 0) return;

  // Two ways to share.  Whole CTAs per unit (a unit of x tiles takes x / q of them, q = tiles a CTA):
  // no CTA works on two units one behind the other, and where a unit has one CTA there is
  // nothing to merge.  Taken where it leaves no CTA more than an eighth (and two rounds of
  // its warps) above q; else the line of all tiles is cut into equal stretches.
  const int q0 = (N + (int)gridDim.x - 1) / (int)gridDim.x;
  bool whole = few;
  if (few) {
    const int want = mine > 0 ? max(1, min(mine / q0, (mine + kMinTiles - 1) / kMinTiles)) : 0;
    const int load = want > 0 ? (mine + want - 1) / want : 0;
    const int top = (int)__reduce_max_sync(0xffffffffu, (unsigned)load);
    if (lane == 0) sm_top[warp] = top;
    int pref;
    const int used = block_scan(1, want, pref);
    int most = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) most = max(most, sm_top[w]);
    whole = used <= (int)gridDim.x && most <= q0 + q0 / 8 + 2 * kWarps;
    if (whole) {
      if (c >= used) return;
      if (pref <= c && c < pref + want) {
        sm_unit[0] = tid;
        sm_unit[1] = pref;
        sm_unit[2] = want;
      }
    }
  }
  // the line: CTA cc takes tiles [bnd(cc), bnd(cc + 1))
  const int P = min((int)gridDim.x, (N + kMinTiles - 1) / kMinTiles);
  const int q = N / P, rem = N - q * P;
  auto bnd = [&](int cc) { return cc * q + min(cc, rem); };
  auto owner = [&](int t) { return t < rem * (q + 1) ? t / (q + 1) : rem + (t - rem * (q + 1)) / q; };
  int r0 = 0, r1 = 1;
  if (!whole) {
    if (c >= P) return;
    r0 = bnd(c);
    r1 = bnd(c + 1);
    if (mine > 0 && before <= r0 && r0 < before + mine) {  // one thread: tile r0 is among its own
      int base = before, s = few ? tid / p.Hkv : tid * per;
      if (few) {
        base -= (tid % p.Hkv) * mine;                      // the item's first unit
      } else {
        for (;; ++s) {
          const int t = tiles_of(item_of(p, s, ROWS).npos) * p.Hkv;
          if (r0 < base + t) break;
          base += t;
        }
      }
      sm_unit[0] = s;
      sm_unit[1] = base;
    }
  }
  __syncthreads();
  int s = whole ? sm_unit[0] / p.Hkv : sm_unit[0], base = sm_unit[1];
  Item it = item_of(p, s, ROWS);

  while (r0 < r1) {
    // ---- the next unit (it, g): its tiles [t_beg, t_end); CTAs c0 .. c0 + n - 1 share it -------
    int nt_item = tiles_of(it.npos);
    int g, t_beg, t_end, c0, n;
    if (whole) {
      g = sm_unit[0] - s * p.Hkv;
      c0 = sm_unit[1];
      n = sm_unit[2];
      const int qq = nt_item / n, rr = nt_item - qq * n, i = c - c0;
      t_beg = i * qq + min(i, rr);
      t_end = t_beg + qq + (i < rr ? 1 : 0);
      r0 = r1;
    } else {
      while (r0 >= base + nt_item * p.Hkv) {
        base += nt_item * p.Hkv;
        it = item_of(p, ++s, ROWS);
        nt_item = tiles_of(it.npos);
      }
      g = (r0 - base) / nt_item;
      const int ts = base + g * nt_item, te = ts + nt_item;
      t_beg = r0 - ts;
      t_end = min(r1, te) - ts;
      c0 = owner(ts);
      n = owner(te - 1) - c0 + 1;
      r0 = min(r1, te);
    }
    const int b = it.b, row0 = it.rg * ROWS, nr = min(ROWS, p.R - row0);
    if (tid < nr) sm_off[tid] = out_at(b, g, row0 + tid);

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
      if (FP8 && p.idx) {
        const int tk = __ldg(p.idx + (size_t)b * p.k + i);
        if ((unsigned)tk < (unsigned)p.n_max) return tk;
        if (lane < 16) record_error(p.ws_header, CLSA_ERR_BAD_INDEX, ((long long)b << 32) | (unsigned)i);
        return -1;
      }
      return i < it.keep ? i : i + it.shift;
    };
    uint4 kr[2][KC];
    VecV vr[4][VC];
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

    // the tokens' lines of tile t on their way into L2 (a lane per row; selections are small)
    auto ahead = [&](int t) {
      const int i = t * kTile + (lane & 15);
      if ((FP8 && p.idx) || t >= t_end || i >= it.npos) return;
      const uint8_t* a = (lane < 16 ? kb : vb) + (size_t)(i < it.keep ? i : i + it.shift) * rstr;
#pragma unroll
      for (int x = 0; x < (D * ES + 127) / 128; ++x) asm volatile("prefetch.global.L2 [%0];" ::"l"(a + 128 * x));
    };

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
          // the row's largest element to [2^13, 2^14): e its exponent (zero or not finite: no shift)
          const int e = (mx > 0.f && mx < INFINITY) ? (int)(__float_as_uint(mx) >> 23) - 127 - 13 : 0;
          const int h1 = (-e) >> 1, h2 = -e - h1;    // in two steps: 2^-e may lie outside the floats
          const float s1 = exp2_int(h1), s2 = exp2_int(h2);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float lo = x[ks][2 * i] * s1 * s2, hi = x[ks][2 * i + 1] * s1 * s2;
              qb[0][nt][ks][i] = pack_f16x2(lo, hi);
              if constexpr (F32) qb[1][nt][ks][i] = rest_f16x2(qb[0][nt][ks][i], lo, hi);
            }
          }
          const float f = p.scale_log2 * exp2_int(-h1) * exp2_int(-h2);
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
    int t = t_beg + warp;
#pragma unroll
    for (int x = 1; x < kAhead; ++x) ahead(t + x * kWarps);
    int tok = token(t), tok_n = token(t + kWarps);
    float sc = load_scale(tok);
    load_k(tok);
    load_v(tok);

    if constexpr (FP8) load_q();
    for (; t < t_end; t += kWarps) {
      const int tok_nn = token(t + 2 * kWarps);
      ahead(t + kAhead * kWarps);
      // S^T
      float sa[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sa[nt][0] = sa[nt][1] = sa[nt][2] = sa[nt][3] = 0.f;
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
#pragma unroll
              for (int x = 0; x < NQ; ++x) mma_f16_16816(sa[nt], a, qb[x][nt][4 * i + w][0], qb[x][nt][4 * i + w][1]);
            }
          }
        } else if constexpr (CACHE == kFp32) {
          uint32_t a[3][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            split3(__uint_as_float(w0[2 * e]), __uint_as_float(w0[2 * e + 1]), a[0][2 * e], a[1][2 * e], a[2][2 * e]);
            split3(__uint_as_float(w1[2 * e]), __uint_as_float(w1[2 * e + 1]), a[0][2 * e + 1], a[1][2 * e + 1], a[2][2 * e + 1]);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 6; ++x) mma_bf16_16816(sa[nt], a[kTermA[x]], qb[kTermB[x]][nt][i][0], qb[kTermB[x]][nt][i][1]);
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
      load_k(tok_n);
      // scores of tokens gid, gid + 8 (h) and rows 2 tig, 2 tig + 1 (x): sa[nt][2 h + x]
      const int tk[2] = {__shfl_sync(0xffffffffu, tok, gid), __shfl_sync(0xffffffffu, tok, gid + 8)};
      float kf[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f};
      if constexpr (FP8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          kf[h] = __shfl_sync(0xffffffffu, sc, gid + 8 * h);
          // the value scale 2^e: e from its exponent bits
          ev[h] = (float)((int)((__float_as_uint(__shfl_sync(0xffffffffu, sc, 16 + gid + 8 * h)) >> 23) & 255u) - 127);
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
          if constexpr (FP8) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) mma_f16_16816(o[nt][j], a, pb[x][nt][0], pb[x][nt][1]);
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
              split3(__uint_as_float(va[2 * w + e]), __uint_as_float(vb2[2 * w + e]), a[0][e], a[1][e], a[2][e]);
              split3(__uint_as_float(vc[2 * w + e]), __uint_as_float(vd[2 * w + e]), a[0][2 + e], a[1][2 + e], a[2][2 + e]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int x = 0; x < 6; ++x) mma_bf16_16816(o[nt][2 * i + w], a[kTermA[x]], pb[kTermB[x]][nt][0], pb[kTermB[x]][nt][1]);
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
      load_v(tok_n);
      tok = tok_n;
      tok_n = tok_nn;
    }

    // ---- the warps' results to one -----------------------------------------------------------
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
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float top = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[1][w][nt * 8 + 2 * tig + x]);
        f[x] = fast_exp2(mv[nt][x] - top);
      }
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const int d0 = FP8 ? gid * (D / 8) + 2 * j
                           : CACHE == kBf16 ? 64 * (j >> 2) + 8 * gid + 2 * (j & 3) : 32 * (j >> 1) + 4 * gid + 2 * (j & 1);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          *reinterpret_cast<float2*>(sm_o + ((size_t)warp * ROWS + nt * 8 + 2 * tig + x) * D + d0) =
              make_float2(o[nt][j][x] * f[x], o[nt][j][2 + x] * f[x]);
      }
    }
    __syncthreads();
    auto row_stats = [&](int row, float& M, float& Mv, float& L) {
      M = Mv = kNone;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M = fmaxf(M, sm_m[0][w][row]);
        Mv = fmaxf(Mv, sm_m[1][w][row]);
      }
      L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) L += sm_m[2][w][row] * fast_exp2(sm_m[0][w][row] - M);
    };
    auto warps_sum = [&](int i) {  // float4 i of the unit's rows, over the warps
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(sm_o + (size_t)w * ROWS * D + 4 * i);
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
      }
      return x;
    };
    auto lse_of = [&](int row, float M, float L) {
      if (p.lse) p.lse[sm_off[row] / D] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    };
    if (n == 1) {
      for (int i = tid; i < nr * (D / 4); i += kThreads) {
        const int row = i / (D / 4);
        float M, Mv, L;
        row_stats(row, M, Mv, L);
        const float f = L == 0.f ? 0.f : (FP8 ? exp2f(Mv - M) : 1.f) / L;
        float4 x = warps_sum(i);
        x.x *= f, x.y *= f, x.z *= f, x.w *= f;
        store4(sm_off[row] + (i % (D / 4)) * 4, x);
        if (i % (D / 4) == 0) lse_of(row, M, L);
      }
      __syncthreads();  // shared memory is free again
      continue;
    }
    // slot 1 of a CTA: the unit that begins in its stretch and goes on behind it (at most one);
    // slot 0: the unit that began before it
    const auto slot = [&](int i) { return p.part + (size_t)(2 * (c0 + i) + (i == 0 ? 1 : 0)) * slot_floats<D, NT>(); };
    float* my = slot(c - c0);
    for (int i = tid; i < ROWS * (D / 4); i += kThreads) __stcg(reinterpret_cast<float4*>(my) + i, warps_sum(i));
    if (tid < ROWS) {
      float M, Mv, L;
      row_stats(tid, M, Mv, L);
      __stcg(my + ROWS * D + tid, M);
      __stcg(my + ROWS * (D + 1) + tid, Mv);
      __stcg(my + ROWS * (D + 2) + tid, L);
    }
    uint32_t* ctr = p.counter + (size_t)s * p.Hkv + g;
    __syncthreads();  // every thread's part is stored before the arrival, which releases them
    if (tid == 0) sm_last = atom_add_acq_rel_gpu(ctr, 1u) == (uint32_t)(n - 1);
    __syncthreads();
    if (sm_last) {      // the others' parts, released before their arrivals
      constexpr int kB = 16;  // loads in flight
      float4 y[kB];
      auto fetch = [&](int i, int j0) {
#pragma unroll
        for (int j = 0; j < kB; ++j) y[j] = __ldcg(reinterpret_cast<const float4*>(slot(min(j0 + j, n - 1))) + i);
      };
      if (tid < nr * (D / 4)) fetch(tid, 0);
      for (int row = warp; row < nr; row += kWarps) {
        float M = kNone, Mv = kNone, L = 0.f;
        for (int i = lane; i < n; i += 32) {
          const float* x = slot(i) + ROWS * D + row;
          const float mi = __ldcg(x), vi = __ldcg(x + ROWS), li = __ldcg(x + 2 * ROWS);
          const float top = fmaxf(M, mi);
          L = L * fast_exp2(M - top) + li * fast_exp2(mi - top);
          M = top;
          Mv = fmaxf(Mv, vi);
          sm_o[i * ROWS + row] = vi;
        }
        const float top = warp_max(M);
        L = warp_sum(L * fast_exp2(M - top));
        Mv = warp_max(Mv);
        for (int i = lane; i < n; i += 32) sm_o[i * ROWS + row] = fast_exp2(sm_o[i * ROWS + row] - Mv);
        if (lane == 0) {
          sm_f[row] = L == 0.f ? 0.f : (FP8 ? exp2f(Mv - top) : 1.f) / L;
          lse_of(row, top, L);
        }
      }
      __syncthreads();
      for (int i = tid; i < nr * (D / 4); i += kThreads) {
        const int row = i / (D / 4);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j0 = 0; j0 < n; j0 += kB) {
          if (i != tid || j0 > 0) fetch(i, j0);
#pragma unroll
          for (int j = 0; j < kB; ++j) {
            if (j0 + j < n) {
              const float w = sm_o[(j0 + j) * ROWS + row];
              x.x = fmaf(w, y[j].x, x.x);
              x.y = fmaf(w, y[j].y, x.y);
              x.z = fmaf(w, y[j].z, x.z);
              x.w = fmaf(w, y[j].w, x.w);
            }
          }
        }
        const float f = sm_f[row];
        x.x *= f, x.y *= f, x.z *= f, x.w *= f;
        store4(sm_off[row] + (i % (D / 4)) * 4, x);
      }
      if (tid == 0) *ctr = 0u;  // clean for the next call
    }
    __syncthreads();
  }
}

template <int CACHE, bool F32, int D, int NT>
__global__ void __launch_bounds__(warps_of<CACHE, NT>() * 32, 1) stream_attn_kernel(const Params p) {
  pdl_enter();
  kernel_body<CACHE, F32, D, NT>(p);
}

inline size_t counter_bytes(const Params& p) { return align_up((size_t)p.B * p.nrg * p.Hkv * 4, 256); }

// the row groups of R rows: one or two row tiles
inline int row_tiles(int R, bool f32) { return R <= 8 || f32 ? 1 : 2; }

template <int CACHE, bool F32, int D, int NT>
size_t ws_bytes(const Params& p) {
  const int P = std::max(1, device_info().sm_count);
  return counter_bytes(p) + (size_t)2 * P * slot_floats<D, NT>() * 4;
}

template <int CACHE, bool F32, int D, int NT>
cudaError_t launch(Params p, void* ws_body, cudaStream_t s) {
  const int P = std::max(1, device_info().sm_count);
  p.counter = static_cast<uint32_t*>(ws_body);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws_body) + counter_bytes(p));
  const size_t smem = smem_bytes<CACHE, D, NT>(P);
  auto* k = stream_attn_kernel<CACHE, F32, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) e = launch_pdl(k, dim3(P), dim3(warps_of<CACHE, NT>() * 32), smem, s, p);
  launches_add(1, s);
  return e;
}

}  // namespace stream
}  // namespace clsa
