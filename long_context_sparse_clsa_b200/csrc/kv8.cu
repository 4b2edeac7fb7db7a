// The 8-bit K/V cache: quantising rows as they are written, and reading rows back.
//
// A cache [n][Hkv][d] holds e4m3 codes; each block of `block` tokens and head has a scale
//   s = the smallest power of two >= 2^-100 with max |x| / s <= 448    (at most 2^119)
// and a code stands for code * s.  e4m3 is a floating format, so its relative step (2^-3 of
// the binade) does not depend on s: a power of two loses nothing against max|x| / 448.  It
// gains that x / s is exact, and that codes already in a block are only shifted when a
// larger row joins it: code * (s_old / s_new) is exact but where it becomes subnormal, so a
// cache filled token by token holds what one filled at once holds, up to those.
//
// Both kernels move bytes: HBM (long runs) or launch latency (a decode step) is the bound.
#include <algorithm>
#include <cmath>

#include "fp8.cuh"
#include "kernels.h"
#include "vec32.cuh"

namespace clsa {

namespace {

constexpr int kThreadsW = 256;

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t finite_abs_bits(float x) { return abs_bits(x) < 0x7f800000u ? abs_bits(x) : 0u; }
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)f32x2_to_e4m3x2(a, b) | ((uint32_t)f32x2_to_e4m3x2(c, d) << 16);
}

// 16 elements of a row: their largest |x| as a float's bits (at least 0x7f800000 where one is not finite),
// the largest among the finite ones, and the codes of x * inv (inv a power of two)
template <typename T> struct Load16;
template <> struct Load16<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool) {  // 32-byte loads took the same time or more
    v[0] = ld_stream_v4(p);
    v[1] = ld_stream_v4(p + 8);
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4& q = v[i >> 2];
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
  __device__ __forceinline__ uint32_t amax() const {  // two at a time
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(word(i) & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
  }
  __device__ __forceinline__ uint32_t amax_finite() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      unpack_bf16x2(word(i), a, b);
      m = max(m, max(finite_abs_bits(a), finite_abs_bits(b)));
    }
    return m;
  }
  // the products are exact in bf16 but below 2^-126, where the code is 0 anyway
  __device__ __forceinline__ uint4 codes(float inv) const {
    const uint32_t i2 = pack_bf16x2(inv, inv);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t x, y;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(word(2 * e)), "r"(i2));
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(word(2 * e + 1)), "r"(i2));
      float a, b, c, d;
      unpack_bf16x2(x, a, b);
      unpack_bf16x2(y, c, d);
      w[e] = e4m3x4(a, b, c, d);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Load16<float> {
  uint4 v[4];
  __device__ __forceinline__ void load(const float* p, bool wide) {
    ld_stream_32(p, v[0], v[1], wide);
    ld_stream_32(p + 8, v[2], v[3], wide);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = max(m, max(v[i].x & 0x7fffffffu, v[i].y & 0x7fffffffu));
      m = max(m, max(v[i].z & 0x7fffffffu, v[i].w & 0x7fffffffu));
    }
    return m;
  }
  __device__ __forceinline__ uint32_t amax_finite() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m = max(m, max(finite_abs_bits(__uint_as_float(v[i].x)), finite_abs_bits(__uint_as_float(v[i].y))));
      m = max(m, max(finite_abs_bits(__uint_as_float(v[i].z)), finite_abs_bits(__uint_as_float(v[i].w))));
    }
    return m;
  }
  __device__ __forceinline__ uint4 codes(float inv) const {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = e4m3x4(__uint_as_float(v[e].x) * inv, __uint_as_float(v[e].y) * inv, __uint_as_float(v[e].z) * inv,
                    __uint_as_float(v[e].w) * inv);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// four elements
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  float4 x;
  unpack_bf16x2(v.x, x.x, x.y);
  unpack_bf16x2(v.y, x.z, x.w);
  return x;
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

// the largest of the values of this thread's group of 2^GS threads, and of all groups; `s_max` is free
// again behind the caller's next barrier
template <int GS>
__device__ __forceinline__ uint32_t group_max(uint32_t mx, uint32_t* s_max, uint32_t& all) {
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
  all = 0u;
  const int mine = threadIdx.x >> GS;
#pragma unroll
  for (int w = 0; w < kThreadsW / 32; ++w) {
    all = max(all, s_max[w]);
    if (GS == 8 || w >> (GS - 5) == mine) mx = max(mx, s_max[w]);
  }
  return mx;
}

struct WriteParams {
  const void* K;           // [B][T][Hkv][d] new rows
  const void* V;
  const int32_t* start;    // [B]
  const int32_t* count;    // [B] or null: T rows
  uint8_t* K8;             // [B][n_max][Hkv][d]
  uint8_t* V8;
  float* ks;               // [B][nblk][Hkv]
  float* vs;
  void* ws_header;
  int B, T, n_max, Hkv, d, block, bshift, nblk, jmax;
  int hgroups;             // groups of 256 >> GS heads
  bool wide;               // K and V are 32-byte aligned
};

// One CTA per (sequence, block of tokens that the new rows touch, head, K or V), or for as many heads as
// its threads hold blocks of (2^GS threads a head): the block's new rows stay in registers between
// their maximum and their codes, so they are read once.  A thread holds NU units of 16 elements.  No two CTAs share a
// block's scale or codes.
// Elements are handled two at a time (packed maximum and product), and those that are not finite only where
// the maximum shows one: 4 chunks of 4K to 8K rows of 8 x 128 in bf16, blocks of 64, take 28 us; 37 one
// element at a time, with the integer pipe the bound.  2 x 16384 rows: bf16 33.1 us, 6.1 TB/s, fp32 50.6 (57
// with loads of 16 bytes, of which a lane takes every fourth).  Registers are held to eight CTAs an SM:
// with 54 instead of 32 the first figure was 33.
template <typename T, int NU, int GS>
__global__ void __launch_bounds__(kThreadsW, sizeof(T) == 2 ? (NU == 4 ? 5 : 8) : NU == 1 ? 6 : 8 / NU) kv8_write_kernel(const WriteParams p) {
  pdl_enter();
  static_assert(kThreadsW == 256, "eight warps");
  __shared__ __align__(16) uint32_t s_max[2][kThreadsW / 32];
  unsigned u = blockIdx.x;  // (which, heads, j, b), which fastest
  const bool isv = u & 1u;
  u >>= 1;
  const int h = (u % p.hgroups << (8 - GS)) + (GS == 8 ? 0 : threadIdx.x >> GS);
  u /= p.hgroups;
  constexpr int nthr = 1 << GS;
  const int tid = threadIdx.x & (nthr - 1);  // among the head's threads
  const bool mine = GS == 8 || h < p.Hkv;
  const int j = u % p.jmax;
  const int b = u / p.jmax;
  const int p0 = p.start[b];
  const int cnt = p.count ? max(0, min(p.count[b], p.T)) : p.T;
  if (cnt == 0) return;
  if (p0 < 0 || p0 > p.n_max - cnt) {  // not all rows fit: none is written
    if (j == 0 && h == 0 && !isv && tid == 0)
      record_error(p.ws_header, CLSA_ERR_BAD_INDEX, ((long long)b << 32) | (unsigned)p0);
    return;
  }
  const int blk = (p0 >> p.bshift) + j;
  if (blk > (p0 + cnt - 1) >> p.bshift) return;  // behind the last block touched
  const int first = blk * p.block;         // the block's first token
  const int lo = max(first, p0);           // new rows of this block: tokens [lo, hi)
  const int hi = min(first + p.block, p0 + cnt);
  const int sh = p.d == 128 ? 3 : 2, mask = (1 << sh) - 1;  // a row has 8 or 4 units
  const int units = mine ? (hi - lo) << sh : 0;
  const T* src = static_cast<const T*>(isv ? p.V : p.K) + (((size_t)b * p.T + (lo - p0)) * p.Hkv + h) * p.d;
  const size_t rstr = (size_t)p.Hkv * p.d;
  uint8_t* codes = (isv ? p.V8 : p.K8) + ((size_t)b * p.n_max * p.Hkv + h) * p.d;
  float* sc = (isv ? p.vs : p.ks) + ((size_t)b * p.nblk + blk) * p.Hkv + h;
  const bool kept = mine && lo > first;    // the block holds earlier rows
  const float s_old = kept ? *sc : 0.f;

  Load16<T> x[NU];
  uint32_t mx = 0;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int v = tid + i * nthr;
    if (v < units) x[i].load(src + (size_t)(v >> sh) * rstr + (v & mask) * 16, p.wide);
    else x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < NU; ++i) mx = max(mx, x[i].amax());
  uint32_t all;
  mx = group_max<GS>(mx, s_max[0], all);  // also: every thread has read the old scale
  if (all >= 0x7f800000u) {                // something is not finite: the largest of the rest
    mx = 0;
#pragma unroll
    for (int i = 0; i < NU; ++i) mx = max(mx, x[i].amax_finite());
    mx = group_max<GS>(mx, s_max[1], all);
  }
  float s = exp2_int(kv8_scale_exp(mx));
  if (kept) s = fmaxf(s, s_old);
  const float inv = 1.f / s;               // exact where s is a power of two: all but a kept scale of another program
  if ((__float_as_uint(s) & 0x7fffffu) == 0u) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const int v = tid + i * nthr;
      if (v < units) *reinterpret_cast<uint4*>(codes + (size_t)(lo + (v >> sh)) * rstr + (v & mask) * 16) = x[i].codes(inv);
    }
  } else {                                 // rare: by division, the rows read again (the registers above are all taken)
#pragma unroll 1
    for (int i = tid; i < 4 * units; i += nthr) {
      const int row = i >> (sh + 2), col = (i & (4 * mask + 3)) * 4;
      const float4 y = load4(src + (size_t)row * rstr + col);
      *reinterpret_cast<uint32_t*>(codes + (size_t)(lo + row) * rstr + col) =
          e4m3x4(__fdiv_rn(y.x, s), __fdiv_rn(y.y, s), __fdiv_rn(y.z, s), __fdiv_rn(y.w, s));
    }
  }
  if (tid == 0 && mine && !(kept && s == s_old)) *sc = s;
  if (kept && s > s_old) {                 // the earlier rows move to the larger scale
    const float r = s_old * inv;           // exact: s is new
    const int old_units = (lo - first) << sh;
    for (int v = tid; v < old_units; v += nthr) {
      uint4* at = reinterpret_cast<uint4*>(codes + (size_t)(first + (v >> sh)) * rstr + (v & mask) * 16);
      uint4 q = *at;
      uint32_t* w = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = e4m3x2_to_f32x2((uint16_t)w[e]), g = e4m3x2_to_f32x2((uint16_t)(w[e] >> 16));
        w[e] = e4m3x4(f.x * r, f.y * r, g.x * r, g.y * r);
      }
      *at = q;
    }
  }
}

struct ReadParams {
  const uint8_t* K8;
  const uint8_t* V8;
  const float* ks;
  const float* vs;
  const int32_t* start;   // [B] or null (0)
  const int32_t* idx;     // [B][T] or null
  const int32_t* count;   // [B] or null
  void* K;                // [B][T][Hkv][d]
  void* V;
  void* ws_header;
  int B, T, n_max, Hkv, d, bshift, nblk, tpc;
  bool wide;              // K and V are 32-byte aligned
};

// A thread keeps its place in the row (threadIdx.x: 16 codes of a head, threadIdx.y: the head,
// blockIdx.y: K or V and the heads behind blockDim.y) and walks the rows of the CTA, kReadRows of
// them in flight: no divisions in the loop.  4 x 8001 rows of 8 x 128 as bf16: 32.5 us, 6.0 TB/s, of an index list
// 34.8 (inputs in turn that L2 does not hold).  The choices below on one set of inputs, 31.6 us: 33.1
// with stores of 16 bytes, then 38 with four rows, 44 with eight (more registers, fewer threads), 34.1
// with one step a CTA, 34.9 with four.  One step where the CTAs all fit at once.
constexpr int kReadRows = 2;
template <typename T>
__global__ void __launch_bounds__(256, 5) kv8_read_kernel(const ReadParams p) {
  pdl_enter();
  const int ctas = (p.T + p.tpc - 1) / p.tpc;  // per sequence
  const int b = blockIdx.x / ctas;
  const int t0 = (blockIdx.x - b * ctas) * p.tpc;
  const int cnt = p.count ? min(p.count[b], p.T) : p.T;
  const int t1 = min(t0 + p.tpc, cnt);
  const bool isv = blockIdx.y & 1u;
  const int h = (blockIdx.y >> 1) * blockDim.y + threadIdx.y;
  if (t0 >= t1 || h >= p.Hkv) return;
  const size_t rstr = (size_t)p.Hkv * p.d;
  const int col = h * p.d + threadIdx.x * 16;
  const uint8_t* codes = (isv ? p.V8 : p.K8) + (size_t)b * p.n_max * rstr + col;
  const float* scales = (isv ? p.vs : p.ks) + (size_t)b * p.nblk * p.Hkv + h;
  T* out = static_cast<T*>(isv ? p.V : p.K) + (size_t)b * p.T * rstr + col;
  const long long s0 = p.start ? p.start[b] : 0;
  for (int t = t0 + threadIdx.z; t < t1; t += kReadRows * blockDim.z) {
    uint4 c[kReadRows];
    float s[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int ti = t + i * blockDim.z;
      if (ti >= t1) continue;
      const long long tok = p.idx ? p.idx[(size_t)b * p.T + ti] : s0 + ti;
      c[i] = make_uint4(0u, 0u, 0u, 0u);
      s[i] = 0.f;
      if (tok >= 0 && tok < p.n_max) {
        c[i] = ld_stream_v4(codes + (size_t)tok * rstr);
        s[i] = __ldg(scales + (size_t)(tok >> p.bshift) * p.Hkv);
      } else if (col == 0 && !isv) {
        record_error(p.ws_header, CLSA_ERR_BAD_INDEX, ((long long)b << 32) | (unsigned)ti);
      }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
      const int ti = t + i * blockDim.z;
      if (ti >= t1) continue;
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
      float f[16];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 x = e4m3x2_to_f32x2((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
        f[2 * e] = x.x * s[i];
        f[2 * e + 1] = x.y * s[i];
      }
      if constexpr (sizeof(T) == 2) {
        uint32_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);
        st_32(out + (size_t)ti * rstr, x, p.wide);
      } else {
        st_32(out + (size_t)ti * rstr, reinterpret_cast<const uint32_t*>(f), p.wide);
        st_32(out + (size_t)ti * rstr + 8, reinterpret_cast<const uint32_t*>(f) + 8, p.wide);
      }
    }
  }
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

template <typename T>
cudaError_t launch_write(WriteParams p, cudaStream_t s) {
  // a block of 16 x 64 has 64 units: a CTA takes four heads (2 x 16384 rows of 8 x 64 in such blocks: 22
  // to 24 us; 67 with a head a CTA, most of its threads idle)
  const int units = p.block * (p.d / 16), gs = std::min(8, log2_of(units));
  p.hgroups = (p.Hkv + (kThreadsW >> gs) - 1) >> (8 - gs);
  const dim3 grid((unsigned)(2LL * p.hgroups * p.jmax * p.B));
  if (gs == 6) return launch_pdl(kv8_write_kernel<T, 1, 6>, grid, dim3(kThreadsW), 0, s, p);
  if (gs == 7) return launch_pdl(kv8_write_kernel<T, 1, 7>, grid, dim3(kThreadsW), 0, s, p);
  const int nu = (std::min(p.T, p.block) * (p.d / 16) + kThreadsW - 1) / kThreadsW;  // <= 4: 128 x 128
  if (nu <= 1) return launch_pdl(kv8_write_kernel<T, 1, 8>, grid, dim3(kThreadsW), 0, s, p);
  if (nu <= 2) return launch_pdl(kv8_write_kernel<T, 2, 8>, grid, dim3(kThreadsW), 0, s, p);
  return launch_pdl(kv8_write_kernel<T, 4, 8>, grid, dim3(kThreadsW), 0, s, p);
}

}  // namespace

// blocks that T rows can touch
static long long write_jmax(int T, int block) { return ((long long)T + block - 2) / block + 1; }

bool kv8_write_grid_ok(const clsa_kv8_cache* c, int T) {
  return 2LL * c->Hkv * write_jmax(T, c->block) * c->B <= 0x7fffffffLL;
}

cudaError_t launch_kv8_write(const clsa_kv8_cache* c, const void* K, const void* V, const int32_t* start,
                             const int32_t* count, int T, clsa_dtype dt, void* ws_header, cudaStream_t s) {
  WriteParams p{};
  p.K = K;
  p.V = V;
  p.start = start;
  p.count = count;
  p.K8 = static_cast<uint8_t*>(c->K8);
  p.V8 = static_cast<uint8_t*>(c->V8);
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.ws_header = ws_header;
  p.B = c->B;
  p.T = T;
  p.n_max = c->n_max;
  p.Hkv = c->Hkv;
  p.d = c->d;
  p.block = c->block;
  p.nblk = (c->n_max + c->block - 1) / c->block;
  p.bshift = log2_of(c->block);
  p.wide = (((uintptr_t)K | (uintptr_t)V) & 31) == 0;
  p.jmax = (int)write_jmax(T, c->block);
  const cudaError_t e = dt == CLSA_BF16 ? launch_write<__nv_bfloat16>(p, s) : launch_write<float>(p, s);
  launches_add(1, s);
  return e;
}

// threads of a CTA: a head's units, heads, rows (256 in all); rows a CTA takes
static dim3 read_block(const clsa_kv8_cache* c) {
  const int x = c->d / 16, y = std::min(c->Hkv, 256 / x);
  return dim3(x, y, std::max(1, 256 / (x * y)));
}
static int read_heads(const clsa_kv8_cache* c) { return 2 * ((c->Hkv + read_block(c).y - 1) / read_block(c).y); }  // grid.y
static int read_tpc(const clsa_kv8_cache* c, int T) {
  const int rows = kReadRows * (int)read_block(c).z;
  const double ctas = std::ceil((double)T / rows) * c->B * read_heads(c);
  return ctas >= 10.0 * device_info().sm_count ? 2 * rows : rows;  // five fit on an SM
}

bool kv8_read_grid_ok(const clsa_kv8_cache* c, int T) {
  const int tpc = kReadRows * (int)read_block(c).z;
  return ((long long)T + tpc - 1) / tpc * c->B <= 0x7fffffffLL && c->Hkv <= 1 << 16;
}

cudaError_t launch_kv8_read(const clsa_kv8_cache* c, const int32_t* start, const int32_t* idx, const int32_t* count,
                            int T, clsa_dtype dt, void* K, void* V, void* ws_header, cudaStream_t s) {
  ReadParams p{};
  p.K8 = static_cast<const uint8_t*>(c->K8);
  p.V8 = static_cast<const uint8_t*>(c->V8);
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.start = start;
  p.idx = idx;
  p.count = count;
  p.K = K;
  p.V = V;
  p.ws_header = ws_header;
  p.B = c->B;
  p.T = T;
  p.n_max = c->n_max;
  p.Hkv = c->Hkv;
  p.d = c->d;
  p.bshift = log2_of(c->block);
  p.nblk = (c->n_max + c->block - 1) / c->block;
  p.tpc = read_tpc(c, T);
  p.wide = (((uintptr_t)K | (uintptr_t)V) & 31) == 0;
  const dim3 block = read_block(c);
  const dim3 grid((unsigned)(((long long)T + p.tpc - 1) / p.tpc * c->B), read_heads(c));
  const cudaError_t e = dt == CLSA_BF16 ? launch_pdl(kv8_read_kernel<__nv_bfloat16>, grid, block, 0, s, p)
                                        : launch_pdl(kv8_read_kernel<float>, grid, block, 0, s, p);
  launches_add(1, s);
  return e;
}

}  // namespace clsa
