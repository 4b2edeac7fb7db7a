// Window attention of a chunk of rows on the 5th-generation tensor cores (bf16, d = 64 or 128):
//   row at position p:  O = softmax(q K_j^T scale) V_j  over j <= p with j > p - W or j < S.
//
// Rows.  The G query heads of a KV head share its keys, so a 128-row tile holds 128 / G tokens of
// all G heads: a tile's rows then span few positions, and little of the window is scored for
// rows that do not see it (G = 4, W = 1024: 1087 positions for 64 tokens; 64 tokens of one
// head each would be 4 x 1087).  An item is two such tiles of one (sequence, KV head); where the items
// of the last round would leave half of the SMs idle, they are one tile each (a token tile of an item takes
// a CTA about 2900 cycles with two row tiles, 2600 with one: T = 4096, W = 1024 83 -> 81 us, T = 512, W = 4096
// 65 -> 59 us).
//
// Tokens.  The item's tokens form a line: the sinks (rounded up to 8), then the window's union
// [lo, p_last].  It is cut into tiles of 128; a tile of window tokens is one TMA box, the tile
// that holds the seam is boxes of 32 and 8 rows.  Value rows of tokens that no row of the item
// sees are zeroed in shared memory, so their bytes do not matter (0 * NaN).
//
// Roles (one CTA per SM, persistent over items): one warp issues TMA loads into a ring of K and V
// tiles; one zeroes the unseen value rows; one issues the MMAs; two groups of four warps each own
// one row tile's softmax, a thread a row.  For every token tile and row tile i:
//   S_i = Q_i K^T        M128 N128, both operands in shared memory      -> TMEM
//   P_i = exp2(S_i scale - m)   S from TMEM to registers, bf16 P back over S's columns
//   O_i += P_i V         A = P from TMEM, B = V (MN-major)              -> TMEM
// The MMAs of one row tile run while the other's softmax does.  S of the next token tile (of the next
// item too) is issued right behind P V, which the in-order tensor pipe keeps from
// overwriting P early.  m is a reference that moves only when a score exceeds it by 2^8;
// then O is rescaled in TMEM.  A row's softmax needs no exchange: its 128 scores are one lane.
// P is rounded to bf16, since an MMA's operands have one type and V's is bf16: off by up to 2^-8 of each weight.
// On random values the result's error against 64 bits is then 1.3 to 1.4 times that of weights in fp32 (0.0022 of the
// result for 0.0016, its own rounding to bf16).  The row's sum takes the weights as they were.
// Bound: per token tile and row tile 2 x 128 x 128 x d multiplies and 128 x 128 exponentials, which at
// d = 128 take the tensor cores and the special-function units about 1024 cycles each.
// Measured (32 heads on 8, d = 128; inputs in turn that L2 does not hold): T = 16381, W = 4096 750 us, 1.28 PFLOP/s
// of visible products, over some ms, 860 over longer runs at the power limit; T = 4096, W = 1024 78.5 us, 0.88 PFLOP/s
// (75 with its inputs in L2).  A step of both row tiles takes about 2950 cycles: 1450 for a tile's
// exponentials and P, 400 for its scores and maximum, then 920 until P V and the next S are through
// (768 of them products); the two tiles' chains overlap, but neither pipe fills (tensor cores active 49 %
// at W = 1024).  P leaves columns 64 to 127 of each S free, so half of a tile's next scores could be in TMEM before P V
// has read this one's; they are all issued behind it.  A change of item costs about 5000 cycles more, partly filled
// tiles the rest.
//
// Every wait is bounded; one that runs out records CLSA_ERR_TIMEOUT and the CTA drains its
// loads and returns.
#include <cuda.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"
#include "tma.h"
#include "vec32.cuh"

namespace clsa {

namespace {

constexpr int kTok = 128;                   // tokens of a tile
constexpr int kRows = 128;                  // rows of a row tile
// Warp roles.  The MMA warp comes first: it is the one that must never wait for an issue slot.
constexpr int kMmaWarp = 0, kTmaWarp = 1, kFixWarp = 2, kSoft0 = 4;  // kSoft0 + 0..3: row tile 0, + 4..7: row tile 1
constexpr int kThreadsW = (kSoft0 + 8) * 32;
constexpr uint32_t kAtom = 128 * 128;       // 128 rows x 128 bytes
constexpr float kNone = -3e38f;
constexpr float kTau = 8.f;
constexpr float kLn2 = 0.6931471805599453f;

struct Maps {
  CUtensorMap q, k, v, k8, v8, k32, v32;  // boxes of 128, 8 and 32 rows
};

struct WParams {
  const int32_t* lens;
  __nv_bfloat16* O;     // [B][T][Hq][D]
  float* lse;           // [B][T][Hq] or null
  void* ws_header;
  int B, T, n_max, Hq, Hkv, G, TQ, nqt, window, sinks, items;
  int whole;            // items from here on are one row tile each
  float scale_log2;
  bool wide;            // O is 32-byte aligned
};

template <int D>
struct Smem {
  static constexpr int KA = D / 64;                     // 64-column atoms
  static constexpr uint32_t tile = KA * kAtom;          // Q, K or V tile
  static constexpr int slots = D == 128 ? 5 : 8;        // K and V tiles in the ring
  static_assert(slots <= 8, "at most four V tiles");
  static constexpr uint32_t ring = 2 * tile;            // after the two Q tiles
  static constexpr uint32_t bars = ring + slots * tile;
  static constexpr uint32_t total = bars + 272 + 1024;  // + alignment of the base
};

// an item: rows [t0, t1) of sequence b, KV head g, and its line of tokens
struct WItem {
  int b, g, t0, ntile, len, nkv, npos, keep, keepP, keepM, lo;
};

__device__ __forceinline__ WItem witem(const WParams& p, int i) {
  WItem w;
  int rows = 2 * p.TQ, second = 0;
  if (i >= p.whole) {
    rows = p.TQ;
    second = (i - p.whole) & 1;
    i = p.whole + ((i - p.whole) >> 1);
  }
  w.g = i % p.Hkv;
  i /= p.Hkv;
  w.b = i % p.B;
  const int qt = p.nqt - 1 - i / p.B;  // the latest rows (longest lines) first
  w.t0 = qt * 2 * p.TQ + second * p.TQ;
  w.len = max(0, min(p.lens[w.b], p.n_max));
  w.ntile = rows > p.TQ && w.t0 + p.TQ < p.T ? 2 : 1;
  const int first = w.len - p.T + w.t0, last = w.t0 < p.T ? w.len - p.T + min(p.T, w.t0 + rows) - 1 : -1;
  w.nkv = w.npos = 0;
  w.lo = w.keep = w.keepP = w.keepM = 0;
  if (last < 0) return w;
  w.lo = max(0, max(0, first) - p.window + 1);
  w.keepM = p.sinks;
  if (w.lo <= p.sinks) w.lo = 0;
  else {
    w.keep = p.sinks;
    w.keepP = (p.sinks + 7) & ~7;
  }
  w.npos = w.keepP + last + 1 - w.lo;
  w.nkv = (w.npos + kTok - 1) / kTok;
  return w;
}
// value rows of tile j that no row sees: [a0, a1) behind the sinks, [b0, 128) behind the line
__device__ __forceinline__ bool dead_rows(const WItem& w, int j, int& a0, int& a1, int& b0) {
  a0 = min(max(w.keep - j * kTok, 0), kTok);
  a1 = min(max(w.keepP - j * kTok, 0), kTok);
  b0 = min(w.npos - j * kTok, kTok);
  return a0 < a1 || b0 < kTok;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// one lane of a converged warp.  MMAs are issued under it, and with operands that are the same in
// every lane by construction: then a tcgen05.mma issues in the 64 cycles that it runs (M128 N128
// K16); under `lane == 0` each took about 140.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// bounded wait of a whole warp; false (and CLSA_ERR_TIMEOUT with `site`) once kWaitLimitNs has passed
__device__ __forceinline__ bool wait_full(uint64_t* bar, uint32_t parity, void* ws, int site) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
#pragma unroll 1
    for (int x = 0; x < 32; ++x)
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs)) break;
  }
  if ((threadIdx.x & 31) == 0) record_error(ws, CLSA_ERR_TIMEOUT, site);
  return false;
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// this thread's lane, 8 consecutive columns
__device__ __forceinline__ void st_32x32b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// pairs of floats: two products or sums an instruction
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f32x2_get(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreadsW, 1) window_tc_kernel(const __grid_constant__ Maps maps, const WParams p) {
  using S = Smem<D>;
  pdl_enter();
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + S::bars);
  uint64_t* kv_full = bars;                  // [slots]
  uint64_t* kv_empty = bars + 8;             // [slots]
  uint64_t* q_full = bars + 16;              // [2]
  uint64_t* q_empty = bars + 18;
  uint64_t* s_full = bars + 20;
  uint64_t* p_full = bars + 22;              // [2][2]: the halves of P
  uint64_t* o_full = bars + 26;
  // a V tile's unseen rows are zero; such tiles take the four in turn.  The ring holds at most four V
  // tiles, so the warp that zeroes them is never a whole turn ahead; nor is it one behind: a tile's slot is
  // filled again only when this warp, too, has gone past it (its waits are by parity, and a phase that
  // it missed would stand still).
  uint64_t* fixed = bars + 28;               // [4]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 32);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::slots; ++i) {
      mbar_init(kv_full + i, 1);
      mbar_init(kv_empty + i, 2);  // the products that read the tile, and the warp that zeroes its unseen rows
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + 2 * i, 4);  // one arrival per softmax warp
      mbar_init(p_full + 2 * i + 1, 4);
      mbar_init(o_full + i, 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(fixed + i, 1);
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;  // S_i at 128 i (P_i over its first 64 columns), O_i at 256 + 128 i

  if (warp == kTmaWarp) {
    // ---------------------------------------------------------------- loads
    if (lane == 0) {
      int n = 0;              // K and V tiles issued
      uint32_t qi[2] = {0, 0};  // Q tiles issued
      bool ok = true;
      auto load_kv = [&](const WItem& w, int j, bool v) {
        const int slot = n % S::slots;
        const uint32_t use = (uint32_t)(n / S::slots);
        if (use > 0 && !mbar_wait(kv_empty + slot, (use - 1) & 1u)) {
          record_error(p.ws_header, CLSA_ERR_TIMEOUT, 60);
          return false;
        }
        unsigned char* dst = base + S::ring + slot * S::tile;
        mbar_arrive_expect_tx(kv_full + slot, S::tile);
        const int row0 = w.b * p.n_max;
        const int pos = j * kTok;
        if (pos >= w.keepP) {  // window tokens only
#pragma unroll
          for (int a = 0; a < S::KA; ++a)
            tma_load_2d(dst + a * kAtom, v ? &maps.v : &maps.k, w.g * D + 64 * a, row0 + w.lo + pos - w.keepP, kv_full + slot);
        } else {
          for (int r = 0; r < kTok;) {
            const int q = pos + r;
            const int tok = q < w.keepP ? q : w.lo + q - w.keepP;
            const bool big = r + 32 <= kTok && (q >= w.keepP || q + 32 <= w.keepP);
            const CUtensorMap* map = big ? (v ? &maps.v32 : &maps.k32) : v ? &maps.v8 : &maps.k8;
#pragma unroll
            for (int a = 0; a < S::KA; ++a)
              tma_load_2d(dst + a * kAtom + r * 128, map, w.g * D + 64 * a, row0 + tok, kv_full + slot);
            r += big ? 32 : 8;
          }
        }
        ++n;
        return true;
      };
      for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
        const WItem w = witem(p, i);
        for (int j = 0; j < w.nkv && ok; ++j) {
          ok = load_kv(w, j, false);
          if (j == 0) {
            for (int t = 0; t < w.ntile && ok; ++t) {
              if (qi[t] > 0 && !mbar_wait(q_empty + t, (qi[t] - 1) & 1u)) {
                record_error(p.ws_header, CLSA_ERR_TIMEOUT, 61);
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(q_full + t, (uint32_t)(p.TQ * p.G) * 128u * S::KA);
#pragma unroll
              for (int a = 0; a < S::KA; ++a)
                tma_load_3d(base + t * S::tile + a * kAtom, &maps.q, 64 * a, w.g * p.G, w.b * p.T + w.t0 + t * p.TQ, q_full + t);
              ++qi[t];
            }
          }
          if (ok) ok = load_kv(w, j, true);
        }
      }
      // loads in flight land before the CTA ends, also where a role gave up
      for (int s = std::max(0, n - S::slots); s < n; ++s) mbar_wait(kv_full + s % S::slots, (uint32_t)(s / S::slots) & 1u);
      for (int t = 0; t < 2; ++t)
        if (qi[t] > 0) mbar_wait(q_full + t, (qi[t] - 1) & 1u);
    }
  } else if (warp == kFixWarp) {
    // ---------------------------------------------------------------- value rows that no row sees
    int n = 0, nfix = 0;       // ring position, tiles zeroed
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      const WItem w = witem(p, i);
      for (int j = 0; j < w.nkv && ok; ++j, n += 2) {
        // every phase in its turn (a wait for a phase that lies two ahead would pass at once)
        for (int x = n; x < n + 2 && ok; ++x) {
          ok = wait_full(kv_full + x % S::slots, (uint32_t)(x / S::slots) & 1u, p.ws_header, 72);
          if (ok && x == n && lane == 0) mbar_arrive(kv_empty + x % S::slots);
        }
        if (!ok) break;
        const int slot = (n + 1) % S::slots;
        int a0, a1, b0;
        if (dead_rows(w, j, a0, a1, b0)) {
          unsigned char* v = base + S::ring + slot * S::tile;
          for (int x = lane; x < (a1 - a0 + kTok - b0) * 8; x += 32) {
            const int r = x >> 3, row = r < a1 - a0 ? a0 + r : b0 + r - (a1 - a0);
#pragma unroll
            for (int a = 0; a < S::KA; ++a)
              *reinterpret_cast<uint4*>(v + a * kAtom + row * 128 + (x & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(fixed + (nfix & 3));
          ++nfix;
        }
        if (lane == 0) mbar_arrive(kv_empty + slot);
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMAs
    constexpr uint32_t idesc_qk = tc::idesc_bf16_f32(kRows, kTok);
    constexpr uint32_t idesc_pv = tc::idesc_bf16_f32(kRows, D) | (1u << 16);  // V MN-major
    const uint64_t q0 = tc::sw128_desc(smem_u32(base)), ring0 = tc::sw128_desc(smem_u32(base + S::ring));
    const uint64_t ringv0 = tc::sw128_desc_mn(smem_u32(base + S::ring), kAtom);
    int slot = 0;              // ring position of the current step's K tile, and how often the ring was gone through
    uint32_t use = 0, nq[2] = {0, 0}, np = 0, np1 = 0, nfix = 0;  // phases
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, int site) { return wait_full(bar, parity & 1u, p.ws_header, site); };
    auto qk = [&](auto t, int at) {  // S_t = Q_t K^T
      const uint64_t qd = q0 + t * (S::tile >> 4), kd = ring0 + (uint32_t)uniform(at) * (S::tile >> 4);
      tc::fence_after_sync();
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * kAtom + (ks & 3) * 32) >> 4;
          tc::mma_bf16(tmem + 128u * t, qd + off, kd + off, idesc_qk, ks > 0);
        }
        tc::mma_commit(s_full + t);
      }
      __syncwarp();
    };
    auto pv = [&](auto t, auto h, int at, bool add) {  // O_t += P_t V, tokens [64 h, 64 h + 64)
      const uint64_t vd = ringv0 + (uint32_t)uniform(at) * (S::tile >> 4);
      tc::fence_after_sync();
      if (elect_one()) {
#pragma unroll
        for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
          mma_bf16_ts(tmem + 256u + 128u * t, tmem + 128u * t + 8u * ks, vd + (uint32_t)ks * (16 * 128 >> 4), idesc_pv, add || ks > 0);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc::mma_commit(bar);
      __syncwarp();
    };
    int i = blockIdx.x, j = 0;
    WItem w;
    w.nkv = 0;
    while (i < p.items && (w = witem(p, i)).nkv == 0) i += gridDim.x;
    if (i < p.items) {         // the first item's first scores
      ok = wait(kv_full, 0, 62);
      auto first = [&](auto t) {
        if (t >= w.ntile || !ok) return;
        ok = wait(q_full + t, nq[t]++, 63);
        if (!ok) return;
        qk(t, 0);
        if (w.nkv == 1) commit(q_empty + t);
      };
      first(std::integral_constant<int, 0>{});
      first(std::integral_constant<int, 1>{});
      if (ok) commit(kv_empty);
    }
    while (i < p.items && ok) {
      // the step behind this one: the item's next token tile, or the next item's first
      WItem nw = w;
      int nj = j + 1, ni = i;
      if (nj == w.nkv) {
        nj = 0;
        do ni += gridDim.x;
        while (ni < p.items && (nw = witem(p, ni)).nkv == 0);
      }
      const bool more = ni < p.items;
      int vslot = slot + 1, kslot = slot + 2;
      uint32_t vuse = use, kuse = use;
      if (vslot >= S::slots) vslot -= S::slots, ++vuse;
      if (kslot >= S::slots) kslot -= S::slots, ++kuse;
      int a0, a1, b0;
      const bool fix = dead_rows(w, j, a0, a1, b0);
      ok = fix ? wait(fixed + (nfix & 3), nfix >> 2, 71) : wait(kv_full + vslot, vuse, 64);
      nfix += fix ? 1 : 0;
      bool have_k = false;
      auto step = [&](auto t) {
        if (t < w.ntile && ok) {
          const uint32_t ph = t == 0 ? np : np1;
          ok = wait(p_full + 2 * t, ph, 65);
          if (!ok) return;
          pv(t, std::integral_constant<int, 0>{}, vslot, j > 0);
          ok = wait(p_full + 2 * t + 1, ph, 65);
          if (!ok) return;
          pv(t, std::integral_constant<int, 1>{}, vslot, true);
          if (t == 0) ++np;
          else ++np1;
          if (j == w.nkv - 1) commit(o_full + t);
        }
        if (more && t < nw.ntile && ok) {
          if (!have_k) ok = wait(kv_full + kslot, kuse, 66);
          have_k = true;
          if (ok && nj == 0) ok = wait(q_full + t, nq[t]++, 67);
          if (!ok) return;
          qk(t, kslot);
          if (nj == nw.nkv - 1) commit(q_empty + t);
        }
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      if (!ok) break;
      commit(kv_empty + vslot);
      if (more) commit(kv_empty + kslot);
      slot = kslot;
      use = kuse;
      w = nw;
      i = ni;
      j = nj;
    }
  } else if (warp >= kSoft0) {
    // ---------------------------------------------------------------- softmax
    const int t = (warp - kSoft0) >> 2;                        // row tile
    const int r = (warp & 3) * 32 + lane;           // row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + 128u * t, to = tmem + lanes + 256u + 128u * t;
    uint32_t ns = 0, no = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.items && ok; i += gridDim.x) {
      const WItem w = witem(p, i);
      if (t >= w.ntile) continue;
      const int tok = w.t0 + t * p.TQ + r / p.G;
      const bool live = r < p.TQ * p.G && tok < p.T;
      const long long row = ((long long)w.b * p.T + tok) * p.Hq + w.g * p.G + r % p.G;
      const int pr = w.len - p.T + tok;             // the row's position
      // every row of the tile sees a token tile's columns iff the first and the last row do
      const int pf = w.len - p.T + w.t0 + t * p.TQ, pl = pf + p.TQ - 1;
      float m = kNone, l = 0.f;
      for (int j = 0; j < w.nkv; ++j) {
        ok = wait_full(s_full + t, ns++ & 1u, p.ws_header, 68);
        if (!ok) break;
        tc::fence_after_sync();
        uint32_t v[kTok];
        tc::ld_32x32b_x128(ts, v);
        tc::ld_wait();
        const int w0 = w.lo + j * kTok - w.keepP;   // column c holds token w0 + c from column cw on
        const int cw = w.keepP - j * kTok;
        if (cw > 0 || w0 + kTok - 1 > pf || w0 <= pl - p.window) {
          const int cs = min(w.keepM, pr + 1) - j * kTok;
          const int cl = max(pr - p.window + 1 - w0, cw), ch = pr - w0;
          // bits of the columns below x, 32 at a time: a test and a select per score
          const auto below = [](int x) { return x <= 0 ? 0u : 0xffffffffu >> (32 - min(x, 32)); };
#pragma unroll
          for (int h = 0; h < kTok; h += 32) {
            const uint32_t see = below(cs - h) | (below(ch + 1 - h) & ~below(cl - h));
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(see & (1u << c))) v[h + c] = 0xff800000u;
          }
        }
        float x0 = kNone, x1 = kNone, x2 = kNone, x3 = kNone;
#pragma unroll
        for (int c = 0; c < kTok; c += 8) {
          x0 = fmaxf(fmaxf(x0, __uint_as_float(v[c])), __uint_as_float(v[c + 1]));
          x1 = fmaxf(fmaxf(x1, __uint_as_float(v[c + 2])), __uint_as_float(v[c + 3]));
          x2 = fmaxf(fmaxf(x2, __uint_as_float(v[c + 4])), __uint_as_float(v[c + 5]));
          x3 = fmaxf(fmaxf(x3, __uint_as_float(v[c + 6])), __uint_as_float(v[c + 7]));
        }
        const float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * p.scale_log2;  // scale > 0: the maximum commutes
        const bool up = mx > m + kTau;
        if (__any_sync(0xffffffffu, up)) {          // P V of the token tile before has completed
          const float mn = up ? mx : m;
          const float f = fast_exp2(m - mn);
          if (j > 0) {
#pragma unroll 1
            for (int h = 0; h < D / 32; ++h) {
              uint32_t o[32];
              tc::ld_32x32b_x32(to + 32u * h, o);
              tc::ld_wait();
#pragma unroll
              for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
              tc::st_32x32b_x32(to + 32u * h, o);
            }
          }
          l *= f;
          m = mn;
        }
        uint64_t s0 = 0, s1 = 0;                    // pairs of sums
        const uint64_t sc2 = f32x2(p.scale_log2, p.scale_log2), nm2 = f32x2(-m, -m);
#pragma unroll
        for (int h = 0; h < 8; ++h) {               // 16 columns at a time: few registers beside the scores
          uint32_t pw[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float a, b;
            f32x2_get(fma_f32x2(f32x2(__uint_as_float(v[16 * h + 2 * c]), __uint_as_float(v[16 * h + 2 * c + 1])), sc2, nm2), a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            if (c & 1) s1 = add_f32x2(s1, f32x2(a, b));
            else s0 = add_f32x2(s0, f32x2(a, b));
            pw[c] = pack_bf16x2(a, b);
          }
          st_32x32b_x8(ts + 8u * h, pw);
          if (h == 3) {                             // the first half of P: its MMAs may start
            tc::st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full + 2 * t);
          }
        }
        float sa, sb;
        f32x2_get(add_f32x2(s0, s1), sa, sb);
        l += sa + sb;
        tc::st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 2 * t + 1);
      }
      if (!ok) break;
      uint4* out = reinterpret_cast<uint4*>(p.O + row * D);
      if (w.nkv > 0) {
        ok = wait_full(o_full + t, no++ & 1u, p.ws_header, 69);
        if (!ok) break;
        tc::fence_after_sync();
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int h = 0; h < D / 32; ++h) {
          uint32_t o[32];
          tc::ld_32x32b_x32(to + 32u * h, o);
          tc::ld_wait();
          uint32_t x[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)              // P = 0 everywhere: O is 0, not 0 * NaN
            x[c] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv);
          // lanes write rows of their own: with 32 bytes a lane half the passes through L1 of 16 bytes
          if (live && p.wide) {
            st_global_v8(out + 4 * h, x);
            st_global_v8(out + 4 * h + 2, x + 8);
          } else if (live) {
#pragma unroll
            for (int c = 0; c < 4; ++c) out[4 * h + c] = make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          }
        }
        tc::fence_before_sync();
      } else if (live) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c) out[c] = make_uint4(0u, 0u, 0u, 0u);
      }
      if (live && p.lse) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

bool make_tmap_q(CUtensorMap* map, const void* base, int d, int Hq, long long rows, int box_heads, int box_rows) {
  const TmapEncodeFn fn = tmap_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)Hq, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)Hq * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const Maps& maps, const WParams& p, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(window_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Smem<D>::total);
  if (e != cudaSuccess) return e;
  e = launch_pdl(window_tc_kernel<D>, dim3(std::min(p.items, std::max(1, device_info().sm_count))), dim3(kThreadsW),
                 Smem<D>::total, s, maps, p);
  launches_add(1, s);
  return e;
}

}  // namespace

bool window_tc_supported(const clsa_window_args* a) {
  const int G = a->Hq / a->Hkv;
  if (a->dtype != CLSA_BF16 || G > kRows) return false;
  const long long nqt = (a->T + 2LL * (kRows / G) - 1) / (2 * (kRows / G));
  // rows and items are counted in 32 bits
  return (long long)a->B * a->n_max < (1LL << 31) && (long long)a->B * a->T < (1LL << 31) && nqt * a->B * a->Hkv < (1LL << 31) &&
         (long long)a->Hkv * a->d < (1LL << 31);
}

cudaError_t launch_window_tc(const clsa_window_args* a, float scale, void* ws_header, cudaStream_t s) {
  WParams p{};
  p.lens = a->seq_lens;
  p.O = static_cast<__nv_bfloat16*>(a->O);
  p.lse = a->lse;
  p.ws_header = ws_header;
  p.B = a->B;
  p.T = a->T;
  p.n_max = a->n_max;
  p.Hq = a->Hq;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.TQ = kRows / p.G;
  p.nqt = (int)((a->T + 2LL * p.TQ - 1) / (2 * p.TQ));
  p.window = std::min(a->window, a->n_max);
  p.sinks = std::min(a->sinks, a->n_max);
  p.items = p.whole = p.nqt * p.B * p.Hkv;
  const int over = p.items % std::max(1, device_info().sm_count);
  if (2 * over <= device_info().sm_count) {
    p.whole = p.items - over;
    p.items += over;
  }
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wide = ((uintptr_t)a->O & 31) == 0;
  Maps maps{};
  const uint64_t rows = (uint64_t)a->B * a->n_max, cols = (uint64_t)a->Hkv * a->d;
  if (!make_tmap_q(&maps.q, a->Q, a->d, a->Hq, (long long)a->B * a->T, p.G, p.TQ) ||
      !make_tmap_bf16_2d(&maps.k, a->K, rows, cols, cols * 2, kTok, 64) ||
      !make_tmap_bf16_2d(&maps.v, a->V, rows, cols, cols * 2, kTok, 64))
    return cudaErrorInvalidValue;
  if (p.sinks > 0 &&  // the seam tile's boxes
      (!make_tmap_bf16_2d(&maps.k8, a->K, rows, cols, cols * 2, 8, 64) ||
       !make_tmap_bf16_2d(&maps.v8, a->V, rows, cols, cols * 2, 8, 64) ||
       !make_tmap_bf16_2d(&maps.k32, a->K, rows, cols, cols * 2, 32, 64) ||
       !make_tmap_bf16_2d(&maps.v32, a->V, rows, cols, cols * 2, 32, 64)))
    return cudaErrorInvalidValue;
  return a->d == 128 ? launch_d<128>(maps, p, s) : launch_d<64>(maps, p, s);
}

}  // namespace clsa
