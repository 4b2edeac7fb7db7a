// Attention over the 8-bit K/V cache: decode rows over every cached token, or over the shared
// selection.  The kernel is stream_attn.cuh; here the rows of one KV head are the (layer,
// query head) pairs of its group, up to 8 or 16 of them to a row group.
#include "stream_attn.cuh"

namespace clsa {

namespace {

stream::Params params_of(const clsa_kv8_attn_args* a, float scale) {
  stream::Params p{};
  p.Q = a->Q;
  p.K = a->cache.K8;
  p.V = a->cache.V8;
  p.ks = a->cache.k_scale;
  p.vs = a->cache.v_scale;
  p.idx = a->idx;
  p.count = a->count;
  p.O = a->O;
  p.lse = a->lse;
  p.q_sl = (long long)a->B * a->Hq * a->cache.d;
  p.q_sb = (long long)a->Hq * a->cache.d;
  p.B = a->B;
  p.Hkv = a->cache.Hkv;
  p.G = a->Hq / a->cache.Hkv;
  p.R = a->L * p.G;
  p.n_max = a->cache.n_max;
  p.k = a->k;
  p.nblk = (a->cache.n_max + a->cache.block - 1) / a->cache.block;
  while ((1 << p.bshift) < a->cache.block) ++p.bshift;
  p.seqs = a->cache.B;
  p.scale_log2 = scale * 1.4426950408889634f;
  const int rows = 8 * stream::row_tiles(p.R, a->dtype == CLSA_F32);
  p.nrg = (p.R + rows - 1) / rows;
  return p;
}

// calls f<Cfg>
template <bool RING, typename F>
auto dispatch(const clsa_kv8_attn_args* a, int R, F&& f) {
  using namespace stream;
  const bool d128 = a->cache.d == 128;
  if (a->dtype == CLSA_F32)
    return d128 ? f(Cfg<kE4m3, true, RING, 128, 1>{}) : f(Cfg<kE4m3, true, RING, 64, 1>{});
  if (row_tiles(R, false) == 1)
    return d128 ? f(Cfg<kE4m3, false, RING, 128, 1>{}) : f(Cfg<kE4m3, false, RING, 64, 1>{});
  return d128 ? f(Cfg<kE4m3, false, RING, 128, 2>{}) : f(Cfg<kE4m3, false, RING, 64, 2>{});
}

}  // namespace

size_t kv8_attn_ws_bytes(const clsa_kv8_attn_args* a) {
  const stream::Params p = params_of(a, 1.f);
  const auto f = [&](auto c) { return stream::ws_bytes<decltype(c)>(p); };
  return a->idx ? dispatch<false>(a, p.R, f) : dispatch<true>(a, p.R, f);
}

cudaError_t launch_kv8_attn(const clsa_kv8_attn_args* a, float scale, void* ws_header, void* ws_body, cudaStream_t s) {
  stream::Params p = params_of(a, scale);
  p.ws_header = ws_header;
  const auto f = [&](auto c) { return stream::launch<decltype(c)>(p, ws_body, s); };
  return a->idx ? dispatch<false>(a, p.R, f) : dispatch<true>(a, p.R, f);
}

}  // namespace clsa
