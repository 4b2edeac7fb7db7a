// Attention with a sliding window and sink tokens.
#include "stream_attn.cuh"

namespace clsa {

namespace {

stream::Params params_of(const clsa_window_args* a, float scale) {
  stream::Params p{};
  p.Q = a->Q;
  p.K = a->K;
  p.V = a->V;
  p.count = a->seq_lens;
  p.O = a->O;
  p.lse = a->lse;
  p.q_sl = (long long)a->Hq * a->d;
  p.q_sb = (long long)a->T * a->Hq * a->d;
  p.B = a->B;
  p.Hkv = a->Hkv;
  p.G = a->Hq / a->Hkv;
  p.R = a->T * p.G;
  p.n_max = a->n_max;
  p.seqs = a->B;
  p.T = a->T;
  p.window = std::min(a->window, a->n_max);
  p.sinks = std::min(a->sinks, a->n_max);
  p.scale_log2 = scale * 1.4426950408889634f;
  const int rows = 8 * stream::row_tiles(p.R, a->dtype == CLSA_F32);
  p.nrg = (p.R + rows - 1) / rows;
  return p;
}

// calls f<Cfg>
template <typename F>
auto dispatch(const clsa_window_args* a, int R, F&& f) {
  using namespace stream;
  const bool d128 = a->d == 128;
  if (a->dtype == CLSA_F32) return d128 ? f(Cfg<kFp32, true, false, 128, 1>{}) : f(Cfg<kFp32, true, false, 64, 1>{});
  if (row_tiles(R, false) == 1) return d128 ? f(Cfg<kBf16, false, true, 128, 1>{}) : f(Cfg<kBf16, false, true, 64, 1>{});
  return d128 ? f(Cfg<kBf16, false, true, 128, 2>{}) : f(Cfg<kBf16, false, true, 64, 2>{});
}

// chunks with more rows per KV head than this run in row tiles of 128 on tcgen05
constexpr long long kStreamRows = 64;

bool use_tc(const clsa_window_args* a) {
  return (long long)a->T * (a->Hq / a->Hkv) > kStreamRows && window_tc_supported(a);
}

}  // namespace

size_t window_attn_ws_bytes(const clsa_window_args* a) {
  if (use_tc(a)) return 0;
  const stream::Params p = params_of(a, 1.f);
  return dispatch(a, p.R, [&](auto c) { return stream::ws_bytes<decltype(c)>(p); });
}

cudaError_t launch_window_attn(const clsa_window_args* a, float scale, void* ws_header, void* ws_body, cudaStream_t s) {
  if (use_tc(a)) return launch_window_tc(a, scale, ws_header, s);
  stream::Params p = params_of(a, scale);
  p.ws_header = ws_header;
  return dispatch(a, p.R, [&](auto c) { return stream::launch<decltype(c)>(p, ws_body, s); });
}

}  // namespace clsa
