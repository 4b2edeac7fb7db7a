// Attention with a sliding window and sink tokens: few rows stream over the cache (stream_attn.cuh), many run
// in row tiles on tcgen05 (window_tc.cu).  fp32 always streams.
#include <cmath>

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

// Which form is faster, by a fit to both over T = 8 to 512, windows 256 to 8192, 1 to 4 sequences and five
// head layouts (d = 128, us): the streaming form takes 10 + 1.6e-3 per (16 rows, 16 tokens), at
// 75 to 105 TFLOP/s whatever the split; the tcgen05 form 9.5 + 1.55 per token tile and round of the
// SMs, since few rows leave most SMs idle.  E.g. T = 24, window 8192: 39 and 98; T = 96: 133 and 110;
// T = 48, window 256: 10 and 14; T = 512, window 1024: 125 and 25.
bool use_tc(const clsa_window_args* a) {
  if (!window_tc_supported(a) || (long long)a->T * (a->Hq / a->Hkv) <= 16) return false;  // 16 rows: HBM is the bound
  const double G = a->Hq / a->Hkv, TQ = 128 / (a->Hq / a->Hkv), sms = std::max(1, device_info().sm_count);
  const double seen = std::min((double)a->n_max, (double)a->window + a->sinks);  // of one row
  const double groups = std::ceil(a->T * G / 16) * a->B * a->Hkv, items = std::ceil(a->T / (2 * TQ)) * a->B * a->Hkv;
  const double stream_us = 10 + 1.6e-3 * (a->d / 128.0) * groups * std::ceil((seen + 15) / 16) * (148 / sms);
  const double tc_us = 9.5 + 1.55 * std::ceil(items / sms) * std::ceil(std::min((double)a->n_max, seen + 2 * TQ) / 128);
  return tc_us < stream_us;
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
