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
  const int rows = 8 * stream::row_tiles(p.R, false);
  p.nrg = (p.R + rows - 1) / rows;
  return p;
}

// calls f<Cfg>
template <typename F>
auto dispatch(const clsa_window_args* a, int R, F&& f) {
  using namespace stream;
  const bool d128 = a->d == 128, one = row_tiles(R, false) == 1;
  if (a->dtype == CLSA_F32) {
    if (one) return d128 ? f(Cfg<kFp32, true, true, 128, 1>{}) : f(Cfg<kFp32, true, true, 64, 1>{});
    return d128 ? f(Cfg<kFp32, true, true, 128, 2>{}) : f(Cfg<kFp32, true, true, 64, 2>{});
  }
  if (one) return d128 ? f(Cfg<kBf16, false, true, 128, 1>{}) : f(Cfg<kBf16, false, true, 64, 1>{});
  return d128 ? f(Cfg<kBf16, false, true, 128, 2>{}) : f(Cfg<kBf16, false, true, 64, 2>{});
}

// Which form is faster, by a fit to both over T = 2 to 512, windows 64 to 4096, 1 and 3 sequences and six
// head layouts: of 352 shapes with more than 16 rows it picks one that is over 15 % slower 7 times, and on the
// average loses 0.8 % (us, 148 SMs).  The streaming form: a start, 1.5e-3 per (16 rows, 16 tokens) at
// d = 128, more where so many units share the SMs that a CTA goes through several.  The tcgen05
// form: per round of the SMs 2, and 1.45 (items of one row tile: 1.35) per token tile, however few
// SMs have an item.  E.g. 32 heads on 8, d = 128: T = 24, W = 4096 25 streaming and 52; T = 96, W = 1024
// 30 and 18; 6 on 3, d = 64: T = 48, W = 4096 13 and 45; T = 512, W = 1024 28 and 16.
bool use_tc(const clsa_window_args* a) {
  if (!window_tc_supported(a) || (long long)a->T * (a->Hq / a->Hkv) <= 16) return false;  // 16 rows: HBM is the bound
  const double G = a->Hq / a->Hkv, TQ = 128 / (a->Hq / a->Hkv), sms = std::max(1, device_info().sm_count);
  const double seen = std::min((double)a->n_max, (double)a->window + a->sinks);  // of one row
  const double groups = std::ceil(a->T * G / 16) * a->B, units = groups * a->Hkv;
  const double stream_us = 10 + 1.5e-3 * (0.5 + a->d / 256.0) * units * std::ceil((seen + 15) / 16) * (148 / sms) + (groups > 32 ? 6 : 0);
  const double items = std::ceil(a->T / (2 * TQ)) * a->B * a->Hkv, over = std::fmod(items, sms);
  const bool single = over > 0 && 2 * over <= sms;
  const auto tiles = [&](double rows) { return std::ceil(std::min((double)a->n_max, seen + rows) / 128); };
  const double rounds = std::floor(items / sms) + (over > 0 && !single ? 1 : 0);
  const double tc_us = 4 + rounds * (2 + 1.45 * tiles(2 * TQ)) + (single ? 2 + 1.35 * tiles(TQ) : 0);
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
