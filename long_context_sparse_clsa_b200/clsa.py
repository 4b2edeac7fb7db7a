"""Thin Python binding of libclsa.so (include/clsa.h): argument marshalling only.

Every function takes torch CUDA tensors, passes their device pointers and the
current torch stream to the C ABI and raises ``ClsaError`` on a non-OK status.
All arithmetic happens in the library's CUDA kernels; there is no fallback.  If
the library has not been built, the first call raises ``RuntimeError`` naming
the build command.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libclsa.so")

CLSA_F32, CLSA_BF16 = 0, 1
STATUS = {0: "CLSA_OK", 1: "CLSA_ERR_INVALID_ARG", 2: "CLSA_ERR_UNSUPPORTED", 3: "CLSA_ERR_WORKSPACE",
          4: "CLSA_ERR_CUDA", 5: "CLSA_ERR_TIMEOUT", 6: "CLSA_ERR_BAD_INDEX"}

# every symbol include/clsa.h declares
EXPORTS = [
    "clsa_index_scores", "clsa_topk_workspace_size", "clsa_topk", "clsa_topk_noalloc",
    "clsa_gather_kv_workspace_size",
    "clsa_gather_kv", "clsa_sparse_attn_workspace_size", "clsa_sparse_attn",
    "clsa_distill_workspace_size", "clsa_distill_target", "clsa_attention_mass_workspace_size",
    "clsa_attention_mass",
    "clsa_decode_workspace_size", "clsa_decode_step", "clsa_prefill_workspace_size",
    "clsa_prefill_chunk", "clsa_prefill_attention", "clsa_workspace_size", "clsa_workspace_init", "clsa_read_device_status", "clsa_status_string",
    "clsa_selftest_timeout", "clsa_version", "clsa_last_launch_count", "clsa_time_next_call",
    "clsa_timed_event_count",
    "clsa_rope", "clsa_kv8_workspace_size", "clsa_kv8_write", "clsa_kv8_read",
    "clsa_kv8_attn_workspace_size", "clsa_kv8_attn", "clsa_window_attn_workspace_size", "clsa_window_attn",
]


class ClsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {STATUS.get(code, code)}")
        self.code = code
        self.status = STATUS.get(code, str(code))


_vp, _i, _sz, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
_d = ctypes.c_double


class DecodeArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("B", _i), ("n_max", _i), ("d_idx", _i), ("k", _i), ("L", _i),
                ("Hq", _i), ("Hkv", _i), ("d", _i), ("scale", _f),
                ("q_idx", _vp), ("k_idx", _vp), ("K", _vp), ("V", _vp), ("Q", _vp),
                ("seq_lens", _vp), ("O", _vp), ("idx", _vp), ("count", _vp), ("scores", _vp),
                ("lse", _vp), ("K_S", _vp), ("V_S", _vp)]


class PrefillArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("n", _i), ("T", _i), ("d_idx", _i), ("k", _i), ("L", _i),
                ("Hq", _i), ("Hkv", _i), ("d", _i), ("scale", _f),
                ("q_idx", _vp), ("k_idx", _vp), ("K", _vp), ("V", _vp), ("Q", _vp),
                ("O", _vp), ("idx", _vp), ("count", _vp), ("lse", _vp)]


class RopeArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("Nq", _i), ("Nk", _i), ("n_pos", _i), ("Hq", _i), ("Hk", _i), ("d", _i),
                ("rot", _i), ("layout", _i), ("scaling", _i), ("inverse", _i), ("orig_len", _i),
                ("theta", _d), ("factor", _d), ("beta_fast", _d), ("beta_slow", _d), ("mscale", _d),
                ("q", _vp), ("k", _vp), ("pos", _vp), ("q_out", _vp), ("k_out", _vp)]


class Kv8CacheArgs(ctypes.Structure):
    _fields_ = [("B", _i), ("n_max", _i), ("Hkv", _i), ("d", _i), ("block", _i),
                ("K8", _vp), ("V8", _vp), ("k_scale", _vp), ("v_scale", _vp)]


class Kv8AttnArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("B", _i), ("L", _i), ("Hq", _i), ("k", _i), ("scale", _f), ("cache", Kv8CacheArgs),
                ("Q", _vp), ("idx", _vp), ("count", _vp), ("O", _vp), ("lse", _vp)]


class WindowArgs(ctypes.Structure):
    _fields_ = [("dtype", _i), ("B", _i), ("T", _i), ("n_max", _i), ("Hq", _i), ("Hkv", _i), ("d", _i),
                ("window", _i), ("sinks", _i), ("scale", _f),
                ("Q", _vp), ("K", _vp), ("V", _vp), ("seq_lens", _vp), ("O", _vp), ("lse", _vp)]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libclsa.so (once).  Raises RuntimeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m long_context_sparse_clsa_b200.build`")
    lib = ctypes.CDLL(path)
    S = ctypes.c_int
    sig = {
        "clsa_index_scores": (S, [_vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp]),
        "clsa_topk_workspace_size": (_sz, [_i, _i, _i]),
        "clsa_topk": (S, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
        "clsa_topk_noalloc": (S, [_vp, _vp, _i, _i, _i, _vp, _vp, _vp]),
        "clsa_gather_kv_workspace_size": (_sz, []),
        "clsa_gather_kv": (S, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
        "clsa_sparse_attn_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
        "clsa_sparse_attn": (S, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp,
                                 _sz, _vp]),
        "clsa_distill_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
        "clsa_attention_mass_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
        "clsa_attention_mass": (S, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _sz, _vp]),
        "clsa_distill_target": (S, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _vp, _vp, _vp, _sz, _vp]),
        "clsa_decode_workspace_size": (_sz, [ctypes.POINTER(DecodeArgs)]),
        "clsa_decode_step": (S, [ctypes.POINTER(DecodeArgs), _vp, _sz, _vp]),
        "clsa_prefill_workspace_size": (_sz, [ctypes.POINTER(PrefillArgs)]),
        "clsa_prefill_chunk": (S, [ctypes.POINTER(PrefillArgs), _vp, _sz, _vp]),
        "clsa_prefill_attention": (S, [ctypes.POINTER(PrefillArgs), _i, _vp, _sz, _vp]),
        "clsa_workspace_size": (_sz, [_i, _vp]),
        "clsa_workspace_init": (S, [_vp, _sz, _vp]),
        "clsa_read_device_status": (S, [_vp, _vp, ctypes.POINTER(ctypes.c_int64)]),
        "clsa_status_string": (ctypes.c_char_p, [S]),
        "clsa_selftest_timeout": (S, [_i, _vp, _sz, _vp]),
        "clsa_version": (_i, []),
        "clsa_last_launch_count": (_i, []),
        "clsa_time_next_call": (S, [ctypes.POINTER(ctypes.c_void_p), _i]),
        "clsa_timed_event_count": (_i, []),
        "clsa_rope": (S, [ctypes.POINTER(RopeArgs), _vp]),
        "clsa_kv8_workspace_size": (_sz, []),
        "clsa_kv8_write": (S, [ctypes.POINTER(Kv8CacheArgs), _vp, _vp, _vp, _vp, _i, _i, _vp, _sz, _vp]),
        "clsa_kv8_read": (S, [ctypes.POINTER(Kv8CacheArgs), _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _sz, _vp]),
        "clsa_kv8_attn_workspace_size": (_sz, [ctypes.POINTER(Kv8AttnArgs)]),
        "clsa_kv8_attn": (S, [ctypes.POINTER(Kv8AttnArgs), _vp, _sz, _vp]),
        "clsa_window_attn_workspace_size": (_sz, [ctypes.POINTER(WindowArgs)]),
        "clsa_window_attn": (S, [ctypes.POINTER(WindowArgs), _vp, _sz, _vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


# ---------------------------------------------------------------------------- helpers

def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return CLSA_BF16
    if t.dtype == torch.float32:
        return CLSA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise ClsaError(code, where)


def last_launch_count() -> int:
    """Kernel launches made by the most recent library call on this thread."""
    return load_library().clsa_last_launch_count()


class LaunchTimer:
    """Per-launch device times of one library call: arm() before the call; after the
    stream has synchronized, times_ms() gives each launch's duration (events the library
    records before its first launch and after each launch, on the call's stream)."""

    def __init__(self, max_launches: int = 16):
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(max_launches + 1)]
        for e in self.events:  # torch creates the CUDA event on its first record
            e.record()
        torch.cuda.synchronize()
        self._handles = (ctypes.c_void_p * len(self.events))(*[e.cuda_event for e in self.events])

    def arm(self):
        _check(load_library().clsa_time_next_call(self._handles, len(self.events)), "clsa_time_next_call")

    def times_ms(self):
        n = load_library().clsa_timed_event_count()
        return [self.events[i].elapsed_time(self.events[i + 1]) for i in range(n - 1)]


class Workspace:
    """A zero-initialised device workspace of at least ``nbytes`` bytes."""

    def __init__(self, nbytes: int, device=None):
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device or "cuda")
        self.addr = self.buf.data_ptr()
        _check(load_library().clsa_workspace_init(_p(self.buf), self.nbytes, _stream()), "workspace_init")

    @property
    def ptr(self):
        return _p(self.buf)

    def ensure(self, nbytes: int) -> "Workspace":
        return self if nbytes <= self.nbytes else Workspace(nbytes, self.buf.device)

    def status(self, stream=None):
        """(status name, detail) of the first device-detected error; clears it."""
        detail = ctypes.c_int64(0)
        code = load_library().clsa_read_device_status(self.ptr, _stream(stream), ctypes.byref(detail))
        return STATUS.get(code, str(code)), detail.value


def fused_decode_trace(ws: Workspace):
    """Diagnostics of the fused decode step: the per-CTA phase stamps the last step wrote into
    ``ws`` when the library ran with CLSA_TRACE=1 in the environment (int64 [256][64]:
    globaltimer ns per phase; a row whose slot 0 is 0 belongs to no CTA of that step).
    Slot 31 holds the CTA's candidate slot count, plus 2^32 when the candidate windows decided
    the TopK (0 there: the group took the whole-row selection)."""
    return ws.buf[256:256 + 256 * 64 * 8].view(torch.int64).view(256, 64).cpu()


# ---------------------------------------------------------------------------- calls

def index_scores(q_idx, k_idx, seq_lens, scores=None):
    lib = load_library()
    B, n_max, d_idx = k_idx.shape
    if scores is None:
        scores = torch.empty(B, n_max, dtype=torch.float32, device=k_idx.device)
    _check(lib.clsa_index_scores(_p(q_idx), _p(k_idx), _p(seq_lens), B, n_max, d_idx, _dt(k_idx),
                                 _p(scores), _stream()), "clsa_index_scores")
    return scores


def topk(scores, seq_lens, k, ws: Optional[Workspace] = None, idx=None, count=None):
    lib = load_library()
    B, n_max = scores.shape
    need = lib.clsa_topk_workspace_size(B, n_max, k)
    ws = (ws or Workspace(need)).ensure(need)
    idx = idx if idx is not None else torch.empty(B, k, dtype=torch.int32, device=scores.device)
    count = count if count is not None else torch.empty(B, dtype=torch.int32, device=scores.device)
    _check(lib.clsa_topk(_p(scores), _p(seq_lens), B, n_max, k, _p(idx), _p(count), ws.ptr, ws.nbytes,
                         _stream()), "clsa_topk")
    return idx, count


def topk_noalloc(scores, seq_lens, k, idx=None, count=None):
    """clsa_topk without a workspace (scratch inside the library; see clsa.h)."""
    lib = load_library()
    B, n_max = scores.shape
    idx = idx if idx is not None else torch.empty(B, k, dtype=torch.int32, device=scores.device)
    count = count if count is not None else torch.empty(B, dtype=torch.int32, device=scores.device)
    _check(lib.clsa_topk_noalloc(_p(scores), _p(seq_lens), B, n_max, k, _p(idx), _p(count), _stream()),
           "clsa_topk_noalloc")
    return idx, count


def gather_kv(K, V, idx, count, ws: Optional[Workspace] = None, K_S=None, V_S=None):
    lib = load_library()
    B, n_max, Hkv, d = K.shape
    k = idx.shape[1]
    ws = ws or Workspace(lib.clsa_gather_kv_workspace_size())
    K_S = K_S if K_S is not None else torch.zeros(B, k, Hkv, d, dtype=K.dtype, device=K.device)
    V_S = V_S if V_S is not None else torch.zeros(B, k, Hkv, d, dtype=K.dtype, device=K.device)
    _check(lib.clsa_gather_kv(_p(K), _p(V), _p(idx), _p(count), B, n_max, k, Hkv, d, _dt(K), _p(K_S),
                              _p(V_S), ws.ptr, ws.nbytes, _stream()), "clsa_gather_kv")
    return K_S, V_S


def sparse_attn(Q, K_S, V_S, count, scale: float = 0.0, ws: Optional[Workspace] = None, O=None,
                lse=None, want_lse: bool = True):
    """Q [L][B][Hq][d] (or [B][Hq][d] for one layer); K_S/V_S [B][k][Hkv][d]."""
    lib = load_library()
    squeeze = Q.dim() == 3
    Qv = Q.unsqueeze(0) if squeeze else Q
    L, B, Hq, d = Qv.shape
    _, k, Hkv, _ = K_S.shape
    need = lib.clsa_sparse_attn_workspace_size(B, k, L, Hq, Hkv, d)
    ws = (ws or Workspace(need)).ensure(need)
    O = O if O is not None else torch.empty_like(Qv)
    if want_lse and lse is None:
        lse = torch.empty(L, B, Hq, dtype=torch.float32, device=Q.device)
    _check(lib.clsa_sparse_attn(_p(Qv), _p(K_S), _p(V_S), _p(count), B, k, L, Hq, Hkv, d, scale, _dt(Qv),
                                _p(O), _p(lse), ws.ptr, ws.nbytes, _stream()), "clsa_sparse_attn")
    if squeeze:
        return O[0], (lse[0] if lse is not None else None)
    return O, lse


def decode_args(q_idx, k_idx, K, V, Q, seq_lens, k, O, idx, count, scores=None, lse=None, K_S=None,
                V_S=None, scale: float = 0.0) -> DecodeArgs:
    B, n_max, d_idx = k_idx.shape
    L, _, Hq, d = Q.shape
    Hkv = K.shape[2]
    return DecodeArgs(_dt(K), B, n_max, d_idx, k, L, Hq, Hkv, d, scale, _p(q_idx), _p(k_idx), _p(K),
                      _p(V), _p(Q), _p(seq_lens), _p(O), _p(idx), _p(count), _p(scores), _p(lse),
                      _p(K_S), _p(V_S))


def decode_workspace_size(args: DecodeArgs) -> int:
    return load_library().clsa_decode_workspace_size(ctypes.byref(args))


def attention_mass(Q, K, lse_sparse, seq_lens, scale: float = 0.0, ws: Optional[Workspace] = None,
                   mass=None, lse_all=None, want_lse_all: bool = True):
    """Share of the dense softmax mass on the selection (see clsa.h): returns (mass, lse_all),
    both fp32 [L][B][Hq]; lse_sparse is the decode step's lse output."""
    lib = load_library()
    L, B, Hq, d = Q.shape
    _, n_max, Hkv, _ = K.shape
    need = lib.clsa_attention_mass_workspace_size(B, n_max, L, Hq, Hkv, d)
    ws = (ws or Workspace(need)).ensure(need)
    if mass is None:
        mass = torch.empty(L, B, Hq, dtype=torch.float32, device=Q.device)
    if lse_all is None and want_lse_all:
        lse_all = torch.empty(L, B, Hq, dtype=torch.float32, device=Q.device)
    _check(lib.clsa_attention_mass(_p(Q), _p(K), _p(lse_sparse), _p(seq_lens), B, n_max, L, Hq, Hkv, d, scale,
                                   _dt(K), _p(mass), _p(lse_all), ws.ptr, ws.nbytes, _stream()), "clsa_attention_mass")
    return mass, lse_all


def distill_target(Q, K, scores, seq_lens, scale: float = 0.0, ws: Optional[Workspace] = None,
                   want_abar: bool = True, abar=None, kl=None):
    """Distillation target (forward): Abar [B][n_max] (or None) and kl [B] (see clsa.h).
    abar / kl: optional preallocated outputs (fp32 [B][n_max] / [B])."""
    lib = load_library()
    L, B, Hq, d = Q.shape
    _, n_max, Hkv, _ = K.shape
    need = lib.clsa_distill_workspace_size(B, n_max, L, Hq, Hkv, d)
    ws = (ws or Workspace(need)).ensure(need)
    if abar is None and want_abar:
        abar = torch.empty(B, n_max, dtype=torch.float32, device=Q.device)
    if kl is None:
        kl = torch.empty(B, dtype=torch.float32, device=Q.device)
    _check(lib.clsa_distill_target(_p(Q), _p(K), _p(scores), _p(seq_lens), B, n_max, L, Hq, Hkv, d, scale, _dt(Q),
                                   _p(abar), _p(kl), ws.ptr, ws.nbytes, _stream()), "clsa_distill_target")
    return abar, kl, ws


def selftest_timeout(which: int, ws: Optional[Workspace] = None):
    """Launch the failure-detection self-test (see clsa.h); returns its workspace, whose
    status() then reads CLSA_ERR_TIMEOUT with detail 900 + which."""
    ws = ws or Workspace(512)
    _check(load_library().clsa_selftest_timeout(which, ws.ptr, ws.nbytes, _stream()), "clsa_selftest_timeout")
    return ws


def decode_step_args(args: DecodeArgs, ws: Workspace, stream=None):
    """Run one decode step on prepared arguments (no allocation)."""
    _check(load_library().clsa_decode_step(ctypes.byref(args), ws.ptr, ws.nbytes, _stream(stream)),
           "clsa_decode_step")


def decode_step(q_idx, k_idx, K, V, Q, seq_lens, k, scale: float = 0.0, ws: Optional[Workspace] = None,
                compact: bool = False, want_scores: bool = False, want_lse: bool = True):
    """One CLSA decode step.  Returns dict(O, idx, count, lse, scores, K_S, V_S)."""
    B, n_max, _ = k_idx.shape
    L, _, Hq, d = Q.shape
    Hkv = K.shape[2]
    dev = K.device
    out = {
        "O": torch.empty_like(Q),
        "idx": torch.empty(B, k, dtype=torch.int32, device=dev),
        "count": torch.empty(B, dtype=torch.int32, device=dev),
        "lse": torch.empty(L, B, Hq, dtype=torch.float32, device=dev) if want_lse else None,
        "scores": torch.empty(B, n_max, dtype=torch.float32, device=dev) if want_scores else None,
        "K_S": torch.zeros(B, k, Hkv, d, dtype=K.dtype, device=dev) if compact else None,
        "V_S": torch.zeros(B, k, Hkv, d, dtype=K.dtype, device=dev) if compact else None,
    }
    a = decode_args(q_idx, k_idx, K, V, Q, seq_lens, k, out["O"], out["idx"], out["count"], out["scores"],
                    out["lse"], out["K_S"], out["V_S"], scale)
    need = decode_workspace_size(a)
    if need == 0:
        raise ClsaError(1, "clsa_decode_workspace_size")
    ws = (ws or Workspace(need)).ensure(need)
    decode_step_args(a, ws)
    out["ws"] = ws
    return out


def prefill_args(q_idx, k_idx, K, V, Q, k, O, idx, count, lse=None, scale: float = 0.0) -> PrefillArgs:
    T, d_idx = q_idx.shape
    n = k_idx.shape[0]
    L, _, Hq, d = Q.shape
    Hkv = K.shape[1]
    return PrefillArgs(_dt(K), n, T, d_idx, k, L, Hq, Hkv, d, scale, _p(q_idx), _p(k_idx), _p(K), _p(V),
                       _p(Q), _p(O), _p(idx), _p(count), _p(lse))


def prefill_workspace_size(args: PrefillArgs) -> int:
    return load_library().clsa_prefill_workspace_size(ctypes.byref(args))


def prefill_chunk(q_idx, k_idx, K, V, Q, k, scale: float = 0.0, ws: Optional[Workspace] = None,
                  want_lse: bool = True):
    """Causal prefill of T = q_idx.shape[0] rows at the end of an n-token cache."""
    T = q_idx.shape[0]
    L, _, Hq, d = Q.shape
    dev = K.device
    out = {
        "O": torch.empty_like(Q),
        "idx": torch.empty(T, k, dtype=torch.int32, device=dev),
        "count": torch.empty(T, dtype=torch.int32, device=dev),
        "lse": torch.empty(L, T, Hq, dtype=torch.float32, device=dev) if want_lse else None,
    }
    a = prefill_args(q_idx, k_idx, K, V, Q, k, out["O"], out["idx"], out["count"], out["lse"], scale)
    need = prefill_workspace_size(a)
    if need == 0:
        raise ClsaError(1, "clsa_prefill_workspace_size")
    ws = (ws or Workspace(need)).ensure(need)
    _check(load_library().clsa_prefill_chunk(ctypes.byref(a), ws.ptr, ws.nbytes, _stream()),
           "clsa_prefill_chunk")
    out["ws"] = ws
    return out


def prefill_attention(q_idx, k_idx, K, V, Q, k, idx, count, mode: int = 0, scale: float = 0.0,
                      ws: Optional[Workspace] = None, O=None, lse=None, want_lse: bool = True):
    """The attention stage of a prefill chunk over a selection already in idx / count (as
    prefill_chunk returns it).  mode 0: per row; mode 1: key-centric row pairs."""
    T = q_idx.shape[0]
    L, _, Hq, d = Q.shape
    O = O if O is not None else torch.empty_like(Q)
    if want_lse and lse is None:
        lse = torch.empty(L, T, Hq, dtype=torch.float32, device=K.device)
    a = prefill_args(q_idx, k_idx, K, V, Q, k, O, idx, count, lse, scale)
    need = prefill_workspace_size(a)
    ws = (ws or Workspace(need)).ensure(need)
    _check(load_library().clsa_prefill_attention(ctypes.byref(a), int(mode), ws.ptr, ws.nbytes, _stream()),
           "clsa_prefill_attention")
    return O, lse


# ---------------------------------------------------------------------------- positions, 8-bit cache

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _now(t: torch.Tensor, what: str):
    """(current device, its current stream's handle), what a call runs on; t: its first tensor."""
    if not t.is_cuda:
        raise ValueError(f"{what}: a contiguous CUDA tensor is wanted")
    dev = torch.cuda.current_device()
    return dev, _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream


def _here(t: Optional[torch.Tensor], dev: int, what: str, shape=None, dtype=None):
    """The address of a contiguous tensor on the current device, of the given shape and dtype."""
    if t is None:
        return None
    if t.get_device() != dev or not t.is_contiguous():
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{what}: a contiguous CUDA tensor is wanted")
        raise ValueError(f"{what} is on {t.device}, the current device is cuda:{dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: {dtype} is wanted, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(shape)} is wanted, got {tuple(t.shape)}")
    return t.data_ptr()


def _ws(ws: Workspace, dev: int) -> int:
    if ws.buf.get_device() != dev:
        raise ValueError(f"the workspace is on {ws.buf.device}, the current device is cuda:{dev}")
    return ws.addr


_ROPE_LAYOUT = {"half": 0, "interleaved": 1}
_ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "by_parts": 3}


def rope(q, k, pos, rot: Optional[int] = None, layout: str = "half", theta: float = 10000.0, scaling: str = "plain",
         factor: float = 1.0, orig_len: int = 1, beta_fast: float = 32.0, beta_slow: float = 1.0, mscale: float = 1.0,
         inverse: bool = False, q_out=None, k_out=None):
    """Rotary positions (see clsa.h): q [..., Hq, d] and k [..., Hk, d] (either may be None), pos
    int32 [n_pos]; the rows before the heads run over positions with pos fastest, so Q [L][B][Hq][d]
    takes pos [B].  inverse=True is the transpose (the gradient).  Returns (q_out, k_out);
    q_out=q and k_out=k work in place."""
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    d, dt = x.shape[-1], x.dtype
    Hq, Hk = (q.shape[-2] if q is not None else 0), (k.shape[-2] if k is not None else 0)
    if k is not None and k.shape[-1] != d:
        raise ValueError(f"k: head dimension {d} is wanted, got {k.shape[-1]}")
    dev, stream = _now(x, "q" if q is not None else "k")
    qa, ka = _here(q, dev, "q", None, dt), _here(k, dev, "k", None, dt)
    if q is not None and q_out is None:
        q_out = torch.empty_like(q)
        qo = q_out.data_ptr()
    else:
        qo = _here(q_out, dev, "q_out", q.shape if q is not None else None, dt)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k)
        ko = k_out.data_ptr()
    else:
        ko = _here(k_out, dev, "k_out", k.shape if k is not None else None, dt)
    a = RopeArgs(_dt(x), q.numel() // (Hq * d) if Hq else 0, k.numel() // (Hk * d) if Hk else 0, pos.numel(), Hq, Hk, d,
                 d if rot is None else rot, _ROPE_LAYOUT[layout], _ROPE_SCALING[scaling], bool(inverse), orig_len,
                 theta, factor, beta_fast, beta_slow, mscale, qa, ka, _here(pos, dev, "pos", None, torch.int32), qo, ko)
    _check(load_library().clsa_rope(ctypes.byref(a), stream), "clsa_rope")
    return q_out, k_out


class Kv8Cache:
    """Handle of an 8-bit K/V cache (see clsa.h): codes K8, V8 [B][n_max][Hkv][d] (torch.float8_e4m3fn
    or uint8) and scales k_scale, v_scale fp32 [B][ceil(n_max / block)][Hkv].  It holds the tensors."""

    def __init__(self, K8, V8, k_scale, v_scale, block: int = 64):
        if K8.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise TypeError(f"K8: torch.float8_e4m3fn or torch.uint8 is wanted, got {K8.dtype}")
        self.B, self.n_max, self.Hkv, self.d = K8.shape
        self.block = int(block)
        self.K8, self.V8, self.k_scale, self.v_scale = K8, V8, k_scale, v_scale
        scales = (self.B, -(-self.n_max // max(self.block, 1)), self.Hkv)
        if not K8.is_cuda:
            raise ValueError("K8: a contiguous CUDA tensor is wanted")
        self.device = dev = K8.get_device()
        self.args = Kv8CacheArgs(self.B, self.n_max, self.Hkv, self.d, self.block, _here(K8, dev, "K8"),
                                 _here(V8, dev, "V8", K8.shape, K8.dtype), _here(k_scale, dev, "k_scale", scales, torch.float32),
                                 _here(v_scale, dev, "v_scale", scales, torch.float32))
        self._ref = ctypes.byref(self.args)

    @classmethod
    def empty(cls, B: int, n_max: int, Hkv: int, d: int, block: int = 64, device=None) -> "Kv8Cache":
        """A cache that holds nothing yet (its bytes are zero)."""
        dev = device or "cuda"
        codes = [torch.zeros(B, n_max, Hkv, d, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.zeros(B, -(-n_max // block), Hkv, dtype=torch.float32, device=dev) for _ in range(2)]
        return cls(*codes, *scales, block)


def _on(cache: "Kv8Cache"):
    """_now(), where the cache is on the current device."""
    dev, stream = _now(cache.K8, "cache")
    if cache.device != dev:
        raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{dev}")
    return dev, stream


def kv8_write(cache: Kv8Cache, K, V, start, count=None, ws: Optional[Workspace] = None) -> Kv8Cache:
    """Quantise K, V [B][T][Hkv][d] into the cache as tokens start[b] + t, t < count[b] (see clsa.h)."""
    lib = load_library()
    T = K.shape[1]
    shape = (cache.B, T, cache.Hkv, cache.d)
    ws = ws or Workspace(lib.clsa_kv8_workspace_size(), K.device)
    dev, stream = _on(cache)
    _check(lib.clsa_kv8_write(cache._ref, _here(K, dev, "K", shape), _here(V, dev, "V", shape, K.dtype),
                              _here(start, dev, "start", (cache.B,), torch.int32),
                              _here(count, dev, "count", (cache.B,), torch.int32), T, _dt(K), _ws(ws, dev), ws.nbytes, stream),
           "clsa_kv8_write")
    return cache


def kv8_read(cache: Kv8Cache, K=None, V=None, start=None, idx=None, count=None, T: Optional[int] = None,
             dtype=torch.bfloat16, ws: Optional[Workspace] = None):
    """Rows of the cache as K, V [B][T][Hkv][d]: tokens idx[b][t], or start[b] + t (see clsa.h).
    K and V may be given (rows from count[b] on are left alone); else they start as zeros."""
    lib = load_library()
    if K is None:
        T = idx.shape[1] if idx is not None else T
        if T is None:
            raise ValueError("T, idx or K is wanted")
        K = torch.zeros(cache.B, T, cache.Hkv, cache.d, dtype=dtype, device=cache.K8.device)
    if V is None:
        V = torch.zeros_like(K)
    T = K.shape[1]
    shape = (cache.B, T, cache.Hkv, cache.d)
    ws = ws or Workspace(lib.clsa_kv8_workspace_size(), K.device)
    dev, stream = _on(cache)
    _check(lib.clsa_kv8_read(cache._ref, _here(start, dev, "start", (cache.B,), torch.int32),
                             _here(idx, dev, "idx", (cache.B, T), torch.int32),
                             _here(count, dev, "count", (cache.B,), torch.int32), T, _dt(K), _here(K, dev, "K", shape),
                             _here(V, dev, "V", shape, K.dtype), _ws(ws, dev), ws.nbytes, stream), "clsa_kv8_read")
    return K, V


def _kv8_attn_args(dev, Q, cache, count, idx, scale, O, lse) -> Kv8AttnArgs:
    L, B, Hq, d = Q.shape
    if d != cache.d:
        raise ValueError(f"Q: head dimension {cache.d} is wanted, got {d}")
    if idx is not None and (idx.dim() != 2 or idx.shape[0] != B):
        raise ValueError(f"idx: shape [{B}][k] is wanted, got {tuple(idx.shape)}")
    return Kv8AttnArgs(_dt(Q), B, L, Hq, idx.shape[1] if idx is not None else 0, scale, cache.args, _here(Q, dev, "Q"),
                       _here(idx, dev, "idx", None, torch.int32), _here(count, dev, "count", (B,), torch.int32),
                       _here(O, dev, "O", Q.shape, Q.dtype), _here(lse, dev, "lse", (L, B, Hq), torch.float32))


def _need(size: int, where: str) -> int:
    if size == 0:  # the arguments are refused: the size calls do not say why
        raise ClsaError(1, where)
    return size


def kv8_attn_workspace_size(Q, cache: Kv8Cache, idx=None) -> int:
    """Workspace bytes of kv8_attn for these tensors (Q [L][B][Hq][d] or [B][Hq][d])."""
    Qv = Q.unsqueeze(0) if Q.dim() == 3 else Q
    a = _kv8_attn_args(_on(cache)[0], Qv, cache, None, idx, 0.0, Qv, None)
    a.count = a.Q  # any aligned address: the size does not read it
    return _need(load_library().clsa_kv8_attn_workspace_size(ctypes.byref(a)), "clsa_kv8_attn_workspace_size")


def kv8_attn(Q, cache: Kv8Cache, count, idx=None, scale: float = 0.0, ws: Optional[Workspace] = None, O=None, lse=None,
             want_lse: bool = True):
    """Attention over the 8-bit cache (see clsa.h).  Q [L][B][Hq][d] (or [B][Hq][d] for one layer);
    count int32 [B] cached tokens, or with idx int32 [B][k] selected ones.  cache.B is B or 1.
    Returns (O, lse), shaped as Q (lse without d; None where not wanted)."""
    lib = load_library()
    squeeze = Q.dim() == 3
    if squeeze:
        Q, O, lse = Q.unsqueeze(0), O if O is None else O.unsqueeze(0), lse if lse is None else lse.unsqueeze(0)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
    dev, stream = _on(cache)
    a = _kv8_attn_args(dev, Q, cache, count, idx, scale, O, lse)
    ref = ctypes.byref(a)
    if ws is None:
        ws = Workspace(lib.clsa_kv8_attn_workspace_size(ref), Q.device)  # 0: the call says why
    _check(lib.clsa_kv8_attn(ref, _ws(ws, dev), ws.nbytes, stream), "clsa_kv8_attn")
    return (O[0], lse[0] if lse is not None else None) if squeeze else (O, lse)


def _window_args(dev, Q, K, V, seq_lens, window, sinks, scale, O, lse) -> WindowArgs:
    B, T, Hq, d = Q.shape
    n_max, Hkv = K.shape[1], K.shape[2]
    shape = (B, n_max, Hkv, d)
    return WindowArgs(_dt(Q), B, T, n_max, Hq, Hkv, d, window, sinks, scale, _here(Q, dev, "Q"),
                      _here(K, dev, "K", shape, Q.dtype), _here(V, dev, "V", shape, Q.dtype),
                      _here(seq_lens, dev, "seq_lens", (B,), torch.int32), _here(O, dev, "O", Q.shape, Q.dtype),
                      _here(lse, dev, "lse", (B, T, Hq), torch.float32))


def window_attn_workspace_size(Q, K, window: int, sinks: int = 0) -> int:
    """Workspace bytes of window_attn for these tensors."""
    a = _window_args(_now(Q, "Q")[0], Q, K, K, None, window, sinks, 0.0, Q, None)
    a.seq_lens = a.Q  # any aligned address: the size does not read it
    return _need(load_library().clsa_window_attn_workspace_size(ctypes.byref(a)), "clsa_window_attn_workspace_size")


def window_attn(Q, K, V, seq_lens, window: int, sinks: int = 0, scale: float = 0.0, ws: Optional[Workspace] = None,
                O=None, lse=None, want_lse: bool = True):
    """Attention of the T newest tokens of each sequence with a sliding window and sink tokens (see
    clsa.h): Q [B][T][Hq][d], K, V [B][n_max][Hkv][d], seq_lens int32 [B].  Returns (O, lse)."""
    lib = load_library()
    if O is None:
        O = torch.empty_like(Q)
    if lse is None and want_lse:
        lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
    dev, stream = _now(Q, "Q")
    a = _window_args(dev, Q, K, V, seq_lens, window, sinks, scale, O, lse)
    ref = ctypes.byref(a)
    if ws is None:
        ws = Workspace(lib.clsa_window_attn_workspace_size(ref), Q.device)  # 0: the call says why
    _check(lib.clsa_window_attn(ref, _ws(ws, dev), ws.nbytes, stream), "clsa_window_attn")
    return O, lse


def to_device(inp, device="cuda"):
    """Copy an ``inputs.Inputs`` bundle to the device as torch tensors (bf16 or fp32)."""
    import numpy as np

    def conv(a):
        if a.dtype == np.uint16:
            return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).to(device)
        return torch.from_numpy(np.ascontiguousarray(a)).to(device)
    return {"q_idx": conv(inp.q_idx), "k_idx": conv(inp.k_idx), "K": conv(inp.K), "V": conv(inp.V),
            "Q": conv(inp.Q), "seq_lens": torch.from_numpy(inp.seq_lens.astype(np.int32)).to(device)}
