"""Argument errors of the cache operators, returned before anything is launched (no GPU)."""
import ctypes

import pytest
import torch

from long_context_sparse_clsa_b200 import clsa

NULL = None
P, ODD4, ODD2 = 4096, 4100, 4098  # addresses: 16-byte aligned, 4-byte, 2-byte (never dereferenced)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from long_context_sparse_clsa_b200.build import build
    build()
    return clsa.load_library()


def rope_args(**kw):
    a = clsa.RopeArgs(1, 6, 3, 3, 8, 2, 128, 64, 0, 0, 0, 1, 10000.0, 1.0, 32.0, 1.0, 1.0, P, P, P, P, P)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    ({"dtype": 7}, INVALID), ({"n_pos": 0}, INVALID), ({"Nq": 7}, INVALID), ({"Nk": 4}, INVALID), ({"pos": NULL}, INVALID),
    ({"q": NULL}, INVALID), ({"k_out": NULL}, INVALID), ({"q": NULL, "q_out": NULL}, INVALID), ({"Nk": 0}, INVALID),
    ({"q": NULL, "q_out": NULL, "Nq": 0, "k": NULL, "k_out": NULL, "Nk": 0}, INVALID),
    ({"Hq": 0}, INVALID), ({"layout": 2}, INVALID), ({"scaling": 4}, INVALID), ({"scaling": -1}, INVALID), ({"theta": 1.0}, INVALID),
    ({"theta": float("nan")}, INVALID), ({"theta": float("inf")}, INVALID), ({"mscale": float("nan")}, INVALID),
    ({"scaling": 1, "factor": 0.0}, INVALID), ({"scaling": 2, "factor": float("inf")}, INVALID),
    ({"scaling": 3, "orig_len": 0}, INVALID), ({"scaling": 3, "beta_fast": 1.0}, INVALID), ({"scaling": 3, "beta_slow": -1.0}, INVALID),
    ({"d": 96}, UNSUPPORTED), ({"rot": 8}, UNSUPPORTED), ({"rot": 24}, UNSUPPORTED), ({"rot": 144}, UNSUPPORTED), ({"rot": 0}, UNSUPPORTED),
    ({"q": ODD4}, INVALID), ({"k_out": ODD4}, INVALID), ({"pos": ODD2}, INVALID), ({"n_pos": (1 << 30) + 1, "Nq": (1 << 30) + 1, "Nk": (1 << 30) + 1}, UNSUPPORTED)])
def test_rope_rejects_bad_args(lib, kw, want):
    assert lib.clsa_rope(ctypes.byref(rope_args(**kw)), NULL) == want


def test_null_structs(lib):
    assert lib.clsa_rope(NULL, NULL) == INVALID
    assert lib.clsa_kv8_write(NULL, P, P, P, NULL, 1, 1, P, 256, NULL) == INVALID
    assert lib.clsa_kv8_read(NULL, NULL, NULL, NULL, 1, 1, P, P, P, 256, NULL) == INVALID
    assert lib.clsa_kv8_attn(NULL, P, 1 << 30, NULL) == INVALID and lib.clsa_kv8_attn_workspace_size(NULL) == 0
    assert lib.clsa_window_attn(NULL, P, 1 << 30, NULL) == INVALID and lib.clsa_window_attn_workspace_size(NULL) == 0


def cache(**kw):
    c = clsa.Kv8CacheArgs(2, 100, 2, 128, 64, P, P, P, P)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [({"B": 0}, INVALID), ({"n_max": 0}, INVALID), ({"Hkv": 0}, INVALID), ({"K8": NULL}, INVALID),
              ({"v_scale": NULL}, INVALID), ({"d": 80}, UNSUPPORTED), ({"block": 48}, UNSUPPORTED), ({"block": 0}, UNSUPPORTED),
              ({"block": 256}, UNSUPPORTED), ({"n_max": (1 << 30) + 1}, UNSUPPORTED), ({"V8": ODD4}, INVALID), ({"k_scale": ODD2}, INVALID)]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_kv8_calls_reject_bad_caches(lib, kw, want):
    c = cache(**kw)
    r = ctypes.byref(c)
    assert lib.clsa_kv8_write(r, P, P, P, NULL, 1, 1, P, 256, NULL) == want
    assert lib.clsa_kv8_read(r, NULL, NULL, NULL, 1, 1, P, P, P, 256, NULL) == want
    a = attn_args(cache=c)
    assert lib.clsa_kv8_attn(ctypes.byref(a), P, 1 << 30, NULL) == want


def test_kv8_write_and_read_reject_bad_args(lib):
    r = ctypes.byref(cache())
    w = lambda K=P, V=P, start=P, count=NULL, T=1, dt=1, ws=P, n=256: lib.clsa_kv8_write(r, K, V, start, count, T, dt, ws, n, NULL)  # noqa: E731
    assert [w(K=NULL), w(V=NULL), w(start=NULL), w(T=0), w(dt=2), w(K=ODD4), w(start=ODD2), w(count=ODD2)] == [INVALID] * 8
    assert [w(ws=NULL), w(n=255), w(ws=ODD4)] == [WORKSPACE] * 3
    rd = lambda start=NULL, idx=NULL, count=NULL, T=1, dt=1, K=P, V=P, ws=P, n=256: lib.clsa_kv8_read(r, start, idx, count, T, dt, K, V, ws, n, NULL)  # noqa: E731
    assert [rd(K=NULL), rd(V=ODD4), rd(T=0), rd(dt=9), rd(start=P, idx=P), rd(idx=ODD2), rd(count=ODD2)] == [INVALID] * 7
    assert [rd(ws=NULL), rd(n=0)] == [WORKSPACE] * 2
    assert lib.clsa_kv8_workspace_size() == 256


def attn_args(**kw):
    a = clsa.Kv8AttnArgs(1, 2, 1, 8, 0, 0.0, cache(), P, NULL, P, P, NULL)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    ({"dtype": 3}, INVALID), ({"B": 0}, INVALID), ({"L": 0}, INVALID), ({"Hq": 0}, INVALID), ({"B": 3}, INVALID), ({"Q": NULL}, INVALID),
    ({"count": NULL}, INVALID), ({"O": NULL}, INVALID), ({"idx": P, "k": 0}, INVALID), ({"Hq": 7}, UNSUPPORTED),
    ({"idx": P, "k": (1 << 24) + 1}, UNSUPPORTED), ({"L": 1 << 24}, UNSUPPORTED), ({"Q": ODD4}, INVALID), ({"O": ODD4}, INVALID),
    ({"idx": ODD2, "k": 1}, INVALID), ({"lse": ODD2}, INVALID)])
def test_kv8_attn_rejects_bad_args(lib, kw, want):
    a = attn_args(**kw)
    assert lib.clsa_kv8_attn(ctypes.byref(a), P, 1 << 30, NULL) == want
    assert lib.clsa_kv8_attn_workspace_size(ctypes.byref(a)) == 0


def window_args(**kw):
    a = clsa.WindowArgs(1, 2, 3, 100, 8, 2, 128, 16, 4, 0.0, P, P, P, P, P, NULL)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,want", [
    ({"dtype": 3}, INVALID), ({"B": 0}, INVALID), ({"T": 0}, INVALID), ({"n_max": 0}, INVALID), ({"Hq": 0}, INVALID), ({"Hkv": 0}, INVALID),
    ({"window": 0}, INVALID), ({"sinks": -1}, INVALID), ({"Q": NULL}, INVALID), ({"V": NULL}, INVALID), ({"seq_lens": NULL}, INVALID),
    ({"O": NULL}, INVALID), ({"d": 96}, UNSUPPORTED), ({"Hq": 9}, UNSUPPORTED), ({"Hq": 258}, UNSUPPORTED), ({"T": (1 << 30) + 1}, UNSUPPORTED),
    ({"n_max": (1 << 30) + 1}, UNSUPPORTED), ({"T": 1 << 28}, UNSUPPORTED), ({"K": ODD4}, INVALID), ({"seq_lens": ODD2}, INVALID), ({"lse": ODD2}, INVALID)])
def test_window_attn_rejects_bad_args(lib, kw, want):
    a = window_args(**kw)
    assert lib.clsa_window_attn(ctypes.byref(a), P, 1 << 30, NULL) == want
    assert lib.clsa_window_attn_workspace_size(ctypes.byref(a)) == 0


def test_attention_wants_its_workspace(lib):
    for a, call, size in ((attn_args(), lib.clsa_kv8_attn, lib.clsa_kv8_attn_workspace_size),
                          (window_args(), lib.clsa_window_attn, lib.clsa_window_attn_workspace_size)):
        r = ctypes.byref(a)
        need = size(r)
        assert need > 256
        assert [call(r, NULL, need, NULL), call(r, P, need - 1, NULL), call(r, ODD4, need, NULL)] == [WORKSPACE] * 3


def test_python_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        clsa.rope(x, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        clsa.rope(None, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        clsa.Kv8Cache(torch.zeros(1, 16, 1, 64, dtype=torch.uint8), torch.zeros(1, 16, 1, 64, dtype=torch.uint8),
                      torch.zeros(1, 1, 1), torch.zeros(1, 1, 1), 16)
    with pytest.raises(TypeError):
        clsa.Kv8Cache(x, x, x, x, 16)
    with pytest.raises(ValueError):
        clsa.window_attn(torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 9, 1, 64, dtype=torch.bfloat16),
                         torch.zeros(1, 9, 1, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32), 4)


def test_caches_behind_the_reach_of_their_loads_are_refused(lib):
    """More than 2^31 - 4096 rows over all sequences."""
    for n, want in ((1 << 29, UNSUPPORTED), ((1 << 29) - 1024, WORKSPACE)):
        a = attn_args(B=4, cache=cache(B=4, n_max=n, Hkv=1))
        assert lib.clsa_kv8_attn(ctypes.byref(a), P, 0, NULL) == want
        a = window_args(B=4, n_max=n, Hkv=1)
        assert lib.clsa_window_attn(ctypes.byref(a), P, 0, NULL) == want


def test_rope_refuses_frequencies_out_of_range(lib):
    """Frequencies that leave a double's range, or that no longer have a part of a turn."""
    for kw in ({"scaling": 1, "factor": 1e-310}, {"scaling": 1, "factor": 1e-17}, {"scaling": 2, "factor": 1e-300},
               {"scaling": 3, "factor": 1e-300, "orig_len": 1}):
        assert lib.clsa_rope(ctypes.byref(rope_args(**kw)), NULL) == INVALID, kw


def test_head_counts_behind_the_range_are_refused(lib):
    for h, want in (((1 << 16) + 1, UNSUPPORTED), (1 << 16, WORKSPACE)):
        assert lib.clsa_window_attn(ctypes.byref(window_args(B=1, T=1, n_max=4, Hq=h, Hkv=h)), P, 0, NULL) == want
        c = cache(B=1, n_max=4, Hkv=h)
        assert lib.clsa_kv8_attn(ctypes.byref(attn_args(B=1, Hq=h, cache=c)), P, 0, NULL) == want
        assert lib.clsa_kv8_write(ctypes.byref(c), P, P, P, NULL, 1, 1, P, 0, NULL) == want
        assert lib.clsa_kv8_read(ctypes.byref(c), NULL, NULL, NULL, 1, 1, P, P, P, 0, NULL) == want
