"""Pins of the cache operators' float64 references (no GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C


def test_e4m3_decode_matches_torch_for_every_code():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(C.e4m3_decode(codes), want)


def test_e4m3_encode_matches_torch_and_saturates():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 9, 4000), C.E4M3_VALUES,
                        (C.E4M3_VALUES[1:] + C.E4M3_VALUES[:-1]) / 2, [2.0 ** -10, 3 * 2.0 ** -11]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(C.e4m3_encode(x), want)
    np.testing.assert_array_equal(C.e4m3_encode([449, 1e9, math.inf, -math.inf, math.nan]), [126, 126, 126, 254, 127])


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.1, 1), (224.0, -1), (3.5, -7), (0.0, -100), (1e-38, -100), (2.0 ** 126, 118),
                                    (3.4e38, 119)])
def test_kv8_scale(amax, e):
    assert C.kv8_scale(amax) == 2.0 ** e


def test_kv8_appending_token_by_token_keeps_the_values():
    """Appended one at a time, a block's codes end within one subnormal step of those written at once."""
    rng = np.random.default_rng(1)
    X = rng.standard_normal((1, 40, 2, 16)) * np.exp(rng.standard_normal((1, 40, 1, 1)) * 2)
    z, s0 = np.zeros((1, 48, 2, 16), np.uint8), np.zeros((1, 3, 2))
    once, so = C.kv8_write(z, s0, X, [0], None, 16)
    c, s = z, s0
    for t in range(40):
        c, s = C.kv8_write(c, s, X[:, t:t + 1], [t], None, 16)
    np.testing.assert_array_equal(s, so)
    a, b = C.kv8_values(once, so, 16)[:, :40], C.kv8_values(c, s, 16)[:, :40]
    step = 2.0 ** -9 * np.repeat(so, 16, axis=1)[:, :40, :, None]
    assert (np.abs(a - b) <= step).all()
    normal = np.abs(X) >= 2.0 ** -6 * np.repeat(so, 16, axis=1)[:, :40, :, None]
    assert (np.abs(b - X)[normal] <= 2.0 ** -4 * np.abs(X)[normal]).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_keeps_products_of_equal_offsets_and_inverts(layout):
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    f = C.rope_freqs(32, 10000.0)
    dots = [(C.rope(q, [p], f, layout) * C.rope(k, [p - 7], f, layout)).sum() for p in (7, 100, 5000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)
    back = C.rope(C.rope(q, [123], f, layout, mscale=1.25), [123], f, layout, inverse=True)
    np.testing.assert_allclose(back[..., :32], 1.25 * q[..., :32], atol=1e-12)
    np.testing.assert_array_equal(back[..., 32:], q[..., 32:])


def test_rope_gradient_is_the_transpose():
    """Differences of sum(w * rope(x)) are rope^T w, mscale included."""
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    f = C.rope_freqs(48, 500000.0, "by_parts", 4.0, 8192)
    want = C.rope(w, [777], f, "half", 1.1, inverse=True)
    for i in (0, 5, 23, 24, 47, 48, 63):
        e = np.zeros_like(x)
        e[0, 0, i] = 1e-6
        d = ((C.rope(x + e, [777], f, "half", 1.1) - C.rope(x - e, [777], f, "half", 1.1)) * w).sum() / 2e-6
        assert abs(d - want[0, 0, i]) < 1e-8


def test_by_parts_frequencies_keep_the_fast_and_stretch_the_slow():
    f, g = C.rope_freqs(128, 500000.0), C.rope_freqs(128, 500000.0, "by_parts", 4.0, 8192)
    turns = 8192 * f / (2 * math.pi)
    np.testing.assert_array_equal(g[turns >= 32], f[turns >= 32])
    np.testing.assert_allclose(g[turns <= 1], f[turns <= 1] / 4)
    assert (np.diff(g) < 0).all()


def test_window_sees():
    assert C.window_sees(10, 7, 3, 2).nonzero()[0].tolist() == [0, 1, 5, 6, 7]
    assert C.window_sees(10, 1, 3, 4).nonzero()[0].tolist() == [0, 1]
    assert not C.window_sees(10, -1, 3, 4).any()
