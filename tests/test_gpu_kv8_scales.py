"""Attention over, and writes into, an 8-bit cache whose scales another program made: any finite value from 0
up, not only powers of two.

A code stands for code * scale.  Tolerances as in test_gpu_cache_attn.py, with two differences.  For fp32 rows a
weight enters the second product relative to the next power of two above its token's scale, so the largest
is at least 2^6, not 2^7: a half below 2^-14 costs 2^-25 / 2^6 = 2^-31 where that file has 2^-32.  For bf16 rows the
weight takes the logarithm of the scale, here of size 9 and less: off by 2^-21 and, in the sum with the score, by as
much again, 2^-20 ln 2 of the weight; that file's 2^-11 for its rounding to a half goes up by that."""
import numpy as np
import pytest
import torch

from long_context_sparse_clsa_b200 import clsa
from oracle import cache_oracle as C
from test_gpu_cache import DT, cache_of, dev, f64, host, rows
from test_gpu_cache_attn import check, run8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_clsa_b200.build import build
    build()
    clsa.load_library()


def check_scaled(cache, Q, O, lse, counts, idx, dtype):
    kc, vc, ks, vs = host(cache)
    K, V = C.kv8_values(kc, ks, cache.block), C.kv8_values(vc, vs, cache.block)
    toks = [np.arange(c) if idx is None else idx[b, :c] for b, c in enumerate(counts)]
    wantO, want_lse = C.attention(f64(Q), K, V, toks)
    A, _ = C.attention(f64(Q), K, np.abs(V), toks)
    sc, G = cache.d ** -0.5, Q.shape[2] // cache.Hkv
    mag, floor = np.zeros(want_lse.shape), np.zeros(wantO.shape)
    codes = C.e4m3_decode(vc)
    for b, tk in enumerate(toks):
        for h in range(Q.shape[2]):
            if len(tk):
                g = h // G
                k = K[b, tk, g]
                mag[:, b, h] = sc * (np.abs(f64(Q)[:, b, h]) @ np.abs(k).T).max(-1)
                p = np.exp(sc * f64(Q)[:, b, h] @ k.T - want_lse[:, b, h, None])
                floor[:, b, h] = 2.0 ** -31 * (p * np.abs(vs[b, tk // cache.block, g])).max(-1)[:, None] * np.abs(codes[b, tk, g]).sum(0)
    check(O, lse, wantO, want_lse, A, dtype, 2.0 ** -11 + 2.0 ** -20 if dtype == "bf16" else 2.0 ** -21, mag, max(counts), cache.d, floor)


def foreign(cache, seed, kind):
    """Scales as programs make them: max / 448 of a block, one for a whole head, zeros among them."""
    g = np.random.default_rng(seed)
    for s in (cache.k_scale, cache.v_scale):
        x = np.exp2(g.uniform(-9, -3, tuple(s.shape)))
        if kind == "steps":                             # just above and just below powers of two
            x = np.exp2(np.round(np.log2(x))) * g.choice([1 + 2.0 ** -23, 1 - 2.0 ** -24, 1.0], x.shape)
        if kind == "zeros":
            x *= g.choice([1.0, 1.0, 0.0], x.shape)
        s.copy_(dev(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["any", "steps", "zeros"])
@pytest.mark.parametrize("B,n,L,Hq,Hkv,d,block", [(3, 77, 1, 32, 8, 128, 64), (1, 2000, 5, 8, 2, 128, 16), (2, 300, 2, 6, 3, 64, 32),
                                                  (90, 130, 1, 8, 4, 64, 128)])
def test_kv8_attn_takes_any_scale(dtype, kind, B, n, L, Hq, Hkv, d, block):
    cache = cache_of(B, n, Hkv, d, block, n)
    foreign(cache, B, kind)
    g = np.random.default_rng(n)
    counts = g.integers(1, n + 1, B)
    counts[0] = n
    Q, O, lse, ws = run8(cache, L, B, Hq, dtype, counts)
    check_scaled(cache, Q, O, lse, counts, None, dtype)
    k = min(n, 60)
    idx = np.stack([np.sort(g.permutation(n)[:k]) for _ in range(B)])
    counts = np.full(B, k)
    Q, O, lse, ws = run8(cache, L, B, Hq, dtype, counts, idx)
    check_scaled(cache, Q, O, lse, counts, idx, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kv8_write_behind_rows_of_another_programs_scale(dtype):
    """A block that holds earlier rows keeps its scale, whatever it is, or takes a larger one."""
    B, n, H, d, block, T = 3, 200, 3, 64, 32, 40
    g = np.random.default_rng(2)
    cache = cache_of(B, n, H, d, block, 4)
    foreign(cache, 7, "any")
    for i, start in enumerate(([5, 40, 159], [6, 33, 100], [46, 90, 31])):
        k0, v0, ks0, vs0 = host(cache)
        K, V = rows(g, B, T, H, d, dtype), rows(g, B, T, H, d, dtype)
        clsa.kv8_write(cache, K, V, dev(np.array(start), torch.int32))
        k1, v1, ks1, vs1 = host(cache)
        for codes, scales, X, c1, s1 in ((k0, ks0, K, k1, ks1), (v0, vs0, V, v1, vs1)):
            want, wsc = C.kv8_write(codes, scales, f64(X), start, None, block)
            np.testing.assert_array_equal(s1, wsc)
            np.testing.assert_array_equal(c1, want)


def test_powers_of_two_count_exactly():
    """Every scale from 2^-126 to 2^119, a token a sequence and query 0: the output is code * scale, to the bit in
    fp32, rounded once in bf16; and two tokens whose scales lie 2^k apart."""
    e = np.arange(-126, 120)
    B, d = len(e), 64
    cache = cache_of(B, 32, 1, d, 16, 6)
    cache.v_scale.copy_(dev(np.stack([2.0 ** e.clip(-126, 119), 2.0 ** e[::-1]], 1)[..., None]))
    cache.k_scale.fill_(1.0)
    codes = dev(C.e4m3_decode(host(cache)[1]))
    idx = dev(np.tile([3], (B, 1)), torch.int32)
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    for dtype in ("bf16", "f32"):
        O, lse = clsa.kv8_attn(torch.zeros(1, B, 4, d, dtype=DT[dtype], device="cuda"), cache, one, idx=idx)
        want = (codes[:, 3, 0] * cache.v_scale[:, 0]).to(DT[dtype])[:, None].expand(B, 4, d)
        ok = want.float().abs() >= 2.0 ** -126           # below it, a sum may flush to 0
        assert torch.equal(O[0][ok], want[ok]) and not lse.any()
        O, lse = clsa.kv8_attn(torch.zeros(1, B, 4, d, dtype=DT[dtype], device="cuda"), cache, 2 * one, idx=dev(np.tile([3, 20], (B, 1)), torch.int32))
        want = (codes[:, 3, 0].double() * cache.v_scale[:, 0].double() + codes[:, 20, 0].double() * cache.v_scale[:, 1].double())[:, None] / 2
        mag = (codes[:, 3, 0].double().abs() * cache.v_scale[:, 0].double() + codes[:, 20, 0].double().abs() * cache.v_scale[:, 1].double())[:, None] / 2
        # a weight below 2^-24 of half range is lost, 2^-32 of the larger one's; the result's rounding
        assert ((O[0].double() - want).abs() <= mag * 2.0 ** -22 + 448 * 2.0 ** -32 * cache.v_scale.double().amax(1)[:, None]
                + want.abs() * torch.finfo(DT[dtype]).eps / 2 + 2.0 ** -126).all()
