"""GPU parity of the cache operators against their float64 references: rotary positions and
the 8-bit K/V cache's write and read.

Tolerances.  A result stored in a type t is off by at most finfo(t).eps / 2 of its value.
rope adds fp32 work: the reduced angle's rounding (2^-25 half turns, 2^-23.3 rad), sincospif
(1 ulp, 2^-24), the factor mscale, two products and a sum (2^-24 of each term): under 2^-21
of m (|x1| + |x2|).  Codes and scales of the 8-bit cache are exact: every operation before
the rounding to e4m3 is a product with a power of two."""
import numpy as np
import pytest
import torch

from long_context_sparse_clsa_b200 import clsa
from oracle import cache_oracle as C

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_clsa_b200.build import build
    build()
    clsa.load_library()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


# ----------------------------------------------------------------------------- rope

def check_rope(got, x, pos, freqs, layout, m, inverse):
    want = C.rope(f64(x), pos, freqs, layout, m, inverse)
    rot = 2 * len(freqs)
    mag = np.abs(f64(x))
    pair = np.zeros_like(mag)
    h = rot // 2
    if layout == "half":
        s = mag[..., :h] + mag[..., h:rot]
        pair[..., :h], pair[..., h:rot] = s, s
    else:
        s = mag[..., 0:rot:2] + mag[..., 1:rot:2]
        pair[..., 0:rot:2], pair[..., 1:rot:2] = s, s
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 2.0 ** -21 * m * pair + 1e-38
    assert (np.abs(f64(got) - want) <= tol).all()
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("N,Hq,Hk,d,rot", [(1, 32, 8, 128, 128), (3, 1, 1, 64, 16), (77, 6, 3, 128, 96), (500, 8, 2, 64, 64),
                                           (2003, 1, 1, 128, 48)])
def test_rope(dtype, layout, N, Hq, Hk, d, rot):
    g = np.random.default_rng(N + rot)
    pos = g.integers(-5000, 1 << 20, N).astype(np.int32)
    pos[0] = 0 if N < 3 else pos[0]
    q, k = dev(g.standard_normal((N, Hq, d)), DT[dtype]), dev(g.standard_normal((N, Hk, d)), DT[dtype])
    tp = dev(pos, torch.int32)
    for kw in ({}, {"scaling": "linear", "factor": 3.0}, {"scaling": "base", "factor": 5.0},
               {"scaling": "by_parts", "factor": 4.0, "orig_len": 4096, "beta_fast": 30.0, "beta_slow": 2.0}):
        f = C.rope_freqs(rot, 500000.0, **kw)
        for inverse in (False, True):
            qo, ko = clsa.rope(q, k, tp, rot=rot, layout=layout, theta=500000.0, mscale=1.19, inverse=inverse, **kw)
            check_rope(qo, q, pos, f, layout, 1.19, inverse)
            check_rope(ko, k, pos, f, layout, 1.19, inverse)
    assert clsa.last_launch_count() == 1


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_in_place_one_side_and_layers(layout):
    """In place; q or k alone; Q [L][B][Hq][d] with one position per sequence."""
    g = np.random.default_rng(5)
    pos = dev(np.array([3, 99999, 41]), torch.int32)
    Q = dev(g.standard_normal((4, 3, 8, 128)), torch.bfloat16)
    k = dev(g.standard_normal((3, 2, 128)), torch.bfloat16)
    qo, ko = clsa.rope(Q, k, pos, layout=layout)
    for l in range(4):
        one, none = clsa.rope(Q[l].contiguous(), None, pos, layout=layout)
        assert none is None and torch.equal(one, qo[l])
    none, konly = clsa.rope(None, k, pos, layout=layout)
    assert none is None and torch.equal(konly, ko)
    Q2, k2 = Q.clone(), k.clone()
    clsa.rope(Q2, k2, pos, layout=layout, q_out=Q2, k_out=k2)
    assert torch.equal(Q2, qo) and torch.equal(k2, ko)


def test_rope_gradient_matches_differences():
    g = np.random.default_rng(6)
    x, w = g.standard_normal((2, 1, 64)), g.standard_normal((2, 1, 64))
    pos = dev(np.array([17, 4000]), torch.int32)
    kw = dict(rot=48, layout="interleaved", theta=10000.0, mscale=1.3)
    grad = f64(clsa.rope(dev(w), None, pos, inverse=True, **kw)[0])
    for i in (0, 1, 20, 47, 48, 63):
        e = np.zeros_like(x)
        e[..., i] = 0.5  # the map is linear: differences are exact up to rounding
        d = (f64(clsa.rope(dev(x + e), None, pos, **kw)[0]) - f64(clsa.rope(dev(x - e), None, pos, **kw)[0])) * w
        # each of 128 terms of the two sums is off by a few 2^-21 of its pair's size
        assert np.abs(d.sum((1, 2)) - grad[:, 0, i]).max() <= 2.0 ** -21 * 2 * 64 * 8


# ------------------------------------------------------------------------- write, read

def rows(g, B, T, H, d, dtype, spread=3.0):
    x = g.standard_normal((B, T, H, d)) * np.exp2(g.uniform(-spread, spread, (B, T, H, 1)))
    return dev(x, DT[dtype])


def cache_of(B, n, H, d, block, seed):
    """A cache of arbitrary bytes (no NaN codes) and power-of-two scales."""
    g = np.random.default_rng(seed)
    codes = [g.integers(0, 127, (B, n, H, d)) + 128 * g.integers(0, 2, (B, n, H, d)) for _ in range(2)]
    scales = [2.0 ** g.integers(-9, -3, (B, -(-n // block), H)) for _ in range(2)]
    dv = [dev(c, torch.uint8).view(torch.float8_e4m3fn) for c in codes]
    return clsa.Kv8Cache(*dv, *[dev(s) for s in scales], block)


def host(c):
    return (c.K8.view(torch.uint8).cpu().numpy(), c.V8.view(torch.uint8).cpu().numpy(),
            c.k_scale.cpu().numpy().astype(np.float64), c.v_scale.cpu().numpy().astype(np.float64))


def check_write(cache, K, V, start, count, **kw):
    k0, v0, ks0, vs0 = host(cache)
    ws = clsa.Workspace(256)
    clsa.kv8_write(cache, K, V, dev(start, torch.int32), None if count is None else dev(count, torch.int32), ws=ws)
    k1, v1, ks1, vs1 = host(cache)
    for codes, scales, X, c1, s1 in ((k0, ks0, K, k1, ks1), (v0, vs0, V, v1, vs1)):
        wc, wsc = C.kv8_write(codes, scales, f64(X), start, count, cache.block)
        np.testing.assert_array_equal(s1, wsc)
        np.testing.assert_array_equal(c1, wc)
    return ws


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("B,T,n,H,d", [(3, 1, 200, 2, 128), (2, 130, 300, 3, 64), (1, 300, 331, 1, 128), (5, 17, 64, 8, 64)])
def test_kv8_write_matches_the_reference(dtype, block, B, T, n, H, d):
    g = np.random.default_rng(block + T)
    cache = cache_of(B, n, H, d, block, 7)
    start = g.integers(0, n - T + 1, B)
    start[0] = n - T                              # up to the last token
    count = g.integers(0, T + 1, B)
    count[0] = T
    ws = check_write(cache, rows(g, B, T, H, d, dtype), rows(g, B, T, H, d, dtype), start, count)
    assert ws.status()[0] == "CLSA_OK" and clsa.last_launch_count() == 1
    check_write(cache, rows(g, B, T, H, d, dtype), rows(g, B, T, H, d, dtype), np.maximum(start - 1, 0), None)


@pytest.mark.parametrize("block", [16, 128])
def test_kv8_append_token_by_token(block):
    """A decode loop: blocks that grow their scale, blocks that begin anew, tokens behind left alone."""
    g = np.random.default_rng(11)
    cache = cache_of(2, 150, 2, 64, block, 3)
    for t in range(block - 3, block + 5):
        check_write(cache, rows(g, 2, 1, 2, 64, "bf16", 8.0), rows(g, 2, 1, 2, 64, "bf16", 8.0), np.array([t, t % 7]), None)


def test_kv8_write_special_values():
    """Zeros, infinities, NaN, subnormal and the largest numbers."""
    X = np.zeros((1, 64, 1, 64), np.float32)
    X[0, 1, 0, :4] = [np.inf, -np.inf, np.nan, 3.0]
    X[0, 16, 0, :] = 0.0                                     # a block of zeros
    X[0, 33, 0, :3] = [1e-38, -1e-45, 1e-40]                 # below the smallest scale
    X[0, 50, 0, :3] = [3.4e38, -3.3e38, 1.0]                 # above the largest
    K = dev(X)
    cache = cache_of(1, 64, 1, 64, 16, 1)
    check_write(cache, K, K, np.array([0]), None)
    k, _ = clsa.kv8_read(cache, T=64, dtype=torch.float32)
    assert torch.isnan(k[0, 1, 0, 2]) and int(torch.isnan(k).sum()) == 1
    assert (k[0, 1, 0, :2].abs() >= 3.0).all() and torch.isfinite(k[0, 50]).all()


def test_kv8_write_refuses_rows_outside_and_reports():
    g = np.random.default_rng(2)
    cache = cache_of(4, 40, 2, 64, 16, 9)
    ws = check_write(cache, rows(g, 4, 8, 2, 64, "bf16"), rows(g, 4, 8, 2, 64, "bf16"),
                     np.array([3, 33, -1, 32]), np.array([8, 8, 8, 8]))
    code, detail = ws.status()
    assert code == "CLSA_ERR_BAD_INDEX" and detail >> 32 in (1, 2)
    assert ws.status()[0] == "CLSA_OK"
    ws = check_write(cache, rows(g, 4, 8, 2, 64, "bf16"), rows(g, 4, 8, 2, 64, "bf16"),
                     np.array([33, 33, 33, -5]), np.array([7, 0, -3, 0]))
    assert ws.status()[0] == "CLSA_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,n,H,d,block", [(1, 1, 1, 1, 64, 16), (3, 37, 90, 3, 128, 32), (2, 250, 260, 8, 64, 128)])
def test_kv8_read(dtype, B, T, n, H, d, block):
    """A range and an index list: code * scale, exact in bf16 too (4 significant bits)."""
    g = np.random.default_rng(T)
    cache = cache_of(B, n, H, d, block, 21)
    kc, vc, ks, vs = host(cache)
    kv = [C.kv8_values(kc, ks, block), C.kv8_values(vc, vs, block)]
    start, count = g.integers(0, n - T + 1, B), g.integers(0, T + 1, B)
    idx = np.stack([g.permutation(n)[:T] for _ in range(B)])
    idx[0, 0] = idx[0, -1]                                    # the same token twice
    for use_idx in (False, True):
        tok = idx if use_idx else start[:, None] + np.arange(T)
        for cnt in (None, count):
            mark = torch.full((B, T, H, d), 7.0, device="cuda", dtype=DT[dtype])
            out = [mark.clone(), mark.clone()]
            clsa.kv8_read(cache, *out, start=None if use_idx else dev(start, torch.int32),
                          idx=dev(idx, torch.int32) if use_idx else None,
                          count=None if cnt is None else dev(cnt, torch.int32))
            for o, want in zip(out, kv):
                w = np.stack([want[b, tok[b]] for b in range(B)])
                if cnt is not None:
                    w[np.arange(T)[None] >= cnt[:, None]] = 7.0
                np.testing.assert_array_equal(f64(o), w)


def test_kv8_read_reports_tokens_outside():
    cache = cache_of(2, 30, 2, 64, 16, 4)
    idx = np.array([[0, 30, 5, -1], [29, 1, 2, 3]])
    ws = clsa.Workspace(256)
    K, V = clsa.kv8_read(cache, idx=dev(idx, torch.int32), ws=ws)
    code, detail = ws.status()
    assert code == "CLSA_ERR_BAD_INDEX" and detail in (1, 3)
    assert not K[0, 1].any() and not V[0, 3].any()
    K2, _ = clsa.kv8_read(cache, start=dev(np.array([28, 0]), torch.int32), T=4, ws=ws)
    code, detail = ws.status()
    assert code == "CLSA_ERR_BAD_INDEX" and detail in (2, 3)
    assert not K2[0, 2:].any() and K2[1].any()


def test_write_then_read_in_a_captured_graph():
    """One capture: rope, write, read; replays follow the inputs' new values."""
    g = np.random.default_rng(8)
    B, T, H, d = 2, 5, 2, 64
    K, V = rows(g, B, T, H, d, "bf16"), rows(g, B, T, H, d, "bf16")
    pos = dev(np.arange(T), torch.int32)
    start = dev(np.array([0, 6]), torch.int32)
    cache = clsa.Kv8Cache.empty(B, 32, H, d, 16)
    ws = clsa.Workspace(256)
    Kr, Ko, Vo = torch.empty_like(K), torch.zeros_like(K), torch.zeros_like(K)

    def step():
        clsa.rope(None, K, pos, k_out=Kr)
        clsa.kv8_write(cache, Kr, V, start, ws=ws)
        clsa.kv8_read(cache, Ko, Vo, start=start, ws=ws)
    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for r in range(2):
        K.copy_(rows(np.random.default_rng(30 + r), B, T, H, d, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        a, b = Ko.clone(), Vo.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(a, Ko) and torch.equal(b, Vo)
        rel = (Ko.float() - Kr.float()).norm() / Kr.float().norm()
        assert rel <= 2.0 ** -4
