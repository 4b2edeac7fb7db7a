"""GPU parity of attention over the 8-bit cache and of window attention against their float64
references.

Tolerance of an output row, with A = sum_j p_j |v_j| / sum_j p_j and u = 2^-24:
  * the result's rounding, finfo(dtype).eps / 2 of the value;
  * the rounding of the probabilities that enter the second product, finfo(half).eps / 2 = 2^-11
    (bf16: 2^-8; fp32 rows: two halves, 2^-22, or three bf16 parts, 2^-23) of A;
  * scores: sums of d products in the tensor core, which may cut off rather than round,
    2 (d + 4) u of scale sum |q k|, relative in p and in the sum of p: twice that of A;
  * sums over n tokens: 2 (n + 16) u of A; exponentials: 2 ulp, under 2^-21 of A;
  * 8-bit cache: a half below 2^-14 is off by up to 2^-25 instead of relatively; the weight of
    token j is p_j s_j / S (s_j its value scale), S such that the largest weight is at least 2^7.  So sum_j
    |code_j| 2^-25 S <= 2^-32 max_j (p_j s_j) sum_j |code_j| more, over the sum of p.
The log-sum-exp is off by the score's error, the sum's and 2^-21 + 2^-22 |lse|."""
import numpy as np
import pytest
import torch

from long_context_sparse_clsa_b200 import clsa
from oracle import cache_oracle as C
from test_gpu_cache import DT, cache_of, dev, f64, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_clsa_b200.build import build
    build()
    clsa.load_library()


def check(O, lse, wantO, want_lse, A, dtype, p_eps, score_mag, n, d, floor=0.0):
    """score_mag: per row, the largest scale * sum |q k|."""
    eps = torch.finfo(DT[dtype]).eps / 2
    ds = 2 * (d + 4) * U * score_mag
    tol = eps * np.abs(wantO) + (p_eps + 2 * ds[..., None] + 2 * (n + 16) * U + 2.0 ** -21) * A + floor + 1e-30
    err = np.abs(f64(O) - wantO)
    assert np.isfinite(f64(O)).all()
    assert (err <= tol).all(), float((err / tol).max())
    got = lse.cpu().numpy().astype(np.float64)
    none = np.isneginf(want_lse)
    assert np.isneginf(got[none]).all()
    ltol = ds + 2 * (n + 16) * U + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(none, 0, want_lse))
    lerr = np.abs(np.where(none, 0, got - np.where(none, 0, want_lse)))
    assert (lerr <= ltol).all(), float((lerr / ltol).max())


# ----------------------------------------------------------------------- 8-bit cache

def run8(cache, L, B, Hq, dtype, counts, idx=None, scale=0.0, seed=0, qmag=1.0):
    g = np.random.default_rng(seed)
    Q = dev(g.standard_normal((L, B, Hq, cache.d)) * qmag, DT[dtype])
    need = clsa.kv8_attn_workspace_size(Q, cache, None if idx is None else dev(idx, torch.int32))
    ws = clsa.Workspace(need)
    cnt = dev(np.asarray(counts), torch.int32)
    O, lse = clsa.kv8_attn(Q, cache, cnt, idx=None if idx is None else dev(idx, torch.int32), scale=scale, ws=ws)
    assert clsa.last_launch_count() == 1
    torch.cuda.synchronize()
    return Q, O, lse, ws


def check8(cache, Q, O, lse, counts, idx, dtype, scale=0.0):
    kc, vc, ks, vs = host(cache)
    K, V = C.kv8_values(kc, ks, cache.block), C.kv8_values(vc, vs, cache.block)
    lim = [min(max(int(c), 0), cache.n_max if idx is None else idx.shape[1]) for c in counts]
    toks = [np.arange(m) if idx is None else idx[b, :m] for b, m in enumerate(lim)]
    wantO, want_lse = C.attention(f64(Q), K, V, toks, scale)
    A, _ = C.attention(f64(Q), K, np.abs(V), toks, scale)
    sc = scale if scale > 0 else cache.d ** -0.5
    mag, floor = np.zeros(want_lse.shape), np.zeros(wantO.shape)
    G = Q.shape[2] // cache.Hkv
    for b, tk in enumerate(toks):
        for h in range(Q.shape[2]):
            if len(tk):
                c, g = b % cache.B, h // G
                mag[:, b, h] = sc * (np.abs(f64(Q)[:, b, h]) @ np.abs(K[c][tk, g]).T).max(-1)
                p = np.exp(sc * f64(Q)[:, b, h] @ K[c][tk, g].T - want_lse[:, b, h, None])  # over their sum
                vsc = vs[c, tk // cache.block, g]
                floor[:, b, h] = 2.0 ** -32 * (p * vsc).max(-1)[:, None] * np.abs(V[c][tk, g] / vsc[:, None]).sum(0)
    check(O, lse, wantO, want_lse, A, dtype, 2.0 ** -11 if dtype == "bf16" else 2.0 ** -21, mag, max(lim + [1]), cache.d, floor)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,L,Hq,Hkv,d,block", [
    (1, 1, 1, 8, 2, 128, 16), (3, 77, 1, 32, 8, 128, 64), (2, 300, 2, 6, 3, 64, 32), (4, 1025, 1, 16, 1, 64, 128),
    (1, 2000, 24, 32, 8, 128, 64), (9, 50, 1, 8, 8, 128, 16), (1, 700, 3, 33, 1, 64, 16), (2, 5000, 1, 4, 1, 128, 128)])
def test_kv8_attn_dense(dtype, B, n, L, Hq, Hkv, d, block):
    cache = cache_of(B, n, Hkv, d, block, n)
    counts = np.random.default_rng(n).integers(0, n + 1, B)
    counts[0] = n
    if B > 1:
        counts[1] = 0
    if B > 3:
        counts[3] = 1
    Q, O, lse, ws = run8(cache, L, B, Hq, dtype, counts)
    check8(cache, Q, O, lse, counts, None, dtype)
    assert ws.status()[0] == "CLSA_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,k,L,Hq,Hkv,d,block", [(1, 3000, 512, 24, 32, 8, 128, 64), (5, 200, 40, 2, 6, 3, 64, 16),
                                                    (2, 90, 90, 1, 8, 2, 128, 128), (3, 400, 1, 1, 8, 1, 64, 32)])
def test_kv8_attn_selected(dtype, B, n, k, L, Hq, Hkv, d, block):
    g = np.random.default_rng(k)
    cache = cache_of(B, n, Hkv, d, block, k)
    idx = np.stack([np.sort(g.permutation(n)[:k]) for _ in range(B)])
    counts = g.integers(0, k + 1, B)
    counts[0] = k
    for b in range(B):
        idx[b, counts[b]:] = -1          # as clsa_topk pads
    if k > 3:
        idx[0, 1] = idx[0, 0]            # the same token twice: it counts twice
    Q, O, lse, ws = run8(cache, L, B, Hq, dtype, counts, idx, scale=0.21)
    check8(cache, Q, O, lse, counts, idx, dtype, 0.21)
    assert ws.status()[0] == "CLSA_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kv8_attn_one_cache_for_all_rows(dtype):
    """Rows of a prefill chunk: one cache, each row its own length or selection."""
    cache = cache_of(1, 150, 2, 128, 32, 5)
    counts = np.arange(100, 140)
    Q, O, lse, _ = run8(cache, 2, 40, 8, dtype, counts)
    check8(cache, Q, O, lse, counts, None, dtype)
    idx = np.stack([np.sort(np.random.default_rng(t).permutation(100 + t)[:30]) for t in range(40)])
    counts = np.full(40, 30)
    Q, O, lse, _ = run8(cache, 2, 40, 8, dtype, counts, idx)
    check8(cache, Q, O, lse, counts, idx, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_kv8_attn_scales_far_apart(dtype):
    """Key and value blocks whose scales differ by 2^40: no block is lost beside a larger one."""
    B, n, H, d, block = 2, 600, 2, 64, 16
    cache = cache_of(B, n, H, d, block, 77)
    g = np.random.default_rng(1)
    nb = cache.k_scale.shape[1]
    cache.v_scale.copy_(dev(2.0 ** g.integers(-30, 11, (B, nb, H))))
    cache.k_scale.copy_(dev(2.0 ** g.integers(-40, -7, (B, nb, H))))
    cache.v_scale[:, 0] = 2.0 ** -100
    counts = np.array([600, 16])
    Q, O, lse, _ = run8(cache, 1, B, 4, dtype, counts, qmag=30.0)
    check8(cache, Q, O, lse, counts, None, dtype)


@pytest.mark.parametrize("qmag", [1e-30, 1e-3, 300.0, 1e20])
def test_kv8_attn_query_range(qmag):
    """Queries far outside the half range (their scores scaled back by `scale`)."""
    cache = cache_of(2, 200, 2, 128, 64, 3)
    counts = np.array([200, 33])
    scale = float(np.float32(0.1 / qmag))
    for dtype in ("bf16", "f32"):
        Q, O, lse, _ = run8(cache, 1, 2, 8, dtype, counts, scale=scale, qmag=qmag)
        check8(cache, Q, O, lse, counts, None, dtype, scale)


def test_kv8_attn_leaves_unseen_bytes_out():
    """NaN codes and scales behind the length and outside the selection change nothing; a NaN that is
    seen reaches its rows and no others."""
    cache = cache_of(2, 300, 2, 128, 64, 8)
    counts = np.array([100, 250])
    Q, O, lse, _ = run8(cache, 1, 2, 8, "bf16", counts)
    idx = np.stack([np.arange(0, 100, 2), np.arange(0, 100, 2)])
    Qs, Os, ls, _ = run8(cache, 1, 2, 8, "bf16", [50, 50], idx)
    k, v = cache.K8.view(torch.uint8), cache.V8.view(torch.uint8)
    k[0, 100:] = 127
    v[0, 100:] = 127
    cache.k_scale[0, 2:] = float("nan")
    cache.v_scale[0, 2:] = float("inf")
    Q2, O2, lse2, _ = run8(cache, 1, 2, 8, "bf16", counts)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    k[0, 1:100:2] = 127
    v[0, 1:100:2] = 127
    Q3, O3, l3, _ = run8(cache, 1, 2, 8, "bf16", [50, 50], idx)
    assert torch.equal(Os, O3) and torch.equal(ls, l3)
    v[0, 4, 1, 5] = 127
    _, O4, _, _ = run8(cache, 1, 2, 8, "bf16", [50, 50], idx)
    nan = torch.isnan(O4)
    assert nan[0, 0, 4:, 5].all() and int(nan.sum()) == 4
    k[1, 4, 0, 5] = 127
    _, O5, l5, _ = run8(cache, 1, 2, 8, "bf16", [50, 50], idx)
    assert torch.isnan(O5[0, 1, :4]).all() and torch.isnan(l5[0, 1, :4]).all() and not torch.isnan(O5[0, 1, 4:]).any()


def test_kv8_attn_reports_tokens_outside_and_leaves_them_out():
    cache = cache_of(1, 64, 1, 64, 16, 2)
    idx = np.array([[3, 64, 9, -2, 11]])
    Q, O, lse, ws = run8(cache, 1, 1, 4, "bf16", [5], idx)
    code, detail = ws.status()
    assert code == "CLSA_ERR_BAD_INDEX" and detail in (1, 3)
    check8(cache, Q, O, lse, [3], idx[:, [0, 2, 4]], "bf16")


def test_kv8_attn_repeats_itself_and_shares_a_clean_workspace():
    """Same bits every time; one workspace serves sizes in turn once zeroed, and the same size again and
    again; two streams with a workspace each; a captured graph."""
    cache = cache_of(3, 4000, 2, 128, 64, 4)
    g = np.random.default_rng(0)
    Q = dev(g.standard_normal((1, 3, 8, 128)), torch.bfloat16)
    cnt = dev(np.array([4000, 17, 2500]), torch.int32)
    need = clsa.kv8_attn_workspace_size(Q, cache)
    ws, ws2 = clsa.Workspace(need), clsa.Workspace(need)
    O, lse = clsa.kv8_attn(Q, cache, cnt, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(Q) for _ in range(12)]
    for i, o in enumerate(outs):
        if i % 2:
            with torch.cuda.stream(side):
                clsa.kv8_attn(Q, cache, cnt, ws=ws2, O=o)
        else:
            clsa.kv8_attn(Q, cache, cnt, ws=ws, O=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, O) for o in outs)
    graph = torch.cuda.CUDAGraph()
    o2, l2 = torch.empty_like(Q), torch.empty_like(lse)
    with torch.cuda.graph(graph):
        clsa.kv8_attn(Q, cache, cnt, ws=ws, O=o2, lse=l2)
    for c in ([4000, 17, 2500], [1, 0, 4000], [64, 4000, 3]):
        cnt.copy_(torch.tensor(c, dtype=torch.int32))
        graph.replay()
        want, wl = clsa.kv8_attn(Q, cache, cnt, ws=ws2)
        torch.cuda.synchronize()
        assert torch.equal(o2, want) and torch.equal(l2, wl)
    O1, none = clsa.kv8_attn(Q[0], cache, cnt, want_lse=False)
    assert none is None and torch.equal(O1, o2[0])


# --------------------------------------------------------------------------- window

def run_window(B, T, n, Hq, Hkv, d, dtype, lens, window, sinks, seed=0, scale=0.0):
    g = np.random.default_rng(seed)
    Q = dev(g.standard_normal((B, T, Hq, d)), DT[dtype])
    K, V = (dev(g.standard_normal((B, n, Hkv, d)), DT[dtype]) for _ in range(2))
    ws = clsa.Workspace(clsa.window_attn_workspace_size(Q, K, window, sinks))
    O, lse = clsa.window_attn(Q, K, V, dev(np.asarray(lens), torch.int32), window, sinks, scale=scale, ws=ws)
    assert clsa.last_launch_count() == 1
    torch.cuda.synchronize()
    assert ws.status()[0] == "CLSA_OK"
    return Q, K, V, O, lse


def window_reference(Q, K, V, lens, window, sinks, scale):
    """As the oracle's, over arrays: (O, lse, A, largest scale sum |q k|)."""
    B, T, Hq, d = Q.shape
    G = Hq // K.shape[2]
    O, A = np.zeros(Q.shape), np.zeros(Q.shape)
    lse, mag = np.full(Q.shape[:3], -np.inf), np.zeros(Q.shape[:3])
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        see = np.stack([C.window_sees(n, n - T + t, window, sinks) for t in range(T)])
        any_ = see.any(1)
        for h in range(Hq):
            k, v, q = K[b, :n, h // G], V[b, :n, h // G], Q[b, :, h]
            s = np.where(see, q @ k.T * scale, -np.inf)
            m = np.where(any_, s.max(1), 0.0)
            p = np.exp(s - m[:, None])
            l = np.where(any_, p.sum(1), 1.0)
            O[b, :, h], A[b, :, h] = (p @ v) / l[:, None], (p @ np.abs(v)) / l[:, None]
            lse[b, :, h] = np.where(any_, m + np.log(l), -np.inf)
            mag[b, :, h] = np.where(see, np.abs(q) @ np.abs(k).T * scale, 0).max(1)
    return O, lse, A, mag


def check_window(Q, K, V, O, lse, lens, window, sinks, dtype, scale=0.0):
    d, n = Q.shape[-1], K.shape[1]
    scale = scale if scale > 0 else d ** -0.5
    wO, wl, A, mag = window_reference(f64(Q), f64(K), f64(V), np.clip(lens, 0, n), window, sinks, scale)
    check(O, lse, wO, wl, A, dtype, 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23, mag, min(n, window + sinks + 128), d)


def test_window_reference_is_the_oracle():
    g = np.random.default_rng(3)
    Q, K, V = g.standard_normal((2, 5, 4, 16)), g.standard_normal((2, 20, 2, 16)), g.standard_normal((2, 20, 2, 16))
    a = C.window_attention(Q, K, V, [3, 17], 4, 2)
    b = window_reference(Q, K, V, [3, 17], 4, 2, 0.25)
    np.testing.assert_allclose(a[0], b[0], atol=1e-12)
    np.testing.assert_allclose(a[1], b[1], atol=1e-12)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (7, 4), (64, 0), (129, 5), (100000, 3)])
@pytest.mark.parametrize("B,T,n,Hq,Hkv,d", [(4, 1, 300, 8, 2, 128), (3, 5, 200, 6, 3, 64), (1, 130, 410, 8, 2, 128),
                                            (2, 67, 150, 16, 1, 64)])
def test_window_attn(dtype, window, sinks, B, T, n, Hq, Hkv, d):
    lens = np.random.default_rng(T).integers(0, n + 1, B)
    lens[0] = n
    if B > 1:
        lens[1] = T // 2                     # padded rows in front (T = 1: an empty sequence)
    if B > 2:
        lens[2] = min(n, T + sinks)
    out = run_window(B, T, n, Hq, Hkv, d, dtype, lens, window, sinks)
    check_window(*out, lens, window, sinks, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,n,Hq,Hkv,d,window,sinks", [(1, 1, 9000, 8, 2, 128, 8000, 16), (1, 1000, 1000, 4, 1, 128, 333, 20),
                                                         (1, 515, 2100, 40, 8, 64, 1024, 1), (2, 300, 700, 12, 1, 128, 200, 130),
                                                         (1, 260, 300, 128, 1, 64, 50, 3), (1, 200, 333, 7, 7, 128, 90, 64)])
def test_window_attn_longer(dtype, B, T, n, Hq, Hkv, d, window, sinks):
    lens = np.array([n, n // 2 + 1][:B])
    out = run_window(B, T, n, Hq, Hkv, d, dtype, lens, window, sinks, scale=0.3)
    check_window(*out, lens, window, sinks, dtype, 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 6, 200])
def test_window_attn_leaves_unseen_tokens_out(dtype, T):
    """NaN behind the length, and between the sinks and every row's window, changes nothing; infinities
    and the type's lowest value in K there neither."""
    n, Hq, Hkv, d, window, sinks = 700, 8, 2, 128, 90, 5
    lens = np.array([650, 333])
    g = np.random.default_rng(1)
    Q = dev(g.standard_normal((2, T, Hq, d)), DT[dtype])
    K, V = (dev(g.standard_normal((2, n, Hkv, d)), DT[dtype]) for _ in range(2))
    L = dev(lens, torch.int32)
    O, lse = clsa.window_attn(Q, K, V, L, window, sinks)
    for b, m in enumerate(lens):
        V[b, m:] = float("nan")
        K[b, m:] = float("inf")
        far = m - T - window + 1
        if far > sinks:
            V[b, sinks:far] = float("nan")
            K[b, sinks:far] = torch.finfo(DT[dtype]).min
            K[b, sinks + 1] = float("nan")
    O2, lse2 = clsa.window_attn(Q, K, V, L, window, sinks)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)


def test_window_attn_graph_and_repeats():
    g = np.random.default_rng(2)
    for T in (1, 140):
        Q = dev(g.standard_normal((2, T, 8, 128)), torch.bfloat16)
        K, V = (dev(g.standard_normal((2, 900, 2, 128)), torch.bfloat16) for _ in range(2))
        L = dev(np.array([900, 500]), torch.int32)
        ws = clsa.Workspace(clsa.window_attn_workspace_size(Q, K, 256, 4))
        O, lse = clsa.window_attn(Q, K, V, L, 256, 4, ws=ws)
        graph = torch.cuda.CUDAGraph()
        o2 = torch.empty_like(O)
        with torch.cuda.graph(graph):
            clsa.window_attn(Q, K, V, L, 256, 4, ws=ws, O=o2, want_lse=False)
        for lens in ([900, 500], [141, 0], [2, 899]):
            L.copy_(torch.tensor(lens, dtype=torch.int32))
            graph.replay()
            want, _ = clsa.window_attn(Q, K, V, L, 256, 4)
            torch.cuda.synchronize()
            assert torch.equal(o2, want)


# ------------------------------------------------------------------- used together

def test_serving_step_over_the_8bit_cache():
    """A decode step as a program runs it: positions onto queries and keys, the new row into the cache,
    index scores, the shared selection, attention over it; against the same path over the values
    read back, through the library's bf16 calls and through the reference."""
    g = np.random.default_rng(0)
    B, n, Hq, Hkv, d, L, k, block = 2, 1500, 8, 2, 128, 3, 256, 64
    lens = np.array([1200, 777])
    cache = clsa.Kv8Cache.empty(B, n, Hkv, d, block)
    Kp, Vp = (dev(g.standard_normal((B, 1199, Hkv, d)), torch.bfloat16) for _ in range(2))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    clsa.kv8_write(cache, Kp, Vp, zero, dev(lens - 1, torch.int32))
    k_idx = dev(g.standard_normal((B, n, 128)), torch.bfloat16)
    q_idx = dev(g.standard_normal((B, 128)), torch.bfloat16)
    seq = dev(lens, torch.int32)
    Q, Kn, Vn = (dev(g.standard_normal(s), torch.bfloat16) for s in ((L, B, Hq, d), (B, 1, Hkv, d), (B, 1, Hkv, d)))
    pos = dev(lens - 1, torch.int32)
    Qr, Kr = clsa.rope(Q, Kn, pos, scaling="by_parts", factor=4.0, orig_len=1024)
    clsa.kv8_write(cache, Kr, Vn, pos)
    idx, cnt = clsa.topk(clsa.index_scores(q_idx, k_idx, seq), seq, k)
    O, lse = clsa.kv8_attn(Qr, cache, cnt, idx=idx)
    check8(cache, Qr, O, lse, cnt.cpu().numpy(), idx.cpu().numpy(), "bf16")
    K_S, V_S = clsa.kv8_read(cache, idx=idx, count=cnt)
    O2, lse2 = clsa.sparse_attn(Qr, K_S, V_S, cnt)
    # the bf16 path rounds its probabilities and its result: 2^-8 each, of values up to max |v| (here under 6)
    assert (O.float() - O2.float()).abs().max() <= 3 * 2.0 ** -8 * float(V_S.abs().max())
    assert (lse - lse2).abs().max() <= 2e-3
