"""The cache operators at the ends of their ranges: head counts that do not share the SMs evenly, many
sequences, both forms of window attention around the sizes where they change over, caches past
2^32 bytes, calls on two streams at once.  Tolerances as in test_gpu_cache_attn.py."""
import numpy as np
import pytest
import torch

from long_context_sparse_clsa_b200 import clsa
from oracle import cache_oracle as C
from test_gpu_cache import DT, cache_of, dev, f64, host
from test_gpu_cache_attn import U, check, check8, check_window, run8, run_window, window_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_clsa_b200.build import build
    build()
    clsa.load_library()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,L,G,Hkv", [(2, 333, 1, 1, 15), (2, 190, 3, 3, 25), (1, 700, 1, 2, 40), (1, 95, 1, 1, 160),
                                         (40, 60, 1, 1, 25), (70, 130, 1, 4, 2), (33, 40, 5, 4, 1)])
def test_kv8_attn_head_counts_and_many_sequences(dtype, B, n, L, G, Hkv):
    cache = cache_of(B, n, Hkv, 64, 32, n)
    g = np.random.default_rng(B)
    counts = g.integers(0, n + 1, B)
    counts[-1] = n
    Q, O, lse, ws = run8(cache, L, B, G * Hkv, dtype, counts)
    check8(cache, Q, O, lse, counts, None, dtype)
    k = min(n, 50)
    idx = np.stack([np.sort(g.permutation(n)[:k]) for _ in range(B)])
    counts = g.integers(0, k + 1, B)
    Q, O, lse, ws = run8(cache, L, B, G * Hkv, dtype, counts, idx)
    check8(cache, Q, O, lse, counts, idx, dtype)


@pytest.mark.parametrize("B,n,Hq,Hkv,d", [(2, 9000, 16, 1, 128), (1, 5000, 24, 3, 128), (3, 2500, 4, 2, 64)])
def test_kv8_attn_every_length_near_a_split(B, n, Hq, Hkv, d):
    """Lengths around multiples of the tile and of the split: the merge over few and many CTAs."""
    cache = cache_of(B, n, Hkv, d, 128, 1)
    for m in (15, 16, 17, 191, 192, 193, 385, 2999, 4097, n - 1):
        counts = [min(m + 16 * b, n) for b in range(B)]
        Q, O, lse, _ = run8(cache, 1, B, Hq, "bf16", counts)
        check8(cache, Q, O, lse, counts, None, "bf16")


@pytest.mark.parametrize("B,T,n,Hq,Hkv,d,window,sinks", [
    (1, 16, 3000, 1, 1, 128, 2000, 4), (1, 17, 3000, 1, 1, 128, 2000, 4), (1, 2, 900, 64, 8, 128, 512, 1), (1, 3, 900, 64, 8, 128, 512, 1),
    (20, 3, 500, 64, 8, 64, 300, 2), (1, 1, 700, 128, 1, 128, 600, 9), (2, 2, 700, 128, 1, 64, 600, 9), (1, 100, 3000, 8, 1, 128, 2500, 0),
    (150, 1, 90, 4, 2, 64, 50, 3), (90, 40, 140, 2, 1, 64, 33, 7), (2, 1, 333, 15, 15, 128, 100, 2), (1, 30, 200, 160, 160, 64, 64, 1),
    (1, 64, 40, 4, 2, 128, 16, 2), (3, 500, 200, 8, 4, 64, 64, 5), (1, 129, 129, 5, 1, 128, 1, 0), (1, 40, 1100, 96, 1, 128, 1000, 1)])
def test_window_attn_around_its_change_of_form(B, T, n, Hq, Hkv, d, window, sinks):
    """Few and many rows, groups from 1 to 128 heads, more sequences than a warp has lanes, T above n."""
    lens = np.random.default_rng(T).integers(0, n + 1, B)
    lens[0] = n
    out = run_window(B, T, n, Hq, Hkv, d, "bf16", lens, window, sinks)
    check_window(*out, lens, window, sinks, "bf16")


@pytest.mark.parametrize("T", [1, 3, 80])
def test_window_attn_takes_any_lengths(T):
    """Lengths below 0 and above n_max are clamped; the largest window and sink counts an int holds."""
    big = 2 ** 31 - 1
    for lens in ([-5, 300], [big, 0], [-big - 1, 7]):
        for window, sinks in ((big, big), (1, big), (big, 0), (20, 3)):
            out = run_window(2, T, 120, 8, 2, 64, "bf16", lens, window, sinks)
            check_window(*out, np.array(lens), min(window, 120), min(sinks, 120), "bf16")


def test_8bit_cache_past_32_bits():
    """4.3 M tokens of 8 heads of 128: 4.4e9 codes on each side.  Written, read and attended over at the far
    end and, dense, over all of it."""
    n, H, d, block = 4_300_000, 8, 128, 128
    cache = clsa.Kv8Cache.empty(1, n, H, d, block)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for t in (cache.K8, cache.V8):
        u = t.view(torch.uint8).view(-1)
        for i in range(0, u.numel(), 1 << 30):
            u[i:i + (1 << 30)].random_(0, 256, generator=gen).bitwise_and_(0xBF)  # magnitudes below 2, no NaN
    cache.k_scale.fill_(2.0 ** -7)
    cache.v_scale.fill_(2.0 ** -7)
    g = np.random.default_rng(0)
    T = 300
    K, V = (dev(g.standard_normal((1, T, H, d)), torch.bfloat16) for _ in range(2))
    start = dev(np.array([n - T]), torch.int32)
    clsa.kv8_write(cache, K, V, start)
    got = clsa.kv8_read(cache, T=T, start=start, dtype=torch.float32)
    for x, y in zip((K, V), got):
        # e4m3: 2^-4 of the value; below 2^-6 of the scale's unit, half a step of 2^-9 (scales: at most max / 224)
        assert ((x.float() - y).abs() <= x.float().abs() * 2.0 ** -4 + 2.0 ** -10 * float(x.float().abs().max()) / 224).all()
    Q = dev(g.standard_normal((1, 1, 16, d)), torch.bfloat16)
    kv, vv = cache.K8.view(torch.float8_e4m3fn), cache.V8.view(torch.float8_e4m3fn)

    def values(codes, scale, tok, h):
        return codes[0, tok, h].double() * scale[0, tok // block, h].double()[:, None]

    idx = np.sort(np.concatenate([g.integers(0, 5000, 200), g.integers(n - 5000, n, 300)]))
    idx[-1] = n - 1
    ti = dev(idx[None], torch.int32)
    O, lse = clsa.kv8_attn(Q, cache, dev(np.array([500]), torch.int32), idx=ti)
    O2, lse2 = clsa.kv8_attn(Q, cache, dev(np.array([n]), torch.int32))
    # a warp adds up its share of the tokens (n over 18 CTAs of 12 warps), then 216 partials
    for toks, o, ls, terms in ((torch.from_numpy(idx).cuda(), O, lse, 500), (torch.arange(n, device="cuda"), O2, lse2, n // 216 + 300)):
        for h in (0, 7):
            q = Q[0, 0, 2 * h:2 * h + 2].double()
            s, av, vs = [], [], []
            for i in range(0, len(toks), 1 << 19):
                tk = toks[i:i + (1 << 19)]
                s.append(q @ values(kv, cache.k_scale, tk, h).T * d ** -0.5)
            s = torch.cat(s, 1)
            want = torch.logsumexp(s, 1)
            p = torch.exp(s - want[:, None])
            oo, aa, mag, fl, top = 0, 0, torch.zeros(2, device="cuda", dtype=torch.float64), 0, 0.0
            for i in range(0, len(toks), 1 << 19):
                tk = toks[i:i + (1 << 19)]
                v, pc, sv = values(vv, cache.v_scale, tk, h), p[:, i:i + (1 << 19)], cache.v_scale[0, tk // block, h].double()
                oo, aa = oo + pc @ v, aa + pc @ v.abs()
                mag = torch.maximum(mag, (q.abs() @ values(kv, cache.k_scale, tk, h).abs().T).amax(1) * d ** -0.5)
                fl, top = fl + (v.abs() / sv[:, None]).sum(0)[None], max(top, float((pc * sv).max()))
            floor = 2.0 ** -32 * top * fl
            check(o[0, 0, 2 * h:2 * h + 2], ls[0, 0, 2 * h:2 * h + 2], oo.cpu().numpy(), want.cpu().numpy(), aa.cpu().numpy(), "bf16",
                  2.0 ** -11, mag.cpu().numpy(), terms, d, floor.cpu().numpy())


@pytest.mark.parametrize("T", [1, 200])
def test_window_attn_past_32_bits(T):
    """A bf16 cache of 2.2e9 elements on each side, attended over at its far end."""
    n, H, d, window, m = 2_200_000, 8, 128, 700, 1200
    g = np.random.default_rng(T)
    K, V = (torch.zeros(1, n, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (K, V):
        t[:, n - m:] = dev(g.standard_normal((1, m, H, d)), torch.bfloat16)
        t[:, :n - m].fill_(float("nan"))
    Q = dev(g.standard_normal((1, T, 16, d)), torch.bfloat16)
    O, lse = clsa.window_attn(Q, K, V, dev(np.array([n]), torch.int32), window)
    check_window(Q, K[:, n - m:], V[:, n - m:], O, lse, np.array([m]), window, 0, "bf16")


def test_calls_on_two_streams_at_once():
    """Each operator on two streams, side by side on data of their own, as one after the other."""
    g = np.random.default_rng(0)
    B, T, H, d = 2, 900, 4, 128
    side = torch.cuda.Stream()
    sets = []
    for i in range(2):
        cache = cache_of(B, 2048, H, d, 64, i)
        K, V = (dev(g.standard_normal((B, T, H, d)), torch.bfloat16) for _ in range(2))
        Q = dev(g.standard_normal((1, B, 16, d)), torch.bfloat16)
        Kc, Vc = (dev(g.standard_normal((B, 2048, H, d)), torch.bfloat16) for _ in range(2))
        Qc = dev(g.standard_normal((B, T, 16, d)), torch.bfloat16)
        pos = dev(g.integers(0, 9000, B * T), torch.int32)
        start, cnt = dev(np.array([5, 1000]), torch.int32), dev(np.array([900, 1900]), torch.int32)
        sets.append((cache, K, V, Q, Kc, Vc, Qc, pos, start, cnt))
    torch.cuda.synchronize()

    def run(cache, K, V, Q, Kc, Vc, Qc, pos, start, cnt):
        cache = clsa.Kv8Cache(cache.K8.clone(), cache.V8.clone(), cache.k_scale.clone(), cache.v_scale.clone(), cache.block)
        _, Kr = clsa.rope(None, K.view(B * T, H, d), pos)
        clsa.kv8_write(cache, Kr.view(K.shape), V, start)
        out = [*clsa.kv8_attn(Q, cache, cnt), *clsa.kv8_read(cache, T=100, start=start)]
        return out + [cache.K8, cache.V8, cache.k_scale, cache.v_scale, *clsa.window_attn(Qc, Kc, Vc, cnt, 300, 4),
                      *clsa.window_attn(Qc[:, :1].contiguous(), Kc, Vc, cnt, 300, 4)]

    want = [run(*x) for x in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        a = run(*sets[0])
        with torch.cuda.stream(side):
            b = run(*sets[1])
        torch.cuda.synchronize()
        for got, exp in zip((a, b), want):
            assert all(torch.equal(x.view(torch.uint8) if x.dtype.itemsize == 1 else x, y.view(torch.uint8) if y.dtype.itemsize == 1 else y)
                       for x, y in zip(got, exp))


def test_a_workspace_serves_other_sizes_once_zeroed():
    g = np.random.default_rng(1)
    ws = clsa.Workspace(1 << 22)
    K, V = (dev(g.standard_normal((3, 2000, 2, 128)), torch.bfloat16) for _ in range(2))
    for B, Hq, T in ((3, 8, 1), (1, 2, 1), (2, 16, 1), (3, 8, 2), (3, 8, 50)):
        Q = dev(g.standard_normal((B, T, Hq, 128)), torch.bfloat16)
        lens = np.array([2000, 900, 1500][:B])
        ws.buf.zero_()
        O, lse = clsa.window_attn(Q, K[:B], V[:B], dev(lens, torch.int32), 1800, 4, ws=ws)
        check_window(Q, K[:B], V[:B], O, lse, lens, 1800, 4, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,n,H,d,block,at", [(2, 70, 100, 5, 64, 16, 7), (1, 33, 64, 3, 128, 16, 0), (3, 40, 90, 7, 64, 32, 20),
                                               (1, 900, 1000, 1, 64, 16, 3), (2, 1, 50, 9, 64, 16, 17)])
def test_kv8_write_several_heads_a_cta_at_any_alignment(dtype, B, T, n, H, d, block, at):
    """Small blocks share a CTA with other heads', also where the heads do not divide; rows 16- but not
    32-byte aligned; a value that is not finite in one head leaves the others' scales alone."""
    g = np.random.default_rng(T)
    off = 8 if dtype == "bf16" else 4                      # elements: 16 bytes
    rows = []
    for _ in range(2):
        flat = torch.empty(B * T * H * d + off, dtype=DT[dtype], device="cuda")
        x = flat[off:].view(B, T, H, d)
        x.copy_(dev(g.standard_normal((B, T, H, d)) * np.exp2(g.uniform(-9, 9, (B, 1, H, 1))), DT[dtype]))
        assert x.data_ptr() % 32 == 16
        rows.append(x)
    K, V = rows
    K[0, T // 2, H - 1, 5] = float("inf")
    V[B - 1, 0, 0, d - 1] = float("nan")
    cache = cache_of(B, n, H, d, block, 5)
    start = np.full(B, at)
    start[-1] = 0
    count = g.integers(1, T + 1, B)
    count[0] = T
    before = host(cache)
    clsa.kv8_write(cache, K, V, dev(start, torch.int32), dev(count, torch.int32))
    want = [C.kv8_write(c, s, f64(x), start, count, block) for x, c, s in ((K, before[0], before[2]), (V, before[1], before[3]))]
    got = host(cache)
    for side in range(2):
        codes, scales = want[side]
        np.testing.assert_array_equal(got[2 + side], scales)
        nan = (got[side] & 127) == 127
        np.testing.assert_array_equal(nan, (codes & 127) == 127)
        np.testing.assert_array_equal(got[side][~nan], codes[~nan])
    out = [torch.empty(B * T * H * d + off, dtype=DT[dtype], device="cuda")[off:].view(B, T, H, d).fill_(7) for _ in range(2)]
    clsa.kv8_read(cache, *out, start=dev(start, torch.int32), count=dev(count, torch.int32))
    al = clsa.kv8_read(cache, T=T, start=dev(start, torch.int32), dtype=DT[dtype])
    for x, y in zip(out, al):
        for b in range(B):
            assert torch.equal(x[b, :count[b]].nan_to_num(-3), y[b, :count[b]].nan_to_num(-3)) and bool((x[b, count[b]:] == 7).all())


@pytest.mark.parametrize("T,d", [(1, 128), (200, 128), (200, 64)])
def test_attention_outputs_at_any_alignment(T, d):
    """O, Q and the cache 16- but not 32-byte aligned: the same bits as elsewhere."""
    g = np.random.default_rng(d)

    def off(t):
        u = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")[8:].view(t.shape)
        assert u.data_ptr() % 32 == 16
        return u.copy_(t)

    Q = dev(g.standard_normal((2, T, 8, d)), torch.bfloat16)
    K, V = (dev(g.standard_normal((2, 500, 2, d)), torch.bfloat16) for _ in range(2))
    lens = dev(np.array([500, 130]), torch.int32)
    want, wl = clsa.window_attn(Q, K, V, lens, 200, 4)
    got, gl = clsa.window_attn(off(Q), off(K), off(V), lens, 200, 4, O=off(torch.zeros_like(Q)))
    assert torch.equal(want, got) and torch.equal(wl, gl)
    cache = cache_of(2, 300, 2, d, 32, 1)
    Q = dev(g.standard_normal((1, 2, 8, d)), torch.bfloat16)
    cnt = dev(np.array([300, 77]), torch.int32)
    want, wl = clsa.kv8_attn(Q, cache, cnt)
    got, gl = clsa.kv8_attn(off(Q), cache, cnt, O=off(torch.zeros_like(Q)))
    assert torch.equal(want, got) and torch.equal(wl, gl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,L,Hq,Hkv,d", [(300, 60, 1, 8, 2, 64), (90, 130, 2, 32, 8, 64), (40, 200, 1, 6, 3, 128), (260, 33, 1, 15, 15, 64),
                                           (21, 100, 6, 12, 1, 128)])
def test_kv8_attn_more_units_than_ctas(dtype, B, n, L, Hq, Hkv, d):
    """Many short sequences: a warp each, empty ones among them, dense and selected; the same bits in a second
    call."""
    cache = cache_of(B, n, Hkv, d, 16, B)
    g = np.random.default_rng(n)
    counts = g.integers(0, n + 1, B)
    counts[:3] = (n, 0, 1)
    Q, O, lse, ws = run8(cache, L, B, Hq, dtype, counts)
    check8(cache, Q, O, lse, counts, None, dtype)
    O2, lse2 = clsa.kv8_attn(Q, cache, dev(counts, torch.int32), ws=ws)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    k = min(n, 40)
    idx = np.stack([np.sort(g.permutation(n)[:k]) for _ in range(B)])
    counts = g.integers(0, k + 1, B)
    Q, O, lse, ws = run8(cache, L, B, Hq, dtype, counts, idx)
    check8(cache, Q, O, lse, counts, idx, dtype)
    assert ws.status()[0] == "CLSA_OK"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,n,Hq,Hkv,d,window,sinks", [(1, 700, 900, 6, 3, 128, 6, 0), (3, 300, 400, 8, 2, 64, 7, 3), (200, 1, 300, 8, 2, 128, 40, 4),
                                                        (120, 2, 200, 4, 2, 64, 150, 17), (1, 900, 1000, 16, 8, 64, 100, 1)])
def test_window_attn_more_units_than_ctas(dtype, B, T, n, Hq, Hkv, d, window, sinks):
    lens = np.random.default_rng(B).integers(0, n + 1, B)
    lens[-1] = 0
    lens[0] = n
    out = run_window(B, T, n, Hq, Hkv, d, dtype, lens, window, sinks)
    check_window(*out, lens, window, sinks, dtype)


def test_a_decode_loop_back_to_back_is_the_loop_with_pauses():
    """Positions, write, dense and window attention of 60 steps in a row, one launch behind the other, eager and
    captured: every step reads what the launch before it wrote."""
    g = np.random.default_rng(4)
    B, Hq, H, d, steps, n0 = 3, 8, 2, 128, 60, 500
    Q = dev(g.standard_normal((steps, B, Hq, d)), torch.bfloat16)
    Kn, Vn = (dev(g.standard_normal((steps, B, 1, H, d)) * np.exp2(g.uniform(-3, 3, (steps, B, 1, 1, 1))), torch.bfloat16) for _ in range(2))
    K0, V0 = (dev(g.standard_normal((B, n0, H, d)), torch.bfloat16) for _ in range(2))
    zero, lens = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), n0, dtype=torch.int32, device="cuda")
    wws, aws, kws = clsa.Workspace(1 << 22), clsa.Workspace(1 << 22), clsa.Workspace(256)

    def loop(pause, O, W, pos):
        cache = clsa.Kv8Cache.empty(B, n0 + steps, H, d, 32)
        Kb, Vb = (torch.zeros(B, n0 + steps, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        clsa.kv8_write(cache, K0, V0, zero, ws=kws)
        pos.copy_(lens)
        for t in range(steps):
            q, k = clsa.rope(Q[t], Kn[t].view(B, H, d), pos)
            pause()
            clsa.kv8_write(cache, k.view(B, 1, H, d), Vn[t], pos, ws=kws)
            pause()
            clsa.kv8_read(cache, Kb, Vb, ws=kws)
            pause()
            pos += 1
            pause()
            clsa.kv8_attn(q, cache, pos, ws=aws, O=O[t], want_lse=False)
            pause()
            clsa.window_attn(q.view(B, 1, Hq, d), Kb, Vb, pos, 200, 2, ws=wws, O=W[t].view(B, 1, Hq, d), want_lse=False)
            pause()

    outs = []
    for pause in (torch.cuda.synchronize, lambda: None):
        O, W, pos = torch.empty_like(Q), torch.empty_like(Q), lens.clone()
        loop(pause, O, W, pos)
        outs.append((O, W))
    O, W, pos = torch.empty_like(Q), torch.empty_like(Q), lens.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop(lambda: None, O, W, pos)
    for _ in range(3):
        graph.replay()
        outs.append((O.clone(), W.clone()))
    torch.cuda.synchronize()
    for o, w in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(w, outs[0][1])


@pytest.mark.parametrize("T,d", [(888, 128), (1184, 64), (1, 128), (40, 64)])
def test_fp32_sums_are_rounded_not_cut_off(T, d):
    """Means of 3000 positive values (Q = 0: every p is 1).  A tile's products are cut off at 24 bits at most 6
    times (12 u), added to the output n / 16 times (u each), the sum of p 32 at a time; merging, the division
    and the result's rounding: 64 u are plenty.  Sums that the tensor core cuts off all the way lose 6 n / 16
    times up to 2 u, all in one direction."""
    g = np.random.default_rng(d)
    n, W = 4000, 3000
    K = dev(g.standard_normal((1, n, 1, d)))
    V = dev(g.uniform(0.5, 1, (1, n, 1, d)))
    Q = torch.zeros(1, T, 16, d, device="cuda")
    O, lse = clsa.window_attn(Q, K, V, dev(np.array([n]), torch.int32), W)
    c = torch.cat([torch.zeros(1, d, dtype=torch.float64, device="cuda"), V[0, :, 0].double().cumsum(0)])
    p = torch.arange(n - T, n, device="cuda")
    want = ((c[p + 1] - c[p + 1 - W]) / W)[:, None]
    err = ((O[0].double() - want).abs() / want).max()
    assert float(err) <= (W / 16 + 64) * U, float(err) / U
    # the same mean over an 8-bit cache of which every token is seen
    cache = clsa.Kv8Cache.empty(1, W, 1, d, 16)
    codes = g.integers(0x30, 0x38, (1, W, 1, d))                # 0.5 to 0.9375
    cache.V8.view(torch.uint8).copy_(dev(codes, torch.uint8))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    B = max(T, 2)
    O, _ = clsa.kv8_attn(torch.zeros(1, B, 8, d, device="cuda"), cache, torch.full((B,), W, dtype=torch.int32, device="cuda"))
    want = cache.V8.double().mean(1)[0, 0]
    err = ((O[0].double() - want).abs() / want).max()
    assert float(err) <= (W / 16 + 64) * U, float(err) / U
