"""Cases of the library's cache operators, timed and compared: rotary positions, an 8-bit
K/V cache (quantised as it is written, read back, attended over) and attention with a
sliding window and sink tokens.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges, ``prepare``
makes a case's inputs on the GPU, ``run`` makes one pass, ``work`` counts the bytes and
operations a pass cannot do without and ``exact`` gives its outputs in 64 bits.  ``run``
computes the operators from elementary torch operations in 32 bits, or calls the library
where ``own`` is true.

Formulas
--------
rope      pair i of the first ``rot`` elements of a head is turned by a = pos * f_i with
          f_i = theta^(-2i/rot), changed by the scaling: linear f_i / factor; base:
          theta * factor^(rot/(rot-2)) in theta's place; by_parts, with the turns
          r = orig_len f_i / 2 pi and g = clamp((r - slow)/(fast - slow), 0, 1):
          g f_i + (1 - g) f_i / factor.  (x1, x2) -> m (x1 cos a - x2 sin a,
          x2 cos a + x1 sin a); pairs are (i, i + rot/2) ("half") or (2i, 2i + 1)
          ("interleaved"); inverse: the transpose (its gradient).
kv8_write block of tokens and head: scale = the smallest power of two s >= 2^-100 with
          max|x| / s <= 448 over the block's finite rows so far, at most 2^119; codes
          e4m3(x / s), ties to even.  A block that already holds earlier rows keeps its
          scale or takes a larger one; then the earlier codes are rounded to the new scale.
kv8_read  code * scale of a range of tokens or of an index list.
kv8_attn  softmax(Q K^T scale) V over the 8-bit cache, every token or an index list.
window    row t of the T newest tokens, at p = len - T + t, sees the tokens j <= p with
          j > p - window or j < sinks.
"""
import math

import torch

own = False

LN2 = math.log(2.0)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # one decode step of 16 sequences of a 32 / 8 head model: a layer's queries and keys
        {"name": "rope_step", "op": "rope", "N": 16, "Hq": 32, "Hk": 8, "d": 128, "rot": 128, "dtype": "bf16",
         "layout": "half", "scaling": "by_parts", "factor": 4.0, "inverse": False},
        # a 32K prompt of the same model
        {"name": "rope_prompt", "op": "rope", "N": 32768, "Hq": 32, "Hk": 8, "d": 128, "rot": 128, "dtype": "bf16",
         "layout": "half", "scaling": "base", "factor": 4.0, "inverse": False},
        # the gradient of a part-of-the-head rotation in full precision, odd token count
        {"name": "rope_part_grad", "op": "rope", "N": 5001, "Hq": 8, "Hk": 2, "d": 128, "rot": 96, "dtype": "f32",
         "layout": "interleaved", "scaling": "linear", "factor": 8.0, "inverse": True},
        # one token appended to each of 16 sequences
        {"name": "write_step", "op": "write", "B": 16, "T": 1, "n": 8192, "Hkv": 8, "d": 128, "block": 64,
         "dtype": "bf16", "ragged": True},
        # chunks of four prompts, of different lengths, behind what the cache holds
        {"name": "write_chunk", "op": "write", "B": 4, "T": 8192, "n": 16384, "Hkv": 8, "d": 128, "block": 64,
         "dtype": "bf16", "ragged": True},
        # a stretch of the cache read back, for a kernel that wants bf16 rows
        {"name": "read_range", "op": "read", "B": 4, "T": 8001, "n": 16384, "Hkv": 8, "d": 128, "block": 64,
         "dtype": "bf16", "select": False},
        # dense decode over one 128K cache, a layer's call
        {"name": "attn8_128k", "op": "attn8", "B": 1, "n": 131072, "L": 1, "Hq": 32, "Hkv": 8, "d": 128, "block": 64,
         "dtype": "bf16", "k": 0, "lo": 131072},
        # 16 sequences of 16K to 128K tokens, dense
        {"name": "attn8_ragged16", "op": "attn8", "B": 16, "n": 131072, "L": 1, "Hq": 32, "Hkv": 8, "d": 128,
         "block": 64, "dtype": "bf16", "k": 0, "lo": 16384},
        # the shared selection of 2048 tokens, all 24 layers' queries
        {"name": "attn8_selected", "op": "attn8", "B": 1, "n": 131072, "L": 24, "Hq": 32, "Hkv": 8, "d": 128,
         "block": 64, "dtype": "bf16", "k": 2048, "lo": 131072},
        # decode step of a window layer, 16 sequences
        {"name": "window_step", "op": "window", "B": 16, "T": 1, "n": 16384, "window": 1024, "sinks": 4, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16", "lo": 900},
        # a chunk of 4096 new rows
        {"name": "window_chunk", "op": "window", "B": 1, "T": 4096, "n": 8192, "window": 1024, "sinks": 4, "Hq": 32,
         "Hkv": 8, "d": 128, "dtype": "bf16", "lo": 8192},
        # a whole prompt with a wide window, odd length
        {"name": "window_prompt", "op": "window", "B": 1, "T": 16381, "n": 16384, "window": 4096, "sinks": 16,
         "Hq": 32, "Hkv": 8, "d": 128, "dtype": "bf16", "lo": 16381},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn8", "window", "attn8", "window"])
    Hq, Hkv = rng.choice([(32, 8), (8, 2), (6, 3), (8, 8), (16, 1)])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "rope":
        N = _log(rng, 1, 16384)
        return {"op": op, "N": N, "Hq": Hq, "Hk": Hkv, "d": d, "rot": 16 * rng.randint(1, d // 16), "dtype": dtype,
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["plain", "linear", "base", "by_parts"]), "factor": rng.uniform(1.5, 16.0),
                "inverse": rng.random() < 0.3}
    block = rng.choice([16, 32, 64, 128])
    if op in ("write", "read"):
        T = _log(rng, 1, 8192)
        B = min(16, max(1, 16384 // T), _log(rng, 1, 16))
        n = T + rng.randint(1, 4096)
        c = {"op": op, "B": B, "T": T, "n": n, "Hkv": Hkv, "d": d, "block": block, "dtype": dtype}
        if op == "write":
            c["ragged"] = rng.random() < 0.7
        else:
            c["select"] = rng.random() < 0.5
        return c
    if op == "attn8":
        n = _log(rng, 1, 131072)
        B = min(_log(rng, 1, 16), max(1, 600000 // n))
        k = _log(rng, 1, min(n, 4096)) if rng.random() < 0.4 else 0
        L = _log(rng, 1, 24) if k else rng.choice([1, 1, 2])
        if Hq // Hkv * L > 128:
            L = max(1, 128 // (Hq // Hkv))
        return {"op": op, "B": B, "n": n, "L": L, "Hq": Hq, "Hkv": Hkv, "d": d, "block": block, "dtype": dtype, "k": k,
                "lo": rng.randint(1, n)}
    T = 1 if rng.random() < 0.4 else _log(rng, 2, 4096 if dtype == "f32" else 12000)
    W = _log(rng, 1, 1024 if dtype == "f32" else 4096)
    B = rng.randint(1, 16) if T < 64 else 1 if T > 2000 else rng.randint(1, 3)
    n = T + rng.randint(0, 6000)
    return {"op": op, "B": B, "T": T, "n": n, "window": W, "sinks": rng.choice([0, 1, 4, 5, 64]), "Hq": Hq, "Hkv": Hkv,
            "d": d, "dtype": dtype, "lo": rng.randint(T, n)}


# ------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(g, lo, hi, *shape):
    """Whole numbers of [lo, hi]."""
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _keys(g, shape, dtype):
    """Cache rows: normal, a few channels of each head larger, as keys have them."""
    x = _randn(g, *shape)
    x[..., ::37] *= 6.0
    return x.to(DT[dtype])


def _theta(c):
    return 10000.0 if c["scaling"] == "plain" else 500000.0


ORIG_LEN, FAST, SLOW = 32768, 32.0, 1.0


def _cached(g, B, n, Hkv, d, block):
    """A filled 8-bit cache, sequence by sequence (it is large): codes and scales."""
    nb = (n + block - 1) // block
    codes = [torch.empty(B, n, Hkv, d, device="cuda", dtype=E4M3) for _ in range(2)]
    scales = [torch.empty(B, nb, Hkv, device="cuda", dtype=torch.float32) for _ in range(2)]
    for b in range(B):
        for which in range(2):
            x = _randn(g, n, Hkv, d)
            if which == 0:
                x[..., ::37] *= 6.0
            s = _block_scales(x[None], block)[0]
            codes[which][b] = (x / s.repeat_interleave(block, 0)[:n, :, None]).to(E4M3)
            scales[which][b] = s
    return codes[0], codes[1], scales[0], scales[1]


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "rope":
        st["q"] = _randn(g, c["N"], c["Hq"], c["d"]).to(DT[c["dtype"]])
        st["k"] = _randn(g, c["N"], c["Hk"], c["d"]).to(DT[c["dtype"]])
        st["pos"] = _ints(g, 0, 131071, c["N"])
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        return st
    B, n, Hkv, d = c["B"], c["n"], c["Hkv"], c["d"]
    if c["op"] == "write":
        # the cache holds earlier rows, smaller than the new ones now and then, so that some
        # blocks that both share have to take a larger scale
        K8, V8, ks, vs = _cached(g, B, n, Hkv, d, c["block"])
        st.update(K8=K8, V8=V8, ks=ks, vs=vs)
        st["K"], st["V"] = _keys(g, (B, c["T"], Hkv, d), c["dtype"]), (_randn(g, B, c["T"], Hkv, d) * 1.5).to(DT[c["dtype"]])
        st["start"] = _ints(g, 0, n - c["T"], B)
        st["count"] = _ints(g, max(1, c["T"] // 2), c["T"], B) if c["ragged"] else torch.full((B,), c["T"], device="cuda", dtype=torch.int32)
        return st
    if c["op"] == "read":
        K8, V8, ks, vs = _cached(g, B, n, Hkv, d, c["block"])
        st.update(K8=K8, V8=V8, ks=ks, vs=vs)
        if c["select"]:
            st["idx"] = _selection(g, B, n, c["T"])
            st["start"] = None
        else:
            st["idx"], st["start"] = None, _ints(g, 0, n - c["T"], B)
        st["K_out"] = torch.zeros(B, c["T"], Hkv, d, device="cuda", dtype=DT[c["dtype"]])
        st["V_out"] = torch.zeros_like(st["K_out"])
        return st
    Hq = c["Hq"]
    st["lens"] = _ints(g, c["lo"], n, B)
    if c["op"] == "attn8":
        K8, V8, ks, vs = _cached(g, B, n, Hkv, d, c["block"])
        st.update(K8=K8, V8=V8, ks=ks, vs=vs)
        st["Q"] = _randn(g, c["L"], B, Hq, d).to(DT[c["dtype"]])
        st["idx"] = None
        if c["k"]:
            st["idx"] = _selection(g, B, c["lo"], min(c["k"], c["lo"]))
            st["lens"] = torch.full((B,), st["idx"].shape[1], device="cuda", dtype=torch.int32)
        st["O"] = torch.empty_like(st["Q"])
        st["lse"] = torch.empty(c["L"], B, Hq, device="cuda", dtype=torch.float32)
        return st
    st["Q"] = _randn(g, B, c["T"], Hq, d).to(DT[c["dtype"]])
    st["K"], st["V"] = _keys(g, (B, n, Hkv, d), c["dtype"]), _randn(g, B, n, Hkv, d).to(DT[c["dtype"]])
    st["O"] = torch.empty_like(st["Q"])
    st["lse"] = torch.empty(B, c["T"], Hq, device="cuda", dtype=torch.float32)
    return st


def _selection(g, B, n, k):
    """k different tokens of n for each sequence, ascending."""
    return torch.rand(B, n, generator=g, device="cuda").argsort(1)[:, :k].sort(1).values.to(torch.int32).contiguous()


# ------------------------------------------------------------------------ plain forms

def _freqs(c):
    """Radians a token, fp64 [rot / 2]."""
    rot, f = c["rot"], c["factor"]
    theta = _theta(c)
    if c["scaling"] == "base":
        theta = theta * f ** (rot / (rot - 2))
    w = theta ** (-2.0 * torch.arange(rot // 2, device="cuda", dtype=torch.float64) / rot)
    if c["scaling"] == "linear":
        return w / f
    if c["scaling"] == "by_parts":
        g = ((ORIG_LEN * w / (2 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0, 1)
        return g * w + (1 - g) * w / f
    return w


def _mscale(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "by_parts" else 1.0


def _rotate(x, cos, sin, rot, layout):
    y = x.float()
    if layout == "half":
        a, b = y[..., : rot // 2], y[..., rot // 2: rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _pow2_scale(amax):
    """The smallest power of two s in [2^-100, 2^119] with amax / s <= 448."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1): 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-100, 119)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.full_like(e, -100)))


def _block_scales(x, block):
    """Scales [B][blocks][Hkv] of rows [B][n][Hkv][d] that fill their blocks from the first on."""
    B, n, H, d = x.shape
    nb = (n + block - 1) // block
    a = torch.zeros(B, nb * block, H, device=x.device, dtype=torch.float32)
    a[:, :n] = x.abs().amax(-1).float()
    return _pow2_scale(a.view(B, nb, block, H).amax(2))


def _write_plain(X, codes, scales, start, count, block):
    """The rows of X behind start, into codes and scales (in place)."""
    B, T, H, d = X.shape
    n, nb = codes.shape[1], scales.shape[1]
    x = X.float()
    t = torch.arange(T, device=X.device)
    live = t[None] < count[:, None]
    tok = torch.where(live, start[:, None] + t[None], 0).long()
    blk = tok // block
    need = torch.full((B, nb, H), -1.0, device=X.device)
    amax = torch.where(live[..., None], x.abs().amax(-1), -1.0)
    need.scatter_reduce_(1, blk[..., None].expand(B, T, H), amax, "amax")
    touched = need >= 0
    first = torch.arange(nb, device=X.device)[None] * block
    kept = (first < start[:, None])[..., None]  # blocks with earlier rows
    old = scales.clone()
    new = _pow2_scale(need.clamp_min(0))
    new = torch.where(kept, torch.maximum(new, old), new)
    scales.copy_(torch.where(touched, new, old))
    # earlier rows of the one block that both share, rounded to a larger scale
    lo = (start // block) * block
    r = torch.arange(block, device=X.device)
    etok = (lo[:, None] + r[None])
    early = (etok < start[:, None])
    etok = torch.where(early, etok, 0).long()
    bi = torch.arange(B, device=X.device)[:, None]
    eb = (lo // block).long()[:, None]
    ratio = torch.where(early[..., None], old[bi, eb] / scales[bi, eb], 1.0)
    rows = (codes[bi, etok].float() * ratio[..., None]).to(E4M3)
    bs, rs = torch.nonzero(early & (count > 0)[:, None], as_tuple=True)
    codes.view(torch.uint8)[bs, etok[bs, rs]] = rows.view(torch.uint8)[bs, rs]
    s = scales.gather(1, blk[..., None].expand(B, T, H))
    fresh = (x / s[..., None]).clamp(-448.0, 448.0).to(E4M3)
    bs, ts = torch.nonzero(live, as_tuple=True)
    codes.view(torch.uint8)[bs, tok[bs, ts]] = fresh.view(torch.uint8)[bs, ts]


def _softmax_rows(s, v):
    """softmax(s) v and its log-sum-exp over the last axis of s; rows of -inf give 0 and -inf."""
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == -math.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / l.masked_fill(l == 0, 1.0)
    return o, (m + torch.log(l)).squeeze(-1)


def _read_plain(codes, scales, tok, block, b):
    return codes[b, tok].float() * scales[b, tok // block][..., None]


def _attn8_plain(st):
    c = st["case"]
    L, B, Hq, d = st["Q"].shape
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    for b in range(B):  # ragged: one sequence at a time
        tok = st["idx"][b].long() if st["idx"] is not None else torch.arange(c["n"], device="cuda")[: st["lens"][b]]
        k = _read_plain(st["K8"], st["ks"], tok, c["block"], b).transpose(0, 1)  # [Hkv][tokens][d]
        v = _read_plain(st["V8"], st["vs"], tok, c["block"], b).transpose(0, 1)
        q = st["Q"][:, b].float().view(L, Hkv, G, d).transpose(0, 1).reshape(Hkv, L * G, d)
        o, lse = _softmax_rows(q @ k.transpose(1, 2) * d ** -0.5, v)
        st["O"][:, b] = o.view(Hkv, L, G, d).transpose(0, 1).reshape(L, Hq, d).to(st["O"].dtype)
        st["lse"][:, b] = lse.view(Hkv, L, G).transpose(0, 1).reshape(L, Hq)
    return {"O": st["O"], "lse": st["lse"]}


def _window_plain(st):
    c = st["case"]
    B, T, Hq, d = st["Q"].shape
    Hkv, G, W, S = c["Hkv"], c["Hq"] // c["Hkv"], c["window"], c["sinks"]
    rows = 1024  # query rows at a time, over the tokens that any of them sees
    for b, n in enumerate(st["lens"].tolist()):
        for t0 in range(0, T, rows):
            t1 = min(T, t0 + rows)
            p = torch.arange(n - T + t0, n - T + t1, device="cuda")
            lo, hi = max(0, n - T + t0 - W + 1), max(1, n - T + t1)
            j = torch.cat([torch.arange(min(S, lo), device="cuda"), torch.arange(lo, hi, device="cuda")])
            see = (j <= p[:, None]) & ((j > p[:, None] - W) | (j < S))
            k = st["K"][b, j].float().transpose(0, 1)
            v = st["V"][b, j].float().transpose(0, 1)
            q = st["Q"][b, t0:t1].float().view(t1 - t0, Hkv, G, d).permute(1, 2, 0, 3).reshape(Hkv, -1, d)
            s = (q @ k.transpose(1, 2) * d ** -0.5).view(Hkv, G, t1 - t0, -1).masked_fill(~see, -math.inf)
            o, lse = _softmax_rows(s.flatten(1, 2), v)
            st["O"][b, t0:t1] = o.view(Hkv, G, t1 - t0, d).permute(2, 0, 1, 3).reshape(t1 - t0, Hq, d).to(st["O"].dtype)
            st["lse"][b, t0:t1] = lse.view(Hkv, G, t1 - t0).permute(2, 0, 1).reshape(t1 - t0, Hq)
    return {"O": st["O"], "lse": st["lse"]}


def _plain(st):
    c = st["case"]
    if c["op"] == "rope":
        a = st["pos"].double()[:, None] * _freqs(c)
        cos, sin = (torch.cos(a) * _mscale(c)).float()[:, None], (torch.sin(a) * _mscale(c)).float()[:, None]
        if c["inverse"]:
            sin = -sin
        st["q_out"] = _rotate(st["q"], cos, sin, c["rot"], c["layout"])
        st["k_out"] = _rotate(st["k"], cos, sin, c["rot"], c["layout"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if c["op"] == "write":
        _write_plain(st["K"], st["K8"], st["ks"], st["start"], st["count"], c["block"])
        _write_plain(st["V"], st["V8"], st["vs"], st["start"], st["count"], c["block"])
        return {"K8": st["K8"], "V8": st["V8"], "ks": st["ks"], "vs": st["vs"]}
    if c["op"] == "read":
        tok = st["idx"].long() if st["idx"] is not None else st["start"][:, None].long() + torch.arange(c["T"], device="cuda")
        bi = torch.arange(c["B"], device="cuda")[:, None]
        return {"K": _read_plain(st["K8"], st["ks"], tok, c["block"], bi).to(DT[c["dtype"]]),
                "V": _read_plain(st["V8"], st["vs"], tok, c["block"], bi).to(DT[c["dtype"]])}
    return _attn8_plain(st) if c["op"] == "attn8" else _window_plain(st)


# ------------------------------------------------------------------------------- a pass

def run(state):
    if not own:
        return _plain(state)
    from long_context_sparse_clsa_b200 import clsa
    st, c = state, state["case"]
    if c["op"] == "rope":
        q, k = clsa.rope(st["q"], st["k"], st["pos"], rot=c["rot"], layout=c["layout"], theta=_theta(c),
                         scaling=c["scaling"], factor=c["factor"], orig_len=ORIG_LEN, beta_fast=FAST, beta_slow=SLOW,
                         mscale=_mscale(c), inverse=c["inverse"], q_out=st["q_out"], k_out=st["k_out"])
        return {"q": q, "k": k}
    if "ws" not in st:  # the cache handle and the workspace, which a program keeps
        st["cache"] = clsa.Kv8Cache(st["K8"], st["V8"], st["ks"], st["vs"], c["block"]) if "K8" in st else None
        if c["op"] == "attn8":
            need = clsa.kv8_attn_workspace_size(st["Q"], st["cache"], st["idx"])
        elif c["op"] == "window":
            need = clsa.window_attn_workspace_size(st["Q"], st["K"], c["window"], c["sinks"])
        else:
            need = 256
        st["ws"] = clsa.Workspace(need)
    if c["op"] == "write":
        clsa.kv8_write(st["cache"], st["K"], st["V"], st["start"], st["count"], ws=st["ws"])
        return {"K8": st["K8"], "V8": st["V8"], "ks": st["ks"], "vs": st["vs"]}
    if c["op"] == "read":
        K, V = clsa.kv8_read(st["cache"], st["K_out"], st["V_out"], start=st["start"], idx=st["idx"], ws=st["ws"])
        return {"K": K, "V": V}
    if c["op"] == "attn8":
        O, lse = clsa.kv8_attn(st["Q"], st["cache"], st["lens"], idx=st["idx"], ws=st["ws"], O=st["O"], lse=st["lse"])
    else:
        O, lse = clsa.window_attn(st["Q"], st["K"], st["V"], st["lens"], c["window"], c["sinks"], ws=st["ws"],
                                  O=st["O"], lse=st["lse"])
    return {"O": O, "lse": lse}


# ------------------------------------------------------------------------ bytes and flops

def work(case):
    c = case
    if c["op"] == "rope":
        return {"bytes": 2 * c["N"] * (c["Hq"] + c["Hk"]) * c["d"] * SIZE[c["dtype"]] + 4 * c["N"],
                "flops": 3 * c["N"] * (c["Hq"] + c["Hk"]) * c["rot"]}
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] in ("write", "read"):
        rows = B * c["T"] * (0.75 if c.get("ragged") and c["T"] > 1 else 1.0)  # ragged counts: half to all
        return {"bytes": rows * Hkv * 2 * (d * (SIZE[c["dtype"]] + 1) + 4.0 / c["block"]),
                "flops": rows * Hkv * 2 * d}
    if c["op"] == "attn8":
        tok = B * (min(c["k"], c["lo"]) if c["k"] else (c["lo"] + c["n"]) / 2)
        qo = c["L"] * B * c["Hq"] * (2 * d * SIZE[c["dtype"]] + 4)
        return {"bytes": tok * Hkv * 2 * (d + 4.0 / c["block"]) + qo + (4 * tok if c["k"] else 0),
                "flops": 4 * tok * c["L"] * c["Hq"] * d}
    T, W, S = c["T"], c["window"], c["sinks"]
    n = (c["lo"] + c["n"]) // 2
    seen = sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(n - T, n))
    rows = min(n, T + W - 1 + S)
    return {"bytes": B * (rows * Hkv * 2 * d * SIZE[c["dtype"]] + T * c["Hq"] * (2 * d * SIZE[c["dtype"]] + 4)),
            "flops": 4 * B * seen * c["Hq"] * d}


# ---------------------------------------------------------------------------- in 64 bits

def _e4m3_exact(x):
    """x (fp64) on the e4m3 grid: 3 mantissa bits, exponents from -6, ties to even, +-448."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _write_exact(X, codes, scales, start, count, block):
    X, codes, scales = X.double(), codes.double(), scales.double()
    for b in range(X.shape[0]):
        p0, p1 = int(start[b]), int(start[b]) + int(count[b])
        for j in range(p0 // block, (p1 - 1) // block + 1):
            a, z = max(p0, j * block), min(p1, (j + 1) * block)
            x = X[b, a - p0: z - p0]
            top = x.abs().amax((0, 2))
            s = torch.exp2(torch.ceil(torch.log2(top.clamp_min(2.0 ** -200) / 448.0) - 1e-12)).clamp_min(2.0 ** -100)
            if j * block < p0:
                s = torch.maximum(s, scales[b, j])
                codes[b, j * block: p0] = _e4m3_exact(codes[b, j * block: p0] * (scales[b, j] / s)[:, None])
            scales[b, j] = s
            codes[b, a:z] = _e4m3_exact(x / s[:, None])
    return codes, scales


def exact(case, seed):
    c, st = case, prepare(case, seed)
    if c["op"] == "rope":
        out, rot = {}, c["rot"]
        f = _freqs(c).tolist()
        turn = torch.polar(torch.full((c["N"], rot // 2), _mscale(c), device="cuda", dtype=torch.float64),
                           st["pos"].double()[:, None] * torch.tensor(f, device="cuda", dtype=torch.float64))
        turn = turn.conj() if c["inverse"] else turn
        for name in ("q", "k"):
            y = st[name].double().clone()
            part = y[..., :rot]
            pairs = part.unflatten(-1, (2, rot // 2)).transpose(-1, -2) if c["layout"] == "half" else part.unflatten(-1, (rot // 2, 2))
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None])
            y[..., :rot] = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
            out[name] = y
        return out
    if c["op"] == "write":
        K8, ks = _write_exact(st["K"], st["K8"], st["ks"], st["start"], st["count"], c["block"])
        V8, vs = _write_exact(st["V"], st["V8"], st["vs"], st["start"], st["count"], c["block"])
        return {"K8": K8, "V8": V8, "ks": ks, "vs": vs}
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "read":
        out = {}
        for name in ("K", "V"):
            rows = []
            for b in range(B):
                tok = st["idx"][b].long() if c["select"] else torch.arange(c["T"], device="cuda") + int(st["start"][b])
                s = st["ks" if name == "K" else "vs"][b].double().repeat_interleave(c["block"], 0)
                rows.append(st[name + "8"][b].double()[tok] * s[tok][..., None])
            out[name] = torch.stack(rows)
        return out
    G = c["Hq"] // Hkv
    O = torch.zeros_like(st["O"], dtype=torch.float64)
    lse = torch.full_like(st["lse"], -math.inf, dtype=torch.float64)
    if c["op"] == "attn8":
        for b in range(B):
            n = int(st["lens"][b])
            tok = st["idx"][b, :n].long() if c["k"] else torch.arange(n, device="cuda")
            for g in range(Hkv):
                k = st["K8"][b, tok, g].double() * st["ks"][b, tok // c["block"], g].double()[:, None]
                v = st["V8"][b, tok, g].double() * st["vs"][b, tok // c["block"], g].double()[:, None]
                h = slice(g * G, (g + 1) * G)
                s = torch.einsum("lhd,nd->lhn", st["Q"][:, b, h].double(), k) / math.sqrt(d)
                O[:, b, h] = torch.einsum("lhn,nd->lhd", torch.softmax(s, -1), v)
                lse[:, b, h] = torch.logsumexp(s, -1)
        return {"O": O, "lse": lse}
    T, W, S = c["T"], c["window"], c["sinks"]
    for b in range(B):
        n = int(st["lens"][b])
        for t0 in range(0, T, 512):
            t1 = min(T, t0 + 512)
            p = torch.arange(t0, t1, device="cuda") + (n - T)
            far = max(0, n - T + t0 - W + 1)
            j = torch.tensor(sorted(set(range(min(S, n))) | set(range(far, n - T + t1))), device="cuda")
            gap = p[:, None] - j[None]
            see = (gap >= 0) & ((gap < W) | (j[None] < S))
            for g in range(Hkv):
                k, v = st["K"][b, j, g].double(), st["V"][b, j, g].double()
                h = slice(g * G, (g + 1) * G)
                s = torch.einsum("thd,nd->htn", st["Q"][b, t0:t1, h].double(), k) / math.sqrt(d)
                s = s.masked_fill(~see, -math.inf)
                O[b, t0:t1, h] = torch.einsum("htn,nd->thd", torch.softmax(s, -1), v)
                lse[b, t0:t1, h] = torch.logsumexp(s, -1).transpose(0, 1)
    return {"O": O, "lse": lse}
