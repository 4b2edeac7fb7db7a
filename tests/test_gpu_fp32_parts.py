"""fp32 rows on the tensor cores: products and sums as fp32 arithmetic has them, without a drift to one side."""
import numpy as np
import pytest
import torch

from long_context_sparse_clsa_b200 import clsa
from test_gpu_cache import dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_clsa_b200.build import build
    build()
    clsa.load_library()


@pytest.mark.parametrize("d", [64, 128])
def test_products_of_fp32_windows_are_fp32_products(d):
    """One token, one element of q and k that is not 0: the log-sum-exp is the product x y, times the fp32
    constants log2(e) and ln 2.  Off by the parts' dropped products, 3 u (one factor's parts are rounded, the middle
    one at most 2^-8 of it and the last 2^-17, the other's cut off, 2^-7 and 2^-15: 2^-23 + 2^-24), and three
    roundings (the sum of the parts' products, times each constant), u each; what the tensor core cuts off lies
    in the small parts, under 2^-6 u.  6.1 u in all.  No side is favoured: with a spread of about u the mean of
    4096 is within 0.25 u at 16 times its own deviation (parts that are all cut off drop 0.63 u on the average)."""
    g = np.random.default_rng(d)
    B, H = 128, 32
    x, y = (np.float32(g.uniform(1, 2, (B, H))) * np.float32(2.0) ** g.integers(-3, 4, (B, H)) for _ in range(2))
    x[:2], y[:2] = 1 + 2.0 ** -7 - 2.0 ** -23, 1 + 2.0 ** -7 - 2.0 ** -23   # large middle and last parts of a cut
    x[2:4], y[2:4] = 2 - 2.0 ** -23, 1 + 2.0 ** -8 - 2.0 ** -23
    q, k = np.zeros((B, 1, H, d), np.float32), np.zeros((B, 1, H, d), np.float32)
    at = (np.arange(B * H) % d).reshape(B, H)
    np.put_along_axis(q[:, 0], at[..., None], x[..., None], -1)
    np.put_along_axis(k[:, 0], at[..., None], y[..., None], -1)
    V = dev(g.standard_normal((B, 1, H, d)))
    O, lse = clsa.window_attn(dev(q), dev(k), V, torch.ones(B, dtype=torch.int32, device="cuda"), 4, scale=1.0)
    assert torch.equal(O, V)                            # one token: its value
    want = x.astype(np.float64) * y * float(np.float32(1.4426950408889634)) * float(np.float32(0.6931471805599453))
    err = (lse[:, 0].cpu().numpy().astype(np.float64) - want) / want / U
    assert np.abs(err).max() <= 6.1, np.abs(err).max()
    assert abs(err.mean()) <= 0.25, err.mean()


def test_the_largest_fp32_numbers_and_infinities_keep_their_place():
    """The type's largest and lowest numbers in K and V; an infinity stays one, and a NaN.

    The mean of 8: sums cut off and rounded under 20 times and a division, 32 u.  The last score: 3 u of dropped
    products, 3 roundings, the two constants (0.3 u)."""
    d, n = 64, 8
    big = float(torch.finfo(torch.float32).max)
    K, V = torch.zeros(1, n, 1, d, device="cuda"), torch.ones(1, n, 1, d, device="cuda")
    Q = torch.zeros(1, 1, 1, d, device="cuda")
    Q[..., 0] = 1.0
    V[0, 3, 0, :6] = torch.tensor([big, -big, float("inf"), -float("inf"), float("nan"), 3.3953e38], device="cuda")
    lens = torch.full((1,), n, dtype=torch.int32, device="cuda")
    O, _ = clsa.window_attn(Q, K, V, lens, n, scale=1.0)
    got, want = O[0, 0, 0].double(), V[0, :, 0].double().mean(0)
    assert torch.isinf(got[2]) and got[2] > 0 and torch.isinf(got[3]) and got[3] < 0 and torch.isnan(got[4])
    for i in (0, 1, 5, 6, 63):
        assert abs(got[i] - want[i]) <= 32 * U * abs(want[i]), i
    K[0, 5, 0, 0] = -big                                 # its weight is 0
    O, lse = clsa.window_attn(Q, K, V, lens, n, scale=1.0)
    keep = torch.tensor([0, 1, 2, 3, 4, 6, 7], device="cuda")
    assert abs(float(lse) - np.log(7)) <= 16 * U
    assert abs(float(O[0, 0, 0, 0]) - float(V[0, keep, 0, 0].double().mean())) <= 32 * U * big / 7
    K[0, 5, 0, 0] = big                                  # all the weight
    V[0, 3] = 1.0
    V[0, 5] = 2.0
    O, lse = clsa.window_attn(Q * 1e-3, K, V, lens, n, scale=1.0)
    assert abs(float(lse) / (big * float(np.float32(1e-3))) - 1) <= 8 * U and bool((O == 2.0).all())


@pytest.mark.parametrize("d", [64, 128])
def test_sums_over_the_8bit_cache_do_not_drift(d):
    """3000 tokens a row, a warp a row: weights and values of all sizes, so that products fill the sum's 24 bits.
    A sum that the tensor core carries over all tiles is cut off 376 times, always towards zero: 130 u low on
    the average (119 to 142 over 64 rows of such numbers, summed so on the host).  Rounded additions leave
    each output within a few u either way (sqrt(188) half steps), and the mean of many within 32 u."""
    g = np.random.default_rng(d)
    W, B, G = 3000, 900, 8
    cache = clsa.Kv8Cache.empty(1, W, 1, d, 16)
    cache.V8.copy_(dev(2.0 ** g.integers(-3, 3, (1, W, 1, d)) * (1 + g.integers(0, 8, (1, W, 1, d)) / 8)).to(cache.V8.dtype))
    cache.K8.copy_(dev(g.standard_normal((1, W, 1, d))).to(cache.K8.dtype))
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    Q = dev(g.standard_normal((1, B, G, d)) * 0.7)
    O, _ = clsa.kv8_attn(Q, cache, torch.full((B,), W, dtype=torch.int32, device="cuda"))
    K, V = cache.K8[0, :, 0].double(), cache.V8[0, :, 0].double()
    s = Q[0, :64].double() @ K.T * d ** -0.5
    want = torch.softmax(s, -1) @ V
    err = ((O[0, :64].double() - want) / want / U).cpu().numpy()
    assert abs(err.mean()) <= 32, err.mean()
    assert np.abs(err.mean(-1)).max() <= 64, np.abs(err.mean(-1)).max()  # row by row
