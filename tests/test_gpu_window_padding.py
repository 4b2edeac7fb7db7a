"""Window attention's padding rows (seq_lens[b] < T): they see nothing, so O = 0 and lse = -inf, whatever the
bytes of the tokens that other rows of the call see."""
import numpy as np
import pytest
import torch

from long_context_sparse_clsa_b200 import clsa
from test_gpu_cache import DT, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_sparse_clsa_b200.build import build
    build()
    clsa.load_library()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,n,Hq,Hkv,d", [
    (3, 4, 60, 4, 1, 128),      # a CTA a unit
    (2, 7, 60, 6, 3, 64),
    (200, 4, 300, 8, 2, 64),    # a warp a unit
    (90, 16, 100, 2, 2, 128),
    (2, 150, 300, 8, 2, 128),   # row tiles (bf16)
    (1, 400, 410, 8, 2, 64)])
def test_padding_rows_are_zero_beside_values_that_are_not_finite(value, dtype, B, T, n, Hq, Hkv, d):
    g = np.random.default_rng(T)
    Q = dev(g.standard_normal((B, T, Hq, d)), DT[dtype])
    K, V = (dev(g.standard_normal((B, n, Hkv, d)), DT[dtype]) for _ in range(2))
    V[:, 0] = value                                    # every row that sees anything sees token 0
    lens = g.integers(1, T, B)
    lens[0], lens[-1] = T - 1, T // 2
    O, lse = clsa.window_attn(Q, K, V, dev(lens, torch.int32), n)
    for b in range(B):
        pad = T - int(lens[b])
        assert not O[b, :pad].isnan().any() and not O[b, :pad].any(), b
        assert torch.isneginf(lse[b, :pad]).all() and torch.isfinite(lse[b, pad:]).all()
        assert not torch.isfinite(O[b, pad:]).any()    # the others' sums are as the values are
