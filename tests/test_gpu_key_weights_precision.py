"""Key weights held to fp32: scores of one exact product, so that what is left is the
arithmetic of the softmax and its sums."""
import math

import numpy as np
import pytest

import long_context_prefill_trianglemix_b200 as tm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_prefill_trianglemix_b200 import build
    build.build_lib()
    yield
    assert tm.tm_get_device_status() == tm.TM_OK


@pytest.mark.parametrize("N,Hq,H,D,L", [(1, 1, 1, 64, 1), (200, 1, 1, 64, 1), (200, 7, 1, 128, 1),
                                        (1000, 4, 2, 128, 3), (1500, 28, 4, 64, 40), (700, 8, 2, 128, 256),
                                        (6000, 8, 8, 64, 100)])
def test_each_weight_to_fp32(N, Hq, H, D, L):
    """q is the first column's unit, k_j its score: p_ij = e^k_j / sum_(j' <= i) e^k_j'. Relative
    error of a weight: 2^-21 for 2^x and the scale; the log-sum-exp, below 2^5, by 2 steps of
    2^-19 (its logarithm and its sum with the maximum) times ln 2; the additions, 2^-24 each: a
    row's sum has a chain of at most 10 a tile of 128 keys in each of 4 accumulators and 4 for each
    tile, a key's sum the same over its rows. Exponentials or weights in fp16 are off by up to
    2^-11."""
    import torch
    g = torch.Generator().manual_seed(N + D)
    s = (torch.rand((2, N, H), generator=g) * 6 - 3).to(torch.bfloat16)
    q = torch.zeros((2, N, Hq, D), dtype=torch.bfloat16)
    q[..., 0] = 1.0
    k = torch.zeros((2, N, H, D), dtype=torch.bfloat16)
    k[..., 0] = s
    got = tm.key_weights(q.cuda(), k.cuda(), L, scale=1.0).double().cpu().numpy()
    e = np.exp(s.double().numpy())
    rows = np.arange(max(0, N - L), N)
    total = np.cumsum(e, 1)[:, rows]                                    # [2, rows, H]
    seen = np.arange(N)[None] <= rows[:, None]
    want = np.einsum("bnh,brh,rn->bhn", e, 1 / total, seen.astype(float)) * (Hq // H)
    adds = 24 * (-(-N // 128) + -(-L * (Hq // H) // 128) + 4)
    bound = want * (2.0 ** -21 + 2 * math.log(2) * 2.0 ** -19 + adds * 2.0 ** -24)
    assert bound.max() <= want.max() * 2.0 ** -13
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / want).max()
