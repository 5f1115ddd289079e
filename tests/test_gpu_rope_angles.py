"""Rotary angles at any position that the call takes, against exact arithmetic: pos * f
is a rational number, reduced by 2 pi to 70 digits before its cosine is taken."""
from fractions import Fraction

import math

import numpy as np
import pytest

import long_context_prefill_trianglemix_b200 as tm

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Fraction("3.1415926535897932384626433832795028841971693993751058209749445923078164")


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_prefill_trianglemix_b200 import build
    build.build_lib()
    yield
    assert tm.tm_get_device_status() == tm.TM_OK


def turned(pos, f):
    """(cos, sin) of pos * f for every pos and f."""
    t = np.array([[float(Fraction(int(p)) * Fraction(float(x)) % TWO_PI) for x in f] for p in pos])
    return np.cos(t), np.sin(t)


@pytest.mark.parametrize("first", [0, 10 ** 6, 2 ** 31 - 8, -2 ** 31, 2 ** 40 + 12345, -2 ** 47 - 1,
                                   2 ** 52 - 3, -2 ** 52 + 5])
@pytest.mark.parametrize("rot,layout", [(128, 0), (128, 1), (126, 0), (6, 1)])
def test_angles_at_far_positions(first, rot, layout):
    """Rows of ones and zeros, so that the outputs are cosines and sines. Bound: bf16's half step
    (2^-8 of the value) and 2^-20 for the angle (2^-23 of a turn is 2^-20.3) with the fp32 sine's
    2^-23."""
    import torch
    N, D = 4, 128
    f = tm.tm_rope_inv_freq(rot, 500000.0)
    x = torch.zeros((1, N, 1, D), dtype=torch.bfloat16, device="cuda")
    a = slice(0, rot, 2) if layout else slice(0, rot // 2)
    b = slice(1, rot, 2) if layout else slice(rot // 2, rot)
    x[..., a] = 1.0
    o = torch.empty_like(x)
    tm.tm_rope_fwd(x, o, None, None, 1, N, 1, 0, D, D, D, 0, 0, rot, layout, 0,
                   torch.from_numpy(f).cuda(), 1.0, None, first)
    c, s = turned(range(first, first + N), f)
    y = o[0, :, 0].double().cpu().numpy()
    for got, want in ((y[:, a], c), (y[:, b], s)):
        assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -20).all(), np.abs(got - want).max()
    assert (y[:, rot:] == 0).all() and math.isfinite(y.sum())
