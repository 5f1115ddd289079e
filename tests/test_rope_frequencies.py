"""The rotary frequencies when not all of their arguments are given (host arithmetic)."""
import math

import numpy as np
import pytest

import long_context_prefill_trianglemix_b200 as tm
from long_context_prefill_trianglemix_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_lib()
    yield


@pytest.mark.parametrize("rot,base,factor", [(128, 500000.0, 8.0), (64, 10000.0, 4.0), (6, 10000.0, 1.5)])
def test_a_factor_alone_slows_every_pair(rot, base, factor):
    f = base ** (-np.arange(0, rot, 2) / rot)
    np.testing.assert_allclose(tm.tm_rope_inv_freq(rot, base), f, rtol=1e-15)
    np.testing.assert_allclose(tm.tm_rope_inv_freq(rot, base, factor), f / factor, rtol=1e-15)
    np.testing.assert_allclose(tm.tm_rope_inv_freq(rot, base, factor, 8192.0), f / factor, rtol=1e-15)


def test_one_number_of_turns_is_a_step():
    rot, base, trained, turns = 64, 10000.0, 4096.0, 3.0
    f = base ** (-np.arange(0, rot, 2) / rot)
    want = np.where(trained * f / (2 * math.pi) > turns, f, f / 4.0)
    assert 0 < (want == f).sum() < rot // 2
    np.testing.assert_allclose(tm.tm_rope_inv_freq(rot, base, 4.0, trained, turns), want, rtol=1e-14)
    with pytest.raises(tm.TmError):
        tm.tm_rope_inv_freq(rot, base, 4.0, trained, high_turns=turns)
