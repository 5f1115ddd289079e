"""The cache attention where its arithmetic could lose what fp32 holds: ranges of V that
differ within a sequence, and values near the type's largest. Every bound is counted per
key: the mass sum_j p_j |v_j| carries the rounding of the weights, so an error that only
the largest |v| would excuse fails."""
import math

import numpy as np
import pytest

import cache_ref as ref
import long_context_prefill_trianglemix_b200 as tm
from test_gpu_kv8 import Cache, ints, rand

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


@pytest.mark.parametrize("fmt,D,nq", [(ref.INT8, 64, 1), (ref.E4M3, 64, 1), (ref.INT8, 128, 1),
                                      (ref.E4M3, 128, 3), (ref.INT8, 64, 4)])
def test_small_weights_beside_a_larger_range(fmt, D, nq):
    """Of every 64 keys one takes nearly all the weight and has v = 0, 47 have 2^-19.5 of it, and
    16 on a page whose V range is 2^9 times theirs have 2^-31: o is what the 47 give. K holds the
    logarithms of the weights in column 0, q is that column's unit, so scores are exact but for
    the scale (|s| 2^-20, and 2^-21 for 2^x). Bound: bf16's half step 2^-8 of o; fp16's half step
    2^-11 of each weight and the scores' error, of the mass."""
    import torch
    B, G, page, tokens = 96, 4, 16, 8192
    pages = tokens // page
    quiet, faint, one = {ref.INT8: (-78, -125, 127.0), ref.E4M3: (-80, -128, 448.0)}[fmt]
    unit = -19.5 / quiet                                      # log2 of a weight a code
    g = torch.Generator().manual_seed(D)
    k = torch.zeros((pages, 1, page, D))
    k[..., 0] = quiet
    k[::4, :, 0, 0] = 0
    k[3::4, ..., 0] = faint
    v = torch.randint(4, 8, (pages, 1, page, D), generator=g) * 16.0  # 64 .. 112, exact in both formats
    v[::4, :, 0] = 0
    vr = torch.full((pages, 1), one)
    vr[3::4] = one * 512
    dtype = torch.int8 if fmt == ref.INT8 else torch.float8_e4m3fn
    c = tm.Kv8Cache(k.to(dtype).cuda(), v.to(dtype).cuda(), torch.full((pages, 1), one, device="cuda"), vr.cuda())
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    q = torch.zeros((B, nq, G, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = unit * math.log(2.0)
    got = tm.kv8_attention(c, q, ints([tokens] * B), table, scale=scale).double().cpu().numpy()
    kk, vv = k[..., 0].double().numpy().reshape(-1), (v * vr[:, :, None, None] / one).double().numpy().reshape(-1, D)
    s = np.float64(np.float32(scale)) * kk
    for i in range(nq):
        n = tokens - nq + i + 1
        p = np.exp(s[:n])
        p /= p.sum()
        want, mass = p @ vv[:n], p @ np.abs(vv[:n])
        bound = want * 2.0 ** -8 + mass * (2.0 ** -11 + 2 * (np.abs(s).max() * 2.0 ** -20 + 2.0 ** -21))
        err = np.abs(got[:, i] - want)
        assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("nq", [1, 3])
def test_values_near_the_largest(fmt, nq):
    """V of 2^120 to 2^126: o is finite and as precise as for V of ordinary size (its bits are the
    same but for the exponent), in items of one warp, of one CTA and cut between CTAs."""
    import torch
    cache = Cache(130, 6, 2, 128, 64, fmt, 70)
    q, lens = rand((6, nq, 8, 128), 131, 1.5), ints([4480, 1, 63, 64, 65, 1999])
    cache.vr.copy_(2.0 ** torch.randint(-3, 2, cache.vr.shape, device="cuda").float())
    want = cache.attend(q, lens)
    cache.vr.mul_(2.0 ** 125)
    got = cache.attend(q, lens)
    assert torch.isfinite(got).all()
    assert torch.equal(got.double() * 2.0 ** -125, want.double())
