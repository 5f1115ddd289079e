"""The inverse rotation against its definition, in both layouts, in and out of place,
by both kernels (rot a multiple of 16 and not), and on a packed buffer."""
import numpy as np
import pytest

import long_context_prefill_trianglemix_b200 as tm
from test_gpu_rope import check, make

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


@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot", [(3, 1, 32, 8, 128, 128), (2, 77, 28, 4, 64, 32),
                                              (1, 33, 3, 1, 64, 2), (2, 19, 4, 4, 128, 6),
                                              (1, 130, 7, 1, 128, 80), (1, 4, 4, 2, 128, 126)])
@pytest.mark.parametrize("layout", [0, 1])
def test_inverse_matches_its_definition(B, N, Hq, Hkv, D, rot, layout):
    import torch
    q, k = make((B, N, Hq, D), 21), make((B, N, Hkv, D), 22)
    f = tm.tm_rope_inv_freq(rot, 500000.0)
    df = torch.from_numpy(f).cuda()
    pos = np.random.default_rng(23).integers(-5, 2_000_000, (B, N)).astype(np.int32)
    dp = torch.from_numpy(pos).cuda()
    qo, ko = tm.rope(q, k, df, dp, rot=rot, interleaved=layout, mscale=1.25, inverse=True)
    check(qo, q, pos, f, rot, layout, 1.25, inverse=True)
    check(ko, k, pos, f, rot, layout, 1.25, inverse=True)
    q2, k2 = q.clone(), k.clone()
    tm.rope(q2, k2, df, dp, rot=rot, interleaved=layout, mscale=1.25, inverse=True, out=(q2, k2))
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    assert torch.equal(qo[..., rot:], q[..., rot:])


@pytest.mark.parametrize("rot,layout", [(64, 0), (64, 1), (6, 0), (6, 1)])
def test_inverse_at_far_positions(rot, layout):
    """first beyond 32 bits: there and back gives the input, to two roundings of bf16 (2^-8 of
    the pair's length each)."""
    import torch
    x = make((1, 9, 3, 64), 24)
    df = torch.from_numpy(tm.tm_rope_inv_freq(rot, 10000.0)).cuda()
    first = 2 ** 45 + 7
    y, _ = tm.rope(x, None, df, first=first, rot=rot, interleaved=layout)
    z, _ = tm.rope(y, None, df, first=first, rot=rot, interleaved=layout, inverse=True)
    assert not torch.equal(y, x)
    a = x.double()[..., :rot]
    a = a.unflatten(-1, (-1, 2)).norm(dim=-1) if layout else a.unflatten(-1, (2, -1)).norm(dim=-2)
    length = (a.repeat_interleave(2, -1) if layout else torch.cat((a, a), -1)) * 2.0 ** -6
    assert ((z - x).double().abs()[..., :rot] <= length).all()
    assert torch.equal(z[..., rot:], x[..., rot:])
