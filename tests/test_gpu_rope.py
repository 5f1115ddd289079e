"""Rotary positions against the 64-bit rotation. Bound per value: bf16's half
step (2^-8 of the value) and 2^-21 of the pair's length for the fp32 angle,
sine and products."""
import numpy as np
import pytest

import cache_ref as ref
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


def make(shape, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * 2).to(torch.bfloat16).cuda()


def check(got, x, pos, f, rot, layout, mscale=1.0, inverse=False):
    x = x.double().cpu().numpy()
    want = ref.rope(x, pos, f, rot, layout, mscale, inverse)
    length = np.abs(x).max()
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= np.abs(want) * 2.0 ** -8 + length * mscale * 2.0 ** -20).all(), err.max()


CASES = [  # B, N, Hq, Hkv, D, rot
    (1, 1, 1, 1, 64, 64), (3, 1, 32, 8, 128, 128), (2, 77, 28, 4, 64, 32), (1, 130, 7, 1, 128, 64),
    (2, 19, 4, 4, 128, 6), (1, 33, 3, 1, 64, 2), (1, 9, 2, 2, 256, 48), (2, 5, 5, 0, 128, 128),
    (1, 600, 8, 2, 80, 80), (1, 4, 4, 2, 128, 126),
]


@pytest.mark.parametrize("B,N,Hq,Hkv,D,rot", CASES)
@pytest.mark.parametrize("layout", [0, 1])
def test_matches_the_rotation(B, N, Hq, Hkv, D, rot, layout):
    import torch
    q = make((B, N, Hq, D), 1)
    k = make((B, N, Hkv, D), 2) if Hkv else None
    f = tm.tm_rope_inv_freq(rot, 500000.0, 8.0, 8192.0, 1.0, 4.0)
    df = torch.from_numpy(f).cuda()
    rng = np.random.default_rng(3)
    for positions in (None, rng.integers(-5, 2_000_000, (B, N)).astype(np.int32)):
        pos = np.arange(40, 40 + N)[None].repeat(B, 0) if positions is None else positions
        dp = None if positions is None else torch.from_numpy(positions).cuda()
        qo = torch.full_like(q, float("nan"))
        ko = torch.full_like(k, float("nan")) if Hkv else None
        tm.tm_rope_fwd(q, qo, k, ko, B, N, Hq, Hkv, D, Hq * D, Hq * D, Hkv * D, Hkv * D, rot,
                       layout, 0, df, 1.25, dp, 40)
        check(qo, q, pos, f, rot, layout, 1.25)
        if Hkv:
            check(ko, k, pos, f, rot, layout, 1.25)
        # in place, the same bits
        q2, k2 = q.clone(), k.clone() if Hkv else None
        tm.tm_rope_fwd(q2, q2, k2, k2, B, N, Hq, Hkv, D, Hq * D, Hq * D, Hkv * D, Hkv * D, rot,
                       layout, 0, df, 1.25, dp, 40)
        same = q2[..., :rot].contiguous().view(torch.int16)
        assert torch.equal(same, qo[..., :rot].contiguous().view(torch.int16))
        assert torch.equal(q2[..., rot:], q[..., rot:])
        if Hkv:
            assert torch.equal(k2.view(torch.int16), ko.view(torch.int16))


@pytest.mark.parametrize("layout", [0, 1])
def test_packed_projection_in_place_and_out(layout):
    """q and k inside one [B, N, (Hq + 2 Hkv) D] buffer; v's columns stay as they are."""
    import torch
    B, N, Hq, Hkv, D, rot = 2, 45, 8, 2, 128, 96
    W = (Hq + 2 * Hkv) * D
    x = make((B, N, W), 5)
    f = tm.tm_rope_inv_freq(rot, 10000.0)
    df = torch.from_numpy(f).cuda()
    pos = np.arange(7, 7 + N)[None].repeat(B, 0)
    q = x[..., :Hq * D].unflatten(-1, (Hq, D))
    k = x[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
    qo = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    ko = torch.empty((B, N, Hkv, D), dtype=torch.bfloat16, device="cuda")
    tm.tm_rope_fwd(q, qo, k, ko, B, N, Hq, Hkv, D, W, Hq * D, W, Hkv * D, rot, layout, 0, df, 1.0,
                   None, 7)
    check(qo, q, pos, f, rot, layout)
    check(ko, k, pos, f, rot, layout)
    y = x.clone()
    yq, yk = y[..., :Hq * D], y[..., Hq * D:]
    tm.tm_rope_fwd(yq, yq, yk, yk, B, N, Hq, Hkv, D, W, W, W, W, rot, layout, 0, df, 1.0, None, 7)
    assert torch.equal(y[..., :Hq * D], qo.flatten(2))
    assert torch.equal(y[..., Hq * D:(Hq + Hkv) * D], ko.flatten(2))
    assert torch.equal(y[..., (Hq + Hkv) * D:], x[..., (Hq + Hkv) * D:])


def test_inverse_is_the_transpose():
    """<rope(x), y> = <x, rope^T(y)>: the gradient of a rotation is the inverse call.
    Each product differs by bf16's rounding of its rotated factor, 2^-8 of it."""
    import torch
    B, N, H, D = 1, 64, 2, 64
    x, y = make((B, N, H, D), 8), make((B, N, H, D), 9)
    df = torch.from_numpy(tm.tm_rope_inv_freq(D, 10000.0)).cuda()
    outs = []
    for src, inv in ((x, 0), (y, 1)):
        o = torch.empty_like(src)
        tm.tm_rope_fwd(src, o, None, None, B, N, H, 0, D, H * D, H * D, 0, 0, D, 0, inv, df, 1.0,
                       None, 100000)
        outs.append(o.double())
    a, b = (outs[0] * y.double()), (x.double() * outs[1])
    assert abs(a.sum() - b.sum()) <= (a.abs().sum() + b.abs().sum()) * 2.0 ** -8


def test_far_positions_keep_their_angles():
    """At two million positions the fastest pair has turned 300,000 times."""
    import torch
    B, N, D = 1, 8, 128
    q = torch.zeros((B, N, 1, D), dtype=torch.bfloat16, device="cuda")
    q[..., :64] = 1.0
    f = tm.tm_rope_inv_freq(D, 500000.0)
    p = np.array([[0, 1, 4095, 131071, 1_000_003, 1_999_999, 2 ** 31 - 1, -2 ** 31]], np.int32)
    o = torch.empty_like(q)
    tm.tm_rope_fwd(q, o, None, None, B, N, 1, 0, D, D, D, 0, 0, D, 0, 0,
                   torch.from_numpy(f).cuda(), 1.0, torch.from_numpy(p).cuda(), 0)
    check(o, q, p, f, D, 0)


def test_rows_past_32_bits():
    """q of more than 2^32 bytes: the last rows are right."""
    import torch
    N, H, D = 600_000, 32, 128
    q = torch.empty((1, N, H, D), dtype=torch.bfloat16, device="cuda")
    q[:, :3] = make((1, 3, H, D), 11)
    q[:, -3:] = make((1, 3, H, D), 12)
    keep = torch.cat((q[:, :3], q[:, -3:]), 1).clone()
    f = tm.tm_rope_inv_freq(D, 500000.0)
    tm.tm_rope_fwd(q, q, None, None, 1, N, H, 0, D, H * D, H * D, 0, 0, D, 0, 0,
                   torch.from_numpy(f).cuda(), 1.0, None, 0)
    pos = np.array([[0, 1, 2, N - 3, N - 2, N - 1]])
    check(torch.cat((q[:, :3], q[:, -3:]), 1), keep, pos, f, D, 0)
