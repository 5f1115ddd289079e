"""One token a sequence, out of the packed projection that a decode step has: the
sequences' rows lie one packed row apart, and a tensor of one token has no stride
between tokens (torch reports the heads' width there)."""
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


def packed(B, Hq, Hkv, D, seed):
    """q, k, v as views of one [B, 1, (Hq + 2 Hkv) D] buffer."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn((B, 1, (Hq + 2 * Hkv) * D), generator=g) * 2).to(torch.bfloat16).cuda()
    q, k, v = x.split([Hq * D, Hkv * D, Hkv * D], -1)
    return x, q.view(B, 1, Hq, D), k.view(B, 1, Hkv, D), v.view(B, 1, Hkv, D)


def check_rope(got, x, pos, f, rot, layout):
    """Half a step of bf16 (2^-8 of the value), and 2^-20 of the largest element for the fp32
    angle, sine and products."""
    x = x.double().cpu().numpy()
    want = ref.rope(x, pos, f, rot, layout)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= np.abs(want) * 2.0 ** -8 + np.abs(x).max() * 2.0 ** -20).all(), err.max()


@pytest.mark.parametrize("B,Hq,Hkv,D,rot", [(2, 4, 2, 64, 64), (64, 32, 8, 128, 128), (5, 7, 1, 128, 96),
                                            (3, 28, 4, 64, 6), (1, 8, 2, 128, 128)])
@pytest.mark.parametrize("layout", [0, 1])
def test_rope_of_one_token_a_sequence(B, Hq, Hkv, D, rot, layout):
    import torch
    x, q, k, _ = packed(B, Hq, Hkv, D, B)
    W = (Hq + 2 * Hkv) * D
    f = tm.tm_rope_inv_freq(rot, 500000.0)
    df = torch.from_numpy(f).cuda()
    pos = np.random.default_rng(B).integers(0, 131072, (B, 1)).astype(np.int32)
    dp = torch.from_numpy(pos).cuda()
    first = None
    for q_stride, k_stride in ((q.stride(1), k.stride(1)), (q.stride(0), k.stride(0)), (W, W)):
        if B == 1 and q_stride < Hq * D:
            continue
        qo = torch.full((B, 1, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        ko = torch.full((B, 1, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        tm.tm_rope_fwd(q, qo, k, ko, B, 1, Hq, Hkv, D, q_stride, qo.stride(1), k_stride, ko.stride(1),
                       rot, layout, 0, df, 1.0, dp, 0)
        check_rope(qo, q, pos, f, rot, layout)
        check_rope(ko, k, pos, f, rot, layout)
        first = (qo, ko) if first is None else first
        assert torch.equal(qo, first[0]) and torch.equal(ko, first[1])
    qo, ko = tm.rope(q, k, df, dp, rot=rot, interleaved=layout)
    assert torch.equal(qo, first[0]) and torch.equal(ko, first[1])
    # in place: every other column of the buffer keeps its bits
    y = x.clone()
    yq = y[..., :Hq * D].view(B, 1, Hq, D)
    yk = y[..., Hq * D:(Hq + Hkv) * D].view(B, 1, Hkv, D)
    tm.tm_rope_fwd(yq, yq, yk, yk, B, 1, Hq, Hkv, D, yq.stride(1), yq.stride(1), yk.stride(1),
                   yk.stride(1), rot, layout, 0, df, 1.0, dp, 0)
    assert torch.equal(yq, first[0]) and torch.equal(yk, first[1])
    assert torch.equal(y[..., (Hq + Hkv) * D:], x[..., (Hq + Hkv) * D:])


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("B,Hq,Hkv,D,page", [(2, 4, 2, 64, 16), (33, 32, 8, 128, 64), (5, 7, 1, 128, 32),
                                             (1, 8, 2, 64, 128)])
def test_append_of_one_token_a_sequence(B, Hq, Hkv, D, page, fmt):
    """k and v stay in the packed projection; codes and ranges bit for bit, twice in a row (the
    second token meets a block that holds the first)."""
    import torch
    shape, codes = (2 * B, Hkv, page, D), torch.int8 if fmt == ref.INT8 else torch.float8_e4m3fn
    table = torch.randperm(2 * B, generator=torch.Generator().manual_seed(B)).to(torch.int32)
    table = table.view(B, 2).cuda()
    start = np.random.default_rng(B).integers(0, 2 * page - 2, B)
    wk = wv = (np.zeros(shape), np.zeros(shape[:2]))
    caches = [tm.Kv8Cache.empty(2 * B, Hkv, page, D, fmt) for _ in range(4)]
    for step in range(2):
        _, _, k, v = packed(B, Hq, Hkv, D, 100 * B + step)
        lens, W = start + step, (Hq + 2 * Hkv) * D
        dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        args = [(k.double().cpu().numpy(), *wk), (v.double().cpu().numpy(), *wv)]
        wk, wv = (ref.append(x, lens, [1] * B, table.cpu().numpy(), c, r, fmt) for x, c, r in args)
        for c, strides in zip(caches, ((k.stride(1), v.stride(1)), (k.stride(0), v.stride(0)), (W, W), None)):
            if strides is None:
                tm.kv8_append(c, k, v, dl, table)
            else:
                if B == 1 and strides[0] < Hkv * D:
                    strides = W, W
                tm.tm_kv8_append(k, v, *strides, B, 1, 1, Hkv, D, None, None, dl, table, 2, *c, 2 * B,
                                 page, fmt)
            for got, want in ((c.k8, wk[0]), (c.v8, wv[0]), (c.k_range, wk[1]), (c.v_range, wv[1])):
                np.testing.assert_array_equal(got.float().cpu().numpy(), want)
            assert c.k8.dtype == codes
