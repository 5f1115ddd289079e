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


@pytest.mark.parametrize("fmt,D,Hq,H,nq", [(ref.INT8, 64, 4, 1, 1), (ref.E4M3, 64, 8, 2, 1),
                                           (ref.INT8, 128, 12, 1, 1), (ref.E4M3, 128, 4, 1, 8)])
@pytest.mark.parametrize("tokens", [2, 48, 4096])
def test_weights_of_a_sum_that_cancels(fmt, D, Hq, H, nq, tokens):
    """Keys in turn of weight 1 and (1 + 2^-8) / 2, whose values nearly cancel: o is a small part
    of the mass, so its own rounding hides nothing. fp16 holds the second weight (2^-11 of it at
    most); a format of 8 bits would be off by 2^-8 of half the mass, nearly four times the bound."""
    import torch
    B, page = 3, 16
    pages = -(-tokens // page)
    c1, one, v0, v1 = {ref.INT8: (-127, 127.0, 64, 127), ref.E4M3: (-128, 448.0, 64, 128)}[fmt]
    unit = math.log2((1 + 2.0 ** -8) / 2) / c1               # log2 of a weight a code
    k = torch.zeros((pages, H, page, D))
    k[:, :, 1::2, 0] = c1
    v = torch.full((pages, H, page, D), float(v0))
    v[:, :, 1::2] = -float(v1)
    dtype = torch.int8 if fmt == ref.INT8 else torch.float8_e4m3fn
    r = torch.full((pages, H), one, device="cuda")
    c = tm.Kv8Cache(k.to(dtype).cuda(), v.to(dtype).cuda(), r, r.clone())
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    q = torch.zeros((B, nq, Hq, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = unit * math.log(2.0)
    w = torch.zeros((B, H, pages * page), device="cuda")
    got = tm.kv8_attention(c, q, ints([tokens] * B), table, scale=scale, weights=w).double().cpu().numpy()
    s = np.float64(np.float32(scale)) * np.where(np.arange(tokens) % 2, float(c1), 0.0)
    vv = np.where(np.arange(tokens) % 2, -float(v1), float(v0))
    # a score: |s| 2^-20; 2^x: 2^-21; the fp32 sum of the weights: 2^-24 for each of its additions,
    # which 32 lanes and more share
    off = 2 * (np.abs(s).max() * 2.0 ** -20 + 2.0 ** -21) + (tokens / 32 + 32) * 2.0 ** -24
    want_w = np.zeros(tokens)
    for i in range(nq):
        n = tokens - nq + i + 1
        if n <= 0:
            assert (got[:, i] == 0).all()
            continue
        p = np.exp(s[:n])
        p /= p.sum()
        want_w[:n] += p * (Hq // H)
        want, mass = p @ vv[:n], p @ np.abs(vv[:n])
        assert n == 1 or n % 2 or abs(want) * 2.0 ** -8 < mass * 2.0 ** -13
        assert (np.abs(got[:, i] - want) <= abs(want) * 2.0 ** -8 + mass * (2.0 ** -11 + off)).all()
    # the weights of the keys are fp32 throughout: nothing of the order of 2^-11
    bound = want_w * (off + 2.0 ** -20)
    assert (np.abs(w.double().cpu().numpy()[..., :tokens] - want_w) <= bound).all()


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("page,D,Hq,H,nq", [(16, 64, 4, 1, 1), (16, 128, 7, 1, 1), (64, 128, 8, 2, 2),
                                            (32, 64, 24, 2, 3), (128, 128, 16, 1, 1)])
def test_attention_within_a_bound_of_each_key(fmt, page, D, Hq, H, nq):
    """As the tests of test_gpu_kv8.py, with every key's own share: a score is a chain of D / 16
    products of 16 terms and at most 4 additions besides, each off by 2^-23 of sum_d |q_d k_d|
    (and 2^-22 of the score for its scalings), which moves o by p_j |v_j - o| of it."""
    mp = max(2, 640 // page)
    lens = [mp * page, 1, 17, mp * page - 5]
    cache = Cache(140 + page + D, 4, H, D, page, fmt, mp)
    q, scale = rand((4, nq, Hq, D), 141, 1.5), 1 / math.sqrt(D)
    import torch
    w = torch.full((4, H, mp * page), -3.0, device="cuda")
    got = cache.attend(q, ints(lens), w).double().cpu().numpy()
    w = w.double().cpu().numpy()
    kc, vc, kr, vr = cache.image()
    table, qq = cache.table.cpu().numpy(), q.double().cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(H):
            k, _ = ref.values(kc, kr, table, b, h, n, fmt)
            v, _ = ref.values(vc, vr, table, b, h, n, fmt)
            ww, bw = np.zeros(n), np.zeros(n)
            for i in range(max(0, nq - n), nq):
                m = n - nq + i + 1
                for x in range(h * (Hq // H), (h + 1) * (Hq // H)):
                    s = k[:m] @ qq[b, i, x] * scale
                    off = (np.abs(k[:m]) @ np.abs(qq[b, i, x]) * scale * (D / 16 + 4) * 2.0 ** -23
                           + np.abs(s) * 2.0 ** -22 + 2.0 ** -21)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o = p @ v[:m]
                    bound = (np.abs(o) * 2.0 ** -8 + p @ np.abs(v[:m]) * (2.0 ** -11 + m * 2.0 ** -24)
                             + (p * off) @ np.abs(v[:m] - o) * 1.01)
                    assert (np.abs(got[b, i, x] - o) <= bound).all()
                    ww[:m] += p
                    bw[:m] += p * (off + p @ off + m * 2.0 ** -24 + 2.0 ** -20) * 1.01
            assert (np.abs(w[b, h, :n] - ww) <= bw).all()
