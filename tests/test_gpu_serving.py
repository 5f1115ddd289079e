"""A prompt and its decode as a serving program runs them, q, k and v out of packed
projections all the way, with every stage compared with its definition on the
library's own inputs to that stage: rotations, prefill, key weights, selection, stored
codes, attention, the weights it adds and the compacted cache."""
import math

import numpy as np
import pytest

import cache_ref as ref
import long_context_prefill_trianglemix_b200 as tm
import oracle
from gpu_util import assert_close, from_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from long_context_prefill_trianglemix_b200 import build
    build.build_lib()
    oracle.build()
    yield
    assert tm.tm_get_device_status() == tm.TM_OK


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def num(t):
    return t.float().double().cpu().numpy()


class Model:
    def __init__(self, B, Hq, H, D, seed):
        import torch
        self.B, self.Hq, self.H, self.D = B, Hq, H, D
        self.g = torch.Generator().manual_seed(seed)
        self.f = tm.tm_rope_inv_freq(D, 500000.0, 4.0, 128.0, 1.0, 4.0)
        self.df = torch.from_numpy(self.f).cuda()

    def project(self, N):
        """q, k, v of N tokens a sequence, views of one packed buffer."""
        import torch
        B, Hq, H, D = self.B, self.Hq, self.H, self.D
        x = torch.randn((B, N, (Hq + 2 * H) * D), generator=self.g).to(torch.bfloat16).cuda()
        return [t.view(B, N, -1, D) for t in x.split([Hq * D, H * D, H * D], -1)]

    def rotate(self, q, k, pos):
        """By the raw call with the tensors' own strides; against the definition."""
        import torch
        B, N = q.shape[:2]
        qo, ko = (torch.full(t.shape, float("nan"), dtype=t.dtype, device="cuda") for t in (q, k))
        dp = torch.tensor(pos, dtype=torch.int32, device="cuda")
        tm.tm_rope_fwd(q, qo, k, ko, B, N, self.Hq, self.H, self.D, q.stride(1), qo.stride(1), k.stride(1),
                       ko.stride(1), self.D, 0, 0, self.df, 1.0, dp, 0)
        for x, y in ((q, qo), (k, ko)):
            want = ref.rope(num(x), pos, self.f, self.D, 0)
            assert (np.abs(num(y) - want) <= np.abs(want) * 2.0 ** -8 + np.abs(num(x)).max() * 2.0 ** -20).all()
        return qo, ko


def image(cache):
    return [num(t) for t in cache]


def append(cache, fmt, k, v, lens, table, counts=None, index=None):
    """By the raw call; codes and ranges bit for bit."""
    B, n_src, H, D = k.shape
    n = n_src if index is None else index.shape[2]
    k8, v8, kr, vr = image(cache)
    cnt = [n] * B if counts is None else counts.tolist()
    idx = None if index is None else index.cpu().numpy()
    wk = ref.append(num(k), lens.tolist(), cnt, table.cpu().numpy(), k8, kr, fmt, idx)
    wv = ref.append(num(v), lens.tolist(), cnt, table.cpu().numpy(), v8, vr, fmt, idx)
    tm.tm_kv8_append(k, v, k.stride(1), v.stride(1), B, n_src, n, H, D, counts, index, lens, table,
                     table.shape[1], *cache, cache.k8.shape[0], cache.k8.shape[2], fmt)
    for got, want in zip(image(cache), (wk[0], wv[0], wk[1], wv[1])):
        np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("fmt,D,page", [(ref.INT8, 128, 16), (ref.E4M3, 64, 32)])
def test_a_prompt_and_its_decode(fmt, D, page):
    import torch
    B, Hq, H, N, keep, S, W, L = 3, 8, 2, 300, 64, 4, 128, 32
    m = Model(B, Hq, H, D, 200 + D)
    pages, mp = 60, 160 // page
    free = torch.randperm(pages, generator=m.g).to(torch.int32)
    table = free[: B * mp].view(B, mp).cuda()
    cache = tm.Kv8Cache.empty(pages, H, page, D, fmt)
    scale = D ** -0.5

    q, k, v = m.project(N)
    q, k = m.rotate(q, k, np.arange(N)[None].repeat(B, 0))
    o = tm.triangle_attention(q, k, v.contiguous(), S, W, L)
    want = oracle.attention(bits(q), bits(k), bits(v), B, Hq, H, N, D, scale, 0, S, W, L)
    assert_close(from_dev(o), want, "prefill")
    w = tm.key_weights(q, k, L)
    ww, bw = ref.key_weights(num(q), num(k), scale, L, [N] * B)
    assert (np.abs(w.double().cpu().numpy() - ww) <= bw).all()
    index, kept = tm.kv_select(w, keep, 4, 16)
    for b in range(B):
        for h in range(H):
            assert index[b, h].tolist() == ref.select(w[b, h].cpu().numpy(), N, keep, 4, 16)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    append(cache, fmt, k, v, zero, table, kept, index)
    lens, acc = kept.clone(), torch.zeros((B, H, mp * page), device="cuda")
    acc[..., :keep] = w.gather(2, index.long())

    def decode(step, nq, table, lens, acc):
        q, k, v = m.project(nq)
        q, k = m.rotate(q, k, N + step + np.arange(nq)[None].repeat(B, 0))
        append(cache, fmt, k, v, lens, table)
        lens = lens + nq
        before = acc.double().cpu().numpy()
        out = tm.kv8_attention(cache, q, lens, table, weights=acc, accumulate=True)
        k8, v8, kr, vr = image(cache)
        want, bound, ww, bw = ref.attention(num(q), k8, v8, kr, vr, table.cpu().numpy(), lens.tolist(),
                                            scale, fmt)
        assert (np.abs(num(out) - want) <= bound).all()
        after = acc.double().cpu().numpy()
        assert (np.abs(after - before - ww) <= bw + np.abs(after) * 2.0 ** -23).all()
        return lens

    step = 0
    for nq in (1, 1, 3, 1):
        lens = decode(step, nq, table, lens, acc)
        step += nq
    # the cache shrinks
    less = 40
    index, kept = tm.kv_select(acc, less, 4, 8, lens)
    new_table = torch.full((B, mp), -1, dtype=torch.int32)
    blocks = math.ceil((less + 8) / page)
    new_table[:, :blocks] = free[B * mp: B * (mp + blocks)].view(B, blocks)
    new_table = new_table.cuda()
    new_acc = torch.zeros_like(acc)
    k8, v8, kr, vr = image(cache)
    args = index.cpu().numpy(), kept.tolist(), lens.tolist(), table.cpu().numpy(), new_table.cpu().numpy()
    wk, wv = ref.compact(*args, k8, kr, fmt), ref.compact(*args, v8, vr, fmt)
    tm.kv8_compact(cache, index, kept, lens, table, new_table, acc, new_acc)
    for got, want in zip(image(cache), (wk[0], wv[0], wk[1], wv[1])):
        np.testing.assert_array_equal(got, want)
    assert torch.equal(new_acc[..., :less], acc.gather(2, index.long()))
    lens = kept.clone()
    for nq in (1, 2, 1):
        lens = decode(step, nq, new_table, lens, new_acc)
        step += nq
    assert lens.tolist() == [less + 4] * B
