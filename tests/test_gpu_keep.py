"""Key weights and key selection on the GPU, and a run of all the operators around
the attention as a serving program makes it."""
import math

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


def rand(shape, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def ints(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def weights_of(q, k, L, lens=None, out=None, accumulate=0, scale=None, stride=None):
    import torch
    B, N, Hq, D = q.shape
    H = k.shape[2]
    size = tm.tm_key_weights_workspace_size(B, Hq, H, N, D, L)
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((B, H, stride or N), -3.0, device="cuda") if out is None else out
    tm.tm_key_weights_fwd(q, k, B, Hq, H, N, D, scale or 1 / math.sqrt(D), L, lens, out,
                          out.shape[2], accumulate, ws, size)
    return out


CASES = [  # B, N, Hq, Hkv, D, L, lens
    (1, 1, 1, 1, 64, 1, None), (1, 127, 4, 1, 128, 1, None), (1, 128, 4, 4, 64, 128, None),
    (1, 129, 7, 1, 128, 40, None), (2, 300, 14, 2, 64, 300, None), (1, 1000, 8, 2, 128, 64, None),
    (3, 700, 4, 2, 128, 33, [700, 20, 257]), (4, 260, 28, 4, 64, 260, [0, 1, 131, 260]),
    (2, 515, 32, 2, 128, 9, [-4, 10 ** 9]), (1, 640, 24, 1, 64, 17, None), (1, 300, 128, 1, 64, 5, None),
    (1, 5000, 8, 2, 128, 100, None), (2, 2304, 3, 3, 64, 1000, [2304, 1111]),
]


@pytest.mark.parametrize("B,N,Hq,H,D,L,lens", CASES)
def test_key_weights_within_their_bound(B, N, Hq, H, D, L, lens):
    q, k = rand((B, N, Hq, D), 1, 1.5), rand((B, N, H, D), 2, 1.5)
    n = [N] * B if lens is None else [min(max(x, 0), N) for x in lens]
    for b in range(B):  # padding is never read as a key or a query
        q[b, n[b]:], k[b, n[b]:] = float("nan"), float("nan")
    import torch
    qz, kz = torch.nan_to_num(q), torch.nan_to_num(k)
    want, bound = ref.key_weights(qz.double().cpu().numpy(), kz.double().cpu().numpy(),
                                  1 / math.sqrt(D), L, n)
    got = weights_of(q, k, L, None if lens is None else ints(lens), stride=N + 3).double().cpu().numpy()
    for b in range(B):
        err = np.abs(got[b, :, :n[b]] - want[b, :, :n[b]])
        assert (err <= bound[b, :, :n[b]]).all(), (err - bound[b, :, :n[b]]).max()
        assert (got[b, :, n[b]:] == -3.0).all()
        total = min(L, n[b]) * (Hq // H)
        np.testing.assert_allclose(got[b, :, :n[b]].sum(-1), total if n[b] else 0, rtol=1e-4)


def test_key_weights_sharp_scores():
    """Scores of hundreds: one key takes nearly all of each row."""
    q, k = rand((1, 900, 8, 128), 3, 6.0), rand((1, 900, 2, 128), 4, 6.0)
    want, bound = ref.key_weights(q.double().cpu().numpy(), k.double().cpu().numpy(), 0.5, 50, [900])
    got = weights_of(q, k, 50, scale=0.5).double().cpu().numpy()
    assert (np.abs(got - want) <= bound).all()


def test_key_weights_add_up_and_repeat_to_the_bit():
    import torch
    q, k = rand((2, 3000, 8, 128), 5), rand((2, 3000, 2, 128), 6)
    a = weights_of(q, k, 77)
    assert torch.equal(a, weights_of(q, k, 77))
    start = torch.rand_like(a)
    b = weights_of(q, k, 77, out=start.clone(), accumulate=1)
    assert torch.equal(b, start + a)


def test_key_weights_propagate_a_nan():
    import torch
    q, k = rand((1, 256, 2, 64), 7), rand((1, 256, 2, 64), 8)
    k[0, 100, 0, 3] = float("nan")
    w = weights_of(q, k, 16)
    assert torch.isnan(w[0, 0]).all() and torch.isfinite(w[0, 1]).all()


def test_key_weights_captured():
    import torch
    q, k = rand((1, 1500, 8, 64), 9), rand((1, 1500, 2, 64), 10)
    want = weights_of(q, k, 50)
    size = tm.tm_key_weights_workspace_size(1, 8, 2, 1500, 64, 50)
    ws, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.zeros_like(want)
    lens = ints([1500])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tm.tm_key_weights_fwd(q, k, 1, 8, 2, 1500, 64, 0.125, 50, lens, out, 1500, 0, ws, size)
    g.replay()
    assert torch.equal(out, want)
    lens.copy_(ints([700]))
    out.fill_(-1)
    g.replay()
    assert torch.equal(out, weights_of(q, k, 50, lens, out=torch.full_like(out, -1)))


# ------------------------------------------------------------------------------ selection

def pick(w, lens, n, keep, sinks, recent, stride=None):
    import torch
    B, H = w.shape[:2]
    index = torch.full((B, H, keep), 77, dtype=torch.int32, device="cuda")
    kept = torch.full((B,), 77, dtype=torch.int32, device="cuda")
    tm.tm_kv_select(w, w.shape[2], lens, B, H, n, keep, sinks, recent, index, kept)
    return index.cpu().numpy(), kept.cpu().numpy()


@pytest.mark.parametrize("n,keep,sinks,recent", [
    (1, 1, 0, 0), (5, 8, 2, 3), (100, 1, 0, 0), (100, 10, 4, 6), (100, 99, 0, 1), (1000, 100, 0, 0),
    (4097, 600, 4, 64), (20000, 5000, 64, 256), (70001, 4096, 1, 0)])
def test_select_is_the_definition(n, keep, sinks, recent):
    import torch
    B, H = 3, 2
    g = torch.Generator().manual_seed(n)
    w = (torch.randn((B, H, n + 5), generator=g) * 3).exp()
    w[torch.rand(w.shape, generator=g) < 0.3] = 0.0
    w[0, 1] = torch.randint(0, 4, (n + 5,), generator=g).float()    # many ties
    w[1, 0] = 1.0                                                   # nothing but ties
    w[2, 0, ::7] = float("nan")
    w[2, 1, ::3], w[2, 1, 1::5], w[2, 1, 2::11] = float("inf"), -w[2, 1, 1::5], float("-inf")
    w[2, 1, 4::13] = -0.0
    lens = [n, max(1, n // 2), max(0, n - 3)]
    index, kept = pick(w.cuda(), ints(lens), n, keep, sinks, recent)
    for b in range(B):
        assert kept[b] == min(lens[b], keep)
        for h in range(H):
            want = ref.select(w[b, h, :lens[b]].numpy(), lens[b], keep, sinks, recent)
            assert index[b, h, :kept[b]].tolist() == want, (b, h)
            assert (index[b, h, kept[b]:] == -1).all()


def test_select_one_long_row_and_no_lens():
    import torch
    n, keep = 400_003, 9000
    g = torch.Generator().manual_seed(1)
    w = torch.rand((1, 1, n), generator=g)
    w[0, 0, ::17] = 0.5
    index, kept = pick(w.cuda(), None, n, keep, 5, 11)
    assert kept[0] == keep
    assert index[0, 0].tolist() == ref.select(w[0, 0].numpy(), n, keep, 5, 11)
    index, kept = pick(w.cuda(), ints([10 ** 9]), 1000, 10, 0, 0)
    assert index[0, 0].tolist() == ref.select(w[0, 0, :1000].numpy(), 1000, 10, 0, 0)


def test_select_many_rows_on_several_streams():
    import torch
    w = torch.rand((16, 8, 3000), device="cuda")
    want = pick(w, None, 3000, 100, 1, 2)[0]
    outs = []
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        out = torch.empty((16, 8, 100), dtype=torch.int32, device="cuda")
        tm.tm_kv_select(w, 3000, None, 16, 8, 3000, 100, 1, 2, out, None, s)
        outs.append(out)
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o.cpu().numpy(), want)


def test_positions_selection_and_compact_captured():
    """One graph of rotary positions, selection and compact, replayed on new inputs and lengths,
    against the calls themselves."""
    import torch
    B, H, D, page, mp, keep = 2, 2, 64, 16, 8, 24
    c = tm.Kv8Cache.empty(40, H, page, D)
    g = torch.Generator().manual_seed(3)
    c.k8.copy_(torch.randint(-127, 128, c.k8.shape, generator=g).to(torch.int8))
    c.v8.copy_(torch.randint(-127, 128, c.v8.shape, generator=g).to(torch.int8))
    c.k_range.copy_(torch.rand(40, H, generator=g).to(torch.bfloat16).float() + 1)
    c.v_range.copy_(torch.rand(40, H, generator=g).to(torch.bfloat16).float() + 1)
    pages = torch.randperm(40, generator=g).to(torch.int32)
    table, to = pages[:16].view(B, mp).cuda(), pages[16:20].view(B, 2).cuda()
    w, lens = torch.rand((B, H, 128), device="cuda"), ints([128, 60])
    index, kept = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, H, keep), (B,)))
    nw = torch.zeros((B, H, keep), device="cuda")
    q, f = rand((B, 5, 4, D), 92), torch.from_numpy(tm.tm_rope_inv_freq(D, 10000.0)).cuda()
    pos, out = ints(np.arange(10).reshape(2, 5)), torch.empty_like(q)

    def step():
        tm.rope(q, None, f, pos, out=(out, None))
        tm.tm_kv_select(w, 128, lens, B, H, 128, keep, 2, 5, index, kept)
        tm.kv8_compact(c, index, kept, lens, table, to, w, nw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, seed in (([128, 60], 1), ([17, 128], 2), ([0, 5], 3)):
        w.copy_(torch.rand(w.shape, generator=torch.Generator().manual_seed(seed)))
        lens.copy_(ints(n))
        q.copy_(rand(q.shape, 100 + seed))
        pos.copy_(pos * 3 + seed)
        graph.replay()
        got = [t.clone() for t in (out, index, kept, c.k8, c.v8, c.k_range, c.v_range, nw)]
        for t in (out, index, kept):
            t.fill_(-7)
        step()
        for a, b in zip(got, (out, index, kept, c.k8, c.v8, c.k_range, c.v_range, nw)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_a_prompt_and_its_decode_with_eviction(fmt):
    """Positions, triangle prefill, key weights, keep the heaviest, store them, decode with
    accumulated weights, shrink the cache, decode on. Every stage is compared with its
    definition on the library's own inputs to that stage."""
    import torch
    B, N, Hq, H, D, page, keep = 2, 500, 8, 2, 128, 16, 64
    W = (Hq + 2 * H) * D
    x = rand((B, N, W), 20)
    f = tm.tm_rope_inv_freq(D, 500000.0, 4.0, 128.0, 1.0, 4.0)
    df = torch.from_numpy(f).cuda()
    q = torch.empty((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")
    k = torch.empty((B, N, H, D), dtype=torch.bfloat16, device="cuda")
    tm.tm_rope_fwd(x, q, x[..., Hq * D:], k, B, N, Hq, H, D, W, Hq * D, W, H * D, D, 0, 0, df, 1.0,
                   None, 0)
    v = x[..., (Hq + H) * D:].unflatten(-1, (H, D))
    o = tm.triangle_attention(q, k, v.contiguous(), 4, 128, 32)
    assert torch.isfinite(o).all()
    w = weights_of(q, k, 32)
    index, kept = (torch.empty(s, dtype=torch.int32, device="cuda") for s in ((B, H, keep), (B,)))
    tm.tm_kv_select(w, N, None, B, H, N, keep, 4, 16, index, kept)
    wn = w.cpu().numpy()
    for b in range(B):
        for h in range(H):
            assert index[b, h].tolist() == ref.select(wn[b, h], N, keep, 4, 16)
    mp, pages = 6, 40
    shape = (pages, H, page, D)
    k8 = torch.zeros(shape, dtype=torch.int8, device="cuda")
    v8 = torch.zeros(shape, dtype=torch.int8, device="cuda")
    if fmt == ref.E4M3:
        k8, v8 = k8.view(torch.float8_e4m3fn), v8.view(torch.float8_e4m3fn)
    kr, vr = torch.zeros((pages, H), device="cuda"), torch.zeros((pages, H), device="cuda")
    table = torch.randperm(pages)[: B * mp].view(B, mp).to(torch.int32).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    tm.tm_kv8_append(k, v, k.stride(1), v.stride(1), B, N, keep, H, D, kept, index, lens, table, mp,
                     k8, v8, kr, vr, pages, page, fmt)
    lens = kept.clone()
    acc = torch.zeros((B, H, mp * page), device="cuda")
    acc[..., :keep] = w.gather(2, index.long())

    def decode(step, table, lens, acc):
        t = rand((B, 1, W), 30 + step)
        pos = ints([[N + step]] * B)
        dq = torch.empty((B, 1, Hq, D), dtype=torch.bfloat16, device="cuda")
        dk = torch.empty((B, 1, H, D), dtype=torch.bfloat16, device="cuda")
        tm.tm_rope_fwd(t, dq, t[..., Hq * D:], dk, B, 1, Hq, H, D, W, Hq * D, W, H * D, D, 0, 0, df,
                       1.0, pos, 0)
        tm.tm_kv8_append(dk, t[..., (Hq + H) * D:], H * D, W, B, 1, 1, H, D, None, None, lens, table,
                         mp, k8, v8, kr, vr, pages, page, fmt)
        lens = lens + 1
        size = tm.tm_kv8_attn_workspace_size(B, 1, Hq, H, D, mp, page, True)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(dq)
        before = acc.clone()
        tm.tm_kv8_attn_fwd(dq, out, B, 1, Hq, H, D, D ** -0.5, k8, v8, kr, vr, pages, page, fmt,
                           table, mp, lens, acc, mp * page, 1, ws, size)
        codes = [(c if fmt == ref.INT8 else c.float()).double().cpu().numpy() for c in (k8, v8)]
        want, bound, ww, bw = ref.attention(dq.double().cpu().numpy(), *codes,
                                            kr.double().cpu().numpy(), vr.double().cpu().numpy(),
                                            table.cpu().numpy(), lens.tolist(), D ** -0.5, fmt)
        assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()
        got = (acc - before).double().cpu().numpy()
        slack = np.abs(acc.double().cpu().numpy()) * 2.0 ** -23
        assert (np.abs(got - ww) <= bw + slack).all()
        return lens

    for step in range(20):
        lens = decode(step, table, lens, acc)
    assert lens.tolist() == [keep + 20] * B
    smaller = 40
    index2 = torch.empty((B, H, smaller), dtype=torch.int32, device="cuda")
    tm.tm_kv_select(acc, mp * page, lens, B, H, mp * page, smaller, 4, 20, index2, kept)
    used = set(table.flatten().tolist())
    free = [p for p in range(pages) if p not in used]
    new_table = torch.full((B, mp), -1, dtype=torch.int32)
    new_table[:, :4] = torch.tensor(free[: 4 * B]).view(B, 4).to(torch.int32)
    new_table = new_table.cuda()
    new_acc = torch.zeros_like(acc)
    tm.tm_kv8_compact(index2, smaller, kept, lens, B, H, D, table, mp, new_table, mp, k8, v8, kr, vr,
                      pages, page, fmt, acc, mp * page, new_acc, mp * page)
    assert torch.equal(new_acc[..., :smaller], acc.gather(2, index2.long()))
    lens = kept.clone()
    for step in range(20, 24):
        lens = decode(step, new_table, lens, new_acc)
    assert lens.tolist() == [smaller + 4] * B


def test_conveniences_allocate_on_the_stream_they_run_on():
    """With the current stream busy: a result's zeros come before its kernel, a workspace that
    is given back is not overwritten from the current stream."""
    import torch
    B, N, Hq, H, D, L = 2, 300, 8, 2, 64, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn((B, N, h, D), generator=g, device="cuda").to(torch.bfloat16)
               for h in (Hq, H, H))
    f = torch.from_numpy(tm.tm_rope_inv_freq(D, 1e4)).cuda()
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    full = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    table = torch.arange(2 * 5, dtype=torch.int32, device="cuda").view(2, 5)
    cache = tm.Kv8Cache.empty(10, H, 64, D)

    def steps(stream):
        qr, kr = tm.rope(q, k, f, stream=stream)
        tm.kv8_append(cache, kr, v, lens, table, counts=full, stream=stream)
        w = tm.key_weights(qr, kr, L, lens=full, stream=stream)
        o = tm.kv8_attention(cache, q[:, -1:].contiguous(), full, table, stream=stream)
        index, kept = tm.kv_select(w, 50, 2, 8, lens=full, stream=stream)
        return qr, kr, w, o, index, kept

    want = steps(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)
        ws = tm.tm_key_weights_workspace_size(B, Hq, H, N, D, L)
        with torch.cuda.stream(side):
            last = q[:, -1:].contiguous()
        got = [tm.key_weights(q, k, L, lens=full, stream=stream)]
        fill = torch.full((ws,), 255, dtype=torch.uint8, device="cuda")
        o = tm.kv8_attention(cache, last, full, table, stream=stream)
        got += [o, *tm.kv_select(want[2], 50, 2, 8, lens=full, stream=stream)]
        torch.cuda.synchronize()
        plain = tm.key_weights(q, k, L, lens=full)
        assert torch.equal(got[0], plain) and torch.equal(got[1], want[3])
        assert torch.equal(got[2], want[4]) and torch.equal(got[3], want[5])
        assert int(fill.min()) == 255
    turned = tm.rope(q, k, f, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(turned[0], want[0]) and torch.equal(turned[1], want[1])
