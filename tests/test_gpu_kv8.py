"""The 8-bit cache on the GPU: append and compact bit for bit against the 64-bit
definition (every code and range, and that nothing else moved), attention
within the bound that follows from its arithmetic, and the calls that are easy
to get wrong: empty and short sequences, missing pages, NaN and infinities,
pools past 32 bits, captured graphs, other streams."""
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


class Cache:
    """A pool with every page filled, a random table, and its numpy image."""

    def __init__(self, seed, B, H, D, page, fmt, max_pages, spare=3, extra=0, empty=False):
        import torch
        g = torch.Generator().manual_seed(seed)
        self.H, self.D, self.page, self.fmt, self.max_pages = H, D, page, fmt, max_pages
        n = B * max_pages + spare + extra
        self.n = n
        x = torch.randn((2, n, H, page, D), generator=g)
        if fmt == ref.INT8:
            c = (x * 40).round().clamp(-127, 127).to(torch.int8)
        else:
            c = (x * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
        r = (2 + 6 * torch.rand((2, n, H), generator=g)).to(torch.bfloat16).float()
        if empty:
            c, r = c.view(torch.int8).zero_().view(c.dtype), r.zero_()
        self.k8, self.v8 = c[0].cuda().contiguous(), c[1].cuda().contiguous()
        self.kr, self.vr = r[0].cuda(), r[1].cuda()
        order = torch.randperm(n, generator=g).to(torch.int32)
        self.table = order[: B * max_pages].view(B, max_pages).cuda().contiguous()
        self.unused = order[B * max_pages:]

    def codes(self, t):
        import torch
        return t.double().cpu().numpy() if t.dtype == torch.int8 else t.float().double().cpu().numpy()

    def image(self):
        return (self.codes(self.k8), self.codes(self.v8), self.kr.double().cpu().numpy(),
                self.vr.double().cpu().numpy())

    def append(self, k, v, lens, counts=None, index=None, n=None, strides=None):
        ks, vs = strides or (k.stride(1), v.stride(1))
        tm.tm_kv8_append(k, v, ks, vs, k.shape[0], k.shape[1], k.shape[1] if n is None else n,
                         self.H, self.D, counts, index, lens, self.table, self.max_pages, self.k8,
                         self.v8, self.kr, self.vr, self.n, self.page, self.fmt)

    def attend(self, q, lens, weights=None, accumulate=0, o=None, ws=None, scale=None, stream=None):
        import torch
        B, nq, Hq, D = q.shape
        o = torch.full_like(q, float("nan")) if o is None else o
        size = tm.tm_kv8_attn_workspace_size(B, nq, Hq, self.H, D, self.max_pages, self.page,
                                             weights is not None)
        if ws is None:
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        tm.tm_kv8_attn_fwd(q, o, B, nq, Hq, self.H, D, scale or 1 / math.sqrt(D), self.k8, self.v8,
                           self.kr, self.vr, self.n, self.page, self.fmt, self.table,
                           self.max_pages, lens, weights,
                           0 if weights is None else weights.shape[2], accumulate, ws, size, stream)
        return o


def ints(x):
    import torch
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rand(shape, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).cuda()


def same(cache, want_k, want_v, want_kr, want_vr):
    k, v, kr, vr = cache.image()
    np.testing.assert_array_equal(kr, want_kr)
    np.testing.assert_array_equal(vr, want_vr)
    np.testing.assert_array_equal(k, want_k)
    np.testing.assert_array_equal(v, want_v)


def check_append(cache, k, v, lens, counts=None, index=None, n=None):
    n = n or k.shape[1]
    kc, vc, kr, vr = cache.image()
    table = cache.table.cpu().numpy()
    cnt = [n] * k.shape[0] if counts is None else np.clip(counts, 0, n)
    with np.errstate(invalid="ignore"):
        wk = ref.append(k.double().cpu().numpy(), lens, cnt, table, kc, kr, cache.fmt, index)
        wv = ref.append(v.double().cpu().numpy(), lens, cnt, table, vc, vr, cache.fmt, index)
    cache.append(k, v, ints(lens), None if counts is None else ints(counts),
                 None if index is None else ints(index), n)
    same(cache, wk[0], wv[0], wk[1], wv[1])


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("page,D,H", [(16, 64, 1), (16, 128, 3), (32, 64, 2), (64, 128, 2),
                                      (128, 128, 1), (128, 64, 2), (64, 64, 5)])
def test_append_is_the_definition(fmt, page, D, H):
    B = 4
    cache = Cache(1, B, H, D, page, fmt, 4)
    for seed, n, lens, counts in [
            (10, 1, [0, 5, page - 1, page], None),          # single tokens, page starts and ends
            (11, 1, [1, 6, page + 3, 4 * page - 1], None),
            (12, 2 * page + 7, [0, 3, page, 2 * page - 1], None),   # past the table's end in part
            (13, page + 5, [2, 2, 2, 2], [0, 1, page + 5, 999]),
            (14, 3, [4 * page, 5 * page, 10 ** 9, -7], None)]:      # full, beyond, negative
        check_append(cache, rand((B, n, H, D), seed, 3.0), rand((B, n, H, D), seed + 50), lens, counts)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_append_rounds_ties_and_every_ratio(fmt):
    """Blocks whose largest value and elements run through all bf16 significands,
    the exact ties of the quotient (x = r / 2 gives 63.5, r = 254 2^e halves) among
    them, at magnitudes from 2^-126 (bf16's least normal ones) to 2^111."""
    import torch
    H, D, page = 1, 64, 16
    cache = Cache(2, 128, H, D, page, fmt, 1)
    tops = torch.arange(128, 256).double()
    e = torch.tensor([-118.0, -80.0, -20.0, 0.0, 15.0, 110.0])[torch.arange(128) % 6].double()
    x = torch.zeros((128, page, H, D), dtype=torch.float64)
    low = torch.arange(128, 256).double()
    vals = torch.cat([low * 2.0 ** -s for s in range(0, 8)])[: page * D]      # 1024 values
    for b in range(128):
        row = vals.clone()
        row = torch.where(row > tops[b], row / 2, row)
        row[0], row[1] = tops[b], tops[b] / 2
        row[2::2] *= -1
        x[b, :, 0] = (row * 2.0 ** (e[b] - 7)).view(page, D)
    k = x.to(torch.bfloat16).cuda()
    assert torch.equal(k.double().cpu(), x)
    check_append(cache, k, k.flip(1).contiguous(), [0] * 128)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_append_moves_old_codes_as_the_range_grows(fmt):
    """Token by token with growing and falling magnitudes, against the definition at every step."""
    H, D, page = 2, 64, 16
    cache = Cache(3, 1, H, D, page, fmt, 2)
    for i in range(22):
        k = rand((1, 1, H, D), 100 + i, [1.0, 4.0, 0.1, 2.0 ** (i % 7)][i % 4])
        v = rand((1, 1, H, D), 200 + i, 2.0 ** (i // 3))
        check_append(cache, k, v, [i])


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_append_zeros_nan_and_infinities(fmt):
    import torch
    B, H, D, page = 4, 2, 64, 16
    cache = Cache(4, B, H, D, page, fmt, 2)
    k, v = rand((B, 20, H, D), 5), rand((B, 20, H, D), 6)
    k[0] = 0
    k[1, 3, 0, 7] = float("nan")
    k[2, 18, 1, 9] = float("inf")
    v[3, 0, 0, 0] = float("-inf")
    v[0, 2, 1, 1], v[0, 3, 1, 1] = float("nan"), float("inf")
    check_append(cache, k, v, [0, 0, 5, 9])
    tiny = torch.full((B, 1, H, D), 1e-39, dtype=torch.bfloat16, device="cuda")  # subnormal
    check_append(cache, tiny, tiny * 3, [20, 20, 25, 29])
    check_append(cache, tiny, tiny * 5, [0, 0, 0, 0])
    check_append(cache, k[:, :1].contiguous(), v[:, :1].contiguous(), [1, 1, 1, 1])


def test_append_index_strides_and_missing_pages():
    import torch
    B, H, D, page, n_src = 3, 2, 128, 32, 50
    cache = Cache(6, B, H, D, page, ref.INT8, 3)
    cache.table[0, 1] = -1
    cache.table[1, 0] = cache.n
    cache.table[2, 2] = 2 ** 31 - 1
    packed = rand((B, n_src, (4 + 2 * H) * D), 7, 2.0)
    k, v = packed[..., 4 * D:(4 + H) * D], packed[..., (4 + H) * D:]
    k, v = k.unflatten(-1, (H, D)), v.unflatten(-1, (H, D))
    check_append(cache, k, v, [0, 3, 40])
    rng = np.random.default_rng(8)
    index = np.stack([np.stack([np.sort(rng.permutation(n_src)[:40]) for _ in range(H)])
                      for _ in range(B)])
    index[0, 1, 5], index[1, 0, 0], index[2, 1, 39] = -1, n_src, 2 ** 31 - 1
    check_append(cache, k, v, [0, 10, 20], [40, 31, 17], index, n=40)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("page,D", [(16, 64), (16, 128), (32, 128), (64, 64), (128, 128)])
def test_compact_is_the_definition(fmt, page, D):
    import torch
    B, H, mp, keep = 3, 2, 5, page + 9
    cache = Cache(9, B, H, D, page, fmt, mp, spare=2, extra=2 * B)
    new_table = cache.unused[: 2 * B].view(B, 2).cuda().contiguous()
    lens = [5 * page, 2 * page + 3, 7]
    rng = np.random.default_rng(10)
    index = np.full((B, H, keep), -1)
    kept = [min(keep, n) for n in lens]
    for b in range(B):
        for h in range(H):
            index[b, h, : kept[b]] = np.sort(rng.permutation(lens[b])[: kept[b]])
    index[0, 0, 3] = lens[0]           # outside: stores zeros
    index[1, 1, 2] = -5
    cache.table[0, 4] = -1             # a page that is not there
    w = torch.rand((B, H, 5 * page), device="cuda")
    nw = torch.full((B, H, keep + 3), -7.0, device="cuda")
    kc, vc, kr, vr = cache.image()
    t = cache.table.cpu().numpy()
    wk = ref.compact(index, kept, lens, t, new_table.cpu().numpy(), kc, kr, fmt)
    wv = ref.compact(index, kept, lens, t, new_table.cpu().numpy(), vc, vr, fmt)
    tm.tm_kv8_compact(ints(index), keep, ints(kept), ints(lens), B, H, D, cache.table, mp, new_table,
                      2, cache.k8, cache.v8, cache.kr, cache.vr, cache.n, page, fmt, w, 5 * page, nw,
                      keep + 3)
    same(cache, wk[0], wv[0], wk[1], wv[1])
    w, nw = w.cpu().numpy(), nw.cpu().numpy()
    for b in range(B):
        for h in range(H):
            for i in range(keep + 3):
                want = -7.0
                if i < kept[b]:
                    j = index[b, h, i]
                    ok = 0 <= j < lens[b] and 0 <= t[b, j // page] < cache.n
                    want = w[b, h, j] if ok else 0.0
                assert nw[b, h, i] == np.float32(want)


# ------------------------------------------------------------------------------ attention

def check_attention(cache, q, lens, weights=False, scale=None, **more):
    import torch
    scale = scale or 1 / math.sqrt(q.shape[3])
    kc, vc, kr, vr = cache.image()
    o, bo, w, bw = ref.attention(q.double().cpu().numpy(), kc, vc, kr, vr, cache.table.cpu().numpy(),
                                 lens, scale, cache.fmt)
    cap = cache.max_pages * cache.page
    dw = torch.full((q.shape[0], cache.H, cap + 2), -3.0, device="cuda") if weights else None
    got = cache.attend(q, ints(lens), dw, scale=scale, **more)
    err = np.abs(got.double().cpu().numpy() - o)
    assert (err <= bo).all(), (err - bo).max()
    if weights:
        x = dw.double().cpu().numpy()
        for b, n in enumerate(lens):
            n = min(max(n, 0), cap)
            err = np.abs(x[b, :, :n] - w[b, :, :n])
            assert (err <= bw[b, :, :n]).all(), (err - bw[b, :, :n]).max()
            assert (x[b, :, n:] == -3.0).all()
    return got


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("page,D", [(16, 64), (16, 128), (32, 128), (64, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("Hq,H,nq", [(1, 1, 1), (4, 1, 1), (14, 2, 1), (8, 2, 3), (16, 1, 2), (6, 2, 8)])
def test_attention_within_its_bound(fmt, page, D, Hq, H, nq):
    mp = max(2, 160 // page)
    cache = Cache(20 + page + D, 5, H, D, page, fmt, mp)
    lens = [mp * page, 0, 1, 17, mp * page - 5]
    check_attention(cache, rand((5, nq, Hq, D), 21, 1.5), lens, weights=(Hq + nq) % 2 == 0)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_attention_ragged_long_and_split(fmt):
    """One long sequence among short ones: items cut between CTAs and many within one."""
    cache = Cache(30, 6, 2, 128, 64, fmt, 70)
    check_attention(cache, rand((6, 1, 8, 128), 31, 1.5), [4480, 1, 63, 64, 65, 1999], weights=True)


def test_attention_one_head_of_one_sequence():
    cache = Cache(33, 1, 1, 128, 16, ref.INT8, 300)
    for n in (1, 15, 16, 17, 1000, 4799, 4800):
        check_attention(cache, rand((1, 1, 4, 128), n, 1.5), [n], weights=True)


def test_attention_many_short_sequences():
    rng = np.random.default_rng(35)
    cache = Cache(34, 300, 2, 64, 16, ref.E4M3, 3)
    check_attention(cache, rand((300, 1, 4, 64), 36, 1.5), rng.integers(0, 49, 300).tolist(), True)


def test_attention_lengths_are_clamped_and_missing_pages_skipped():
    cache = Cache(37, 4, 2, 128, 32, ref.INT8, 4)
    cache.table[1, 2] = -1
    cache.table[2, 0] = cache.n
    cache.table[3] = 2 ** 31 - 1
    got = check_attention(cache, rand((4, 2, 8, 128), 38), [10 ** 9, 128, 70, 128], True)
    assert (got[3] == 0).all()
    assert (check_attention(cache, rand((4, 2, 8, 128), 38), [-3, 0, 0, 0]) == 0).all()


def test_attention_extreme_scores_and_values():
    """Sharp and flat rows, large and tiny q, ranges over many magnitudes."""
    cache = Cache(39, 3, 2, 128, 16, ref.INT8, 12)
    import torch
    cache.vr.copy_(2.0 ** torch.randint(-30, 30, cache.vr.shape, device="cuda").float())
    q = rand((3, 1, 8, 128), 40)
    check_attention(cache, q * 60, [192, 100, 33], True)
    check_attention(cache, q * 0, [192, 100, 33], True)
    check_attention(cache, q * 2.0 ** 100, [192, 100, 33], scale=2.0 ** -103)
    check_attention(cache, q * 2.0 ** -100, [192, 100, 33], scale=2.0 ** 97)
    mixed = q.clone()
    mixed[..., ::3] *= 2.0 ** -18
    check_attention(cache, mixed, [192, 100, 33], True)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
def test_attention_of_rows_that_do_not_see_a_nan(fmt):
    """A NaN block in the last page reaches the rows that see it and no other; garbage
    behind the last token (NaN codes among it) reaches none."""
    import torch
    cache = Cache(41, 2, 1, 64, 16, fmt, 3)
    last = int(cache.table[0, 2])
    cache.kr[last], cache.vr[last] = float("nan"), float("nan")
    cache.k8.view(torch.int8)[int(cache.table[1, 1]), :, 3:] = 0x7F
    cache.v8.view(torch.int8)[int(cache.table[1, 1]), :, 3:] = 0x7F
    q = rand((2, 3, 4, 64), 42)
    got = cache.attend(q, ints([33, 19]))
    assert torch.isfinite(got[0, :2]).all() and torch.isnan(got[0, 2]).all()
    assert torch.isfinite(got[1]).all()
    clean = Cache(41, 2, 1, 64, 16, fmt, 3)
    want = clean.attend(q, ints([33, 19]))
    assert torch.equal(got[0, :2], want[0, :2]) and torch.equal(got[1], want[1])


def test_attention_of_rows_that_do_not_see_an_infinity():
    """An infinite range reads as NaN to the rows that see its block and not at all to others."""
    import torch
    for fmt in (ref.INT8, ref.E4M3):
        cache = Cache(41, 1, 1, 64, 16, fmt, 3)
        q, last = rand((1, 3, 4, 64), 42), int(cache.table[0, 2])
        want = cache.attend(q, ints([33]))
        cache.vr[last] = float("inf")
        got = cache.attend(q, ints([33]))
        assert torch.equal(got[0, :2], want[0, :2]) and torch.isnan(got[0, 2]).all()


def test_attention_with_a_far_larger_range_that_weighs_nothing():
    """Keys of weight 2^-40 and less whose values are 2^20 times the others' (and the other way
    round, and ranges that fall by 2^60 a page): the others keep the precision they would have
    alone. Bound: 2^-8 of o for bf16, 2^-10 of the weighted |v| for P (2^-11) and the scores."""
    import torch
    H, D, page, mp = 1, 128, 16, 8
    for fmt in (ref.INT8, ref.E4M3):
        for big in ([0], [7], [3], [0, 2, 4, 6]):
            cache = Cache(60, 1, H, D, page, fmt, mp)
            q = rand((1, 1, 4, D), 61).abs()
            # |q| only, and keys that are all of one sign: theirs are far below the others' scores
            signs = cache.k8.float().abs().clamp(min=1)
            cache.k8.copy_(signs.to(cache.k8.dtype))
            for j in big:
                pg = int(cache.table[0, j])
                cache.k8[pg] = (-signs[pg]).to(cache.k8.dtype)
                cache.vr[pg] *= 2.0 ** 20
            kc, vc, kr, vr = cache.image()
            tab = cache.table.cpu().numpy()
            k, _ = ref.values(kc, kr, tab, 0, 0, mp * page, fmt)
            v, _ = ref.values(vc, vr, tab, 0, 0, mp * page, fmt)
            scale = 8.0 / math.sqrt(D)
            got = cache.attend(q, ints([mp * page]), scale=scale).double().cpu().numpy()
            for g in range(4):
                sc = k @ q[0, 0, g].double().cpu().numpy() * scale
                p = np.exp(sc - sc.max())
                p /= p.sum()
                rows = np.repeat([j in big for j in range(mp)], page)
                assert p[rows].max() < 2.0 ** -60
                err = np.abs(got[0, 0, g] - p @ v)
                assert (err <= np.abs(p @ v) * 2.0 ** -8 + (p @ np.abs(v)) * 2.0 ** -10).all()
    cache = Cache(62, 1, H, D, page, ref.INT8, mp)
    cache.vr[cache.table[0].long(), 0] = 2.0 ** torch.tensor([50.0, 40, -20, -80, -100, 0, 50, -40],
                                                             device="cuda")
    check_attention(cache, rand((1, 1, 4, D), 63), [mp * page])


def test_torch_conveniences_make_the_same_calls():
    import torch
    B, H, Hq, D, page, mp = 2, 2, 8, 64, 16, 4
    a = Cache(70, B, H, D, page, ref.E4M3, mp, extra=8)
    b = Cache(70, B, H, D, page, ref.E4M3, mp, extra=8)
    c = tm.Kv8Cache(b.k8, b.v8, b.kr, b.vr)
    packed = rand((B, 9, (Hq + 2 * H) * D), 71)
    q, k, v = (t.unflatten(-1, (-1, D)) for t in packed.split([Hq * D, H * D, H * D], -1))
    f = torch.from_numpy(tm.tm_rope_inv_freq(D, 10000.0)).cuda()
    qo, ko = tm.rope(q, k, f, first=3)
    in_place = packed.clone()
    q2, k2 = (t.unflatten(-1, (-1, D)) for t in in_place.split([Hq * D, H * D, H * D], -1)[:2])
    tm.rope(q2, k2, f, first=3, out=(q2, k2))
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    lens = ints([5, 11])
    a.append(ko, v, lens, strides=(H * D, (Hq + 2 * H) * D))
    tm.kv8_append(c, ko, v, lens, b.table)
    assert torch.equal(a.k8.view(torch.int8), b.k8.view(torch.int8)) and torch.equal(a.vr, b.vr)
    lens = lens + 9
    w = torch.zeros((B, H, mp * page), device="cuda")
    w2 = torch.zeros_like(w)
    o = a.attend(qo, lens, w)
    assert torch.equal(tm.kv8_attention(c, qo, lens, b.table, weights=w2), o)
    assert torch.equal(w, w2)
    index, kept = tm.kv_select(w, 6, 1, 2, lens)
    new = b.unused[:B].view(B, 1).cuda()
    nw = torch.zeros((B, H, 6), device="cuda")
    tm.kv8_compact(c, index, kept, lens, b.table, new, w, nw)
    assert torch.equal(nw, w.gather(2, index.long()))
    wk = tm.key_weights(qo, ko, 4)
    np.testing.assert_allclose(wk.sum(-1).cpu().numpy(), 4 * Hq / H, rtol=1e-4)


def test_attention_accumulates_weights_and_repeats_to_the_bit():
    import torch
    cache = Cache(43, 4, 2, 128, 16, ref.E4M3, 40)
    q = rand((4, 1, 14, 128), 44)
    lens = ints([640, 333, 0, 1])
    w = torch.rand((4, 2, 640), device="cuda")
    start = w.clone()
    o1 = cache.attend(q, lens, w, 1)
    w0 = torch.zeros_like(w)
    o2 = cache.attend(q, lens, w0, 0)
    assert torch.equal(o1, o2)
    assert torch.equal(w, start + w0)
    for b, n in enumerate(lens.tolist()):  # each row's weights sum to 1: 7 q heads a kv head
        if n:
            np.testing.assert_allclose(w0[b, :, :n].sum(-1).cpu().numpy(), 7.0, rtol=1e-4)
    short = torch.full((4, 2, 100), 9.0, device="cuda")   # keys past the stride are not written
    cache.attend(q, lens, short)
    assert torch.equal(short[0], w0[0, :, :100]) and torch.equal(short[2], torch.full_like(short[2], 9.0))


def test_pools_past_32_bits():
    """Pages at the far end of pools of 5 GB each: append, attention, compact."""
    import torch
    n, H, page, D = 40000, 8, 128, 128
    cache = Cache(45, 1, H, D, page, ref.INT8, 4)
    small = cache.image()
    old = cache.table.clone()
    k8 = torch.empty((n, H, page, D), dtype=torch.int8, device="cuda")
    v8 = torch.empty_like(k8)
    kr, vr = torch.zeros((n, H), device="cuda"), torch.zeros((n, H), device="cuda")
    far = torch.tensor([[39999, 17000, 33000, 39998]], dtype=torch.int32, device="cuda")
    for a, b in zip(old[0].tolist(), far[0].tolist()):
        k8[b], v8[b], kr[b], vr[b] = cache.k8[a], cache.v8[a], cache.kr[a], cache.vr[a]
    big = Cache(45, 1, H, D, page, ref.INT8, 4)
    big.k8, big.v8, big.kr, big.vr, big.n, big.table = k8, v8, kr, vr, n, far
    q = rand((1, 1, 32, D), 46)
    assert torch.equal(big.attend(q, ints([500])), cache.attend(q, ints([500])))
    k, v = rand((1, 100, H, D), 47), rand((1, 100, H, D), 48)
    big.append(k, v, ints([400]))
    cache.append(k, v, ints([400]))
    for a, b in zip(old[0].tolist(), far[0].tolist()):
        assert torch.equal(k8[b], cache.k8[a]) and torch.equal(vr[b], cache.vr[a])
    index = torch.arange(0, 400, 4, dtype=torch.int32, device="cuda").expand(1, H, 100).contiguous()
    to = torch.tensor([[39997]], dtype=torch.int32, device="cuda")
    tm.tm_kv8_compact(index, 100, None, ints([500]), 1, H, D, far, 4, to, 1, k8, v8, kr, vr, n, page,
                      0, None, 0, None, 0)
    spare = cache.unused[:1].view(1, 1).cuda()
    tm.tm_kv8_compact(index, 100, None, ints([500]), 1, H, D, cache.table, 4, spare, 1, cache.k8,
                      cache.v8, cache.kr, cache.vr, cache.n, page, 0, None, 0, None, 0)
    assert torch.equal(k8[39997, :, :100], cache.k8[int(spare), :, :100])
    assert torch.equal(v8[39997, :, :100], cache.v8[int(spare), :, :100])
    assert small[0].shape[0] == cache.n


def test_captured_steps_replay_with_new_lengths():
    """append + attention captured once and replayed as the sequence grows, against eager
    steps; two graphs that share one workspace, replayed in turn."""
    import torch
    B, H, Hq, D, page, mp, steps = 3, 2, 8, 128, 16, 4, 20
    a, b = (Cache(50, B, H, D, page, ref.INT8, mp) for _ in range(2))
    k, v = rand((B, steps, H, D), 51), rand((B, steps, H, D), 52)
    q = rand((B, steps, Hq, D), 53)
    lens = ints([0, 7, 30])
    size = tm.tm_kv8_attn_workspace_size(B, 1, Hq, H, D, mp, page, True)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    kk, vv, qq = (torch.empty((B, 1, h, D), dtype=torch.bfloat16, device="cuda") for h in (H, H, Hq))
    o, w = torch.empty_like(qq), torch.zeros((B, H, mp * page), device="cuda")
    after = lens.clone()

    def step():
        a.append(kk, vv, lens)
        after.copy_(lens + 1)
        a.attend(qq, after, w, 1, o, ws)
        lens.copy_(after)

    o_other = torch.empty_like(qq)
    keep = a.k8.clone(), a.v8.clone(), a.kr.clone(), a.vr.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    for t, x in zip((a.k8, a.v8, a.kr, a.vr), keep):
        t.copy_(x)
    lens.copy_(ints([0, 7, 30]))
    w.zero_()
    g, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    with torch.cuda.graph(other):
        b.attend(qq, after, None, 0, o_other, ws)
    lens.copy_(ints([0, 7, 30]))
    ref_lens, rw = ints([0, 7, 30]), torch.zeros_like(w)
    c = Cache(50, B, H, D, page, ref.INT8, mp)
    for i in range(steps):
        for dst, src in ((kk, k), (vv, v), (qq, q)):
            dst.copy_(src[:, i:i + 1])
        g.replay()
        other.replay()
        c.append(kk, vv, ref_lens)
        ref_lens = ref_lens + 1
        want = c.attend(qq, ref_lens, rw, 1)
        assert torch.equal(o, want), i
        assert torch.equal(o_other, b.attend(qq, ref_lens)), i
    assert torch.equal(w, rw) and torch.equal(a.k8, c.k8) and torch.equal(a.vr, c.vr)


def test_work_on_another_stream_is_ordered_by_it():
    import torch
    cache = Cache(54, 2, 2, 128, 64, ref.E4M3, 30)
    q = rand((2, 1, 8, 128), 55)
    lens = ints([1900, 700])
    want = cache.attend(q, lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    late = torch.zeros_like(q)
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late.copy_(q)
        got = cache.attend(late, lens)
    got2 = torch.empty_like(q)
    torch.cuda.synchronize()
    cache.attend(q, lens, o=got2, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got2, want)


def test_two_calls_at_once_with_workspaces_of_their_own():
    """Attention, append and weights on two streams that overlap, against one after the other."""
    import torch
    caches = [Cache(80 + i, 3, 2, 128, 32, fmt, 40) for i, fmt in enumerate((ref.INT8, ref.E4M3))]
    qs = [rand((3, 2, 8, 128), 82 + i) for i in range(2)]
    lens = [ints([1280, 700, 3]), ints([900, 1279, 0])]
    w = [torch.zeros((3, 2, 1280), device="cuda") for _ in range(4)]
    want = [c.attend(q, n, x) for c, q, n, x in zip(caches, qs, lens, w)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for rep in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(caches[i].attend(qs[i], lens[i], w[2 + i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])
        assert torch.equal(w[i], w[2 + i])


def test_sequences_that_share_pages_and_a_large_batch():
    """Pages read by several sequences; a batch of more sequences than a block has threads."""
    cache = Cache(84, 2, 1, 64, 16, ref.INT8, 4)
    cache.table[1, :2] = cache.table[0, :2]
    check_attention(cache, rand((2, 1, 4, 64), 85), [64, 50], True)
    rng = np.random.default_rng(86)
    big = Cache(87, 1100, 1, 64, 16, ref.E4M3, 1)
    check_attention(big, rand((1100, 1, 1, 64), 88), rng.integers(0, 17, 1100).tolist(), True)


def test_many_rows_take_several_tiles():
    """33 rows a kv head: three row tiles, the last one partly filled; and one query of 40 heads."""
    cache = Cache(89, 2, 1, 64, 32, ref.INT8, 3)
    check_attention(cache, rand((2, 11, 3, 64), 90), [96, 7], True)
    check_attention(cache, rand((2, 1, 40, 64), 91), [96, 33], True)


@pytest.mark.parametrize("fmt", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("page,D", [(16, 64), (16, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("Hq,H,nq", [(17, 1, 1), (8, 2, 8), (14, 2, 4), (3, 1, 11), (64, 2, 2)])
def test_attention_of_many_rows(fmt, page, D, Hq, H, nq):
    """17 to 64 rows a kv head: row tiles of 32, full and not, with queries that see nothing."""
    mp = max(2, 320 // page)
    cache = Cache(92 + page + D, 5, H, D, page, fmt, mp)
    check_attention(cache, rand((5, nq, Hq, D), 93, 1.5), [mp * page, 0, 1, 5, mp * page - 7], weights=True)


def test_attention_of_many_rows_long_and_split():
    """32 rows: items cut between CTAs, several in one, and a page that is not there."""
    cache = Cache(94, 4, 2, 128, 64, ref.INT8, 70)
    cache.table[0, 3] = -1
    check_attention(cache, rand((4, 8, 8, 128), 95, 1.5), [4480, 1, 64, 1999], weights=True)
