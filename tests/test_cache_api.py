"""Argument checks of the operators around the attention, without a GPU: every
refusal comes before any CUDA call (the pointers are never dereferenced), the
workspace sizes are host arithmetic, and the rotary frequencies are the
documented formula."""
import ctypes
import math

import numpy as np
import pytest

import cache_ref as ref
import long_context_prefill_trianglemix_b200 as tm
from long_context_prefill_trianglemix_b200 import build

A = 1 << 20          # fake addresses, far apart
INVALID, UNSUPPORTED = tm.TM_ERR_INVALID_ARG, tm.TM_ERR_UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build_lib()
    yield


def call(name, good, **change):
    args = dict(good)
    for k in change:
        assert k in args, k
    args.update(change)
    return getattr(tm.lib(), name)(*args.values())


def refused(name, good, cases):
    for change, want in cases:
        assert call(name, good, **change) == want, change


ROPE = dict(q=A, q_out=A + 0x100000, k=A + 0x200000, k_out=A + 0x300000, B=1, N=4, Hq=4, Hkv=2,
            D=128, q_stride=512, q_out_stride=512, k_stride=256, k_out_stride=256, rot=128,
            layout=0, inverse=0, inv_freq=A + 0x400000, mscale=1.0, positions=None, first=0,
            stream=None)


def test_rope_refusals():
    refused("tm_rope_fwd", ROPE, [
        (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(k=None), INVALID),
        (dict(inv_freq=None), INVALID), (dict(inv_freq=A + 4), INVALID), (dict(B=0), INVALID),
        (dict(N=0), INVALID), (dict(Hq=-1), INVALID), (dict(Hq=0), INVALID), (dict(D=72), UNSUPPORTED),
        (dict(D=1024), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=3), INVALID),
        (dict(rot=130), INVALID), (dict(layout=2), INVALID), (dict(mscale=float("nan")), INVALID),
        (dict(q=A + 8), INVALID), (dict(q_stride=504), INVALID), (dict(q_stride=516), INVALID),
        (dict(k_out_stride=128), INVALID), (dict(positions=A + 2), INVALID),
        (dict(B=1 << 20, N=1 << 12), INVALID), (dict(first=1 << 60), INVALID),
        (dict(q_out=A + 16), INVALID),                      # output over its input
        (dict(q_out=A, q_stride=1024), INVALID),            # in place at another stride
        (dict(k_out=A + 0x100000), INVALID),                # both outputs at one place
        (dict(k_out=A), INVALID),                           # k's output over q
    ])
    # packed rows that interleave without sharing a byte are fine, shared columns are not
    packed = dict(ROPE, q=A, q_out=A, k=A + 1024, k_out=A + 1024, q_stride=1024, q_out_stride=1024,
                  k_stride=1024, k_out_stride=1024)
    assert call("tm_rope_fwd", packed, k_out=A + 1008) == INVALID
    assert call("tm_rope_fwd", packed, k=A + 1024 + 512, k_out=A + 1024 + 256) == INVALID


def test_rope_frequencies():
    base, rot = 10000.0, 64
    f = base ** (-np.arange(0, rot, 2) / rot)
    np.testing.assert_allclose(tm.tm_rope_inv_freq(rot, base), f, rtol=1e-15)
    turns = 4096 * f / (2 * math.pi)
    s = np.clip((turns - 1.0) / (32.0 - 1.0), 0, 1)
    np.testing.assert_allclose(tm.tm_rope_inv_freq(rot, base, 4.0, 4096.0, 1.0, 32.0),
                               f * (s + (1 - s) / 4.0), rtol=1e-14)
    np.testing.assert_allclose(
        tm.tm_rope_inv_freq(rot, base, 4.0, 4096.0, math.inf, math.inf), f / 4.0, rtol=1e-15)
    for bad in [(63, base), (0, base), (64, -1.0), (64, base, 0.5), (64, base, math.nan),
                (64, base, 2.0, 0.0), (64, base, 2.0, 8.0, 2.0, 1.0)]:
        with pytest.raises(tm.TmError):
            tm.tm_rope_inv_freq(*bad)
    assert tm.lib().tm_rope_inv_freq(64, base, 1.0, 1.0, 0.0, 0.0, None) == INVALID


POOL = 64 * 2 * 16 * 64
APPEND = dict(k=A, v=A + 0x100000, k_stride=128, v_stride=128, B=2, n_src=8, n=8, Hkv=2, D=64,
              counts=None, index=None, lens=A + 0x200000, table=A + 0x210000, max_pages=4,
              k8=A + 0x300000, v8=A + 0x400000, k_range=A + 0x500000, v_range=A + 0x510000,
              num_pages=64, page=16, format=0, stream=None)
CACHE_CASES = [
    (dict(k8=None), INVALID), (dict(v8=None), INVALID), (dict(k_range=None), INVALID),
    (dict(k8=A + 0x300008), INVALID), (dict(k_range=A + 0x500002), INVALID),
    (dict(num_pages=0), INVALID), (dict(format=2), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(page=48), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=256), UNSUPPORTED),
    (dict(v8=A + 0x300000 + POOL - 16), INVALID), (dict(table=None), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 28), INVALID), (dict(B=0), INVALID),
    (dict(lens=None), INVALID), (dict(lens=A + 2), INVALID),
]


def test_append_refusals():
    refused("tm_kv8_append", APPEND, CACHE_CASES + [
        (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(n=0), INVALID),
        (dict(n=9), INVALID), (dict(n_src=0), INVALID), (dict(k=A + 8), INVALID),
        (dict(k_stride=120), INVALID), (dict(v_stride=130), INVALID), (dict(B=65536), INVALID),
        (dict(Hkv=40000, k_stride=40000 * 64, v_stride=40000 * 64), INVALID),
        (dict(k=A + 0x300000), INVALID), (dict(v=A + 0x400000), INVALID),
        (dict(counts=A + 1), INVALID), (dict(index=A + 1), INVALID),
    ])


COMPACT = dict(index=A, keep=20, kept=None, lens=A + 0x1000, B=2, Hkv=2, D=64, table=A + 0x2000,
               max_pages=4, new_table=A + 0x3000, new_max_pages=2, k8=A + 0x300000,
               v8=A + 0x400000, k_range=A + 0x500000, v_range=A + 0x510000, num_pages=64, page=16,
               format=1, weights=A + 0x10000, weights_stride=64, new_weights=A + 0x20000,
               new_weights_stride=20, stream=None)


def test_compact_refusals():
    refused("tm_kv8_compact", COMPACT, CACHE_CASES + [
        (dict(index=None), INVALID), (dict(keep=0), INVALID), (dict(keep=33), INVALID),
        (dict(new_table=None), INVALID), (dict(new_max_pages=1), INVALID),
        (dict(weights=None), INVALID), (dict(new_weights=None), INVALID),
        (dict(new_weights_stride=19), INVALID), (dict(weights_stride=0), INVALID),
        (dict(new_weights=A + 0x10000 + 64), INVALID), (dict(kept=A + 1), INVALID),
    ])


ATTN = dict(q=A, o=A + 0x10000, B=2, nq=1, Hq=4, Hkv=2, D=64, scale=0.125, k8=A + 0x300000,
            v8=A + 0x400000, k_range=A + 0x500000, v_range=A + 0x510000, num_pages=64, page=16,
            format=0, table=A + 0x2000, max_pages=4, lens=A + 0x1000, weights=None,
            weights_stride=0, accumulate=0, workspace=1 << 30, workspace_bytes=1 << 28, stream=None)


def test_attention_refusals():
    refused("tm_kv8_attn_fwd", ATTN, CACHE_CASES + [
        (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(nq=0), INVALID),
        (dict(Hq=3), INVALID), (dict(scale=0.0), INVALID), (dict(scale=math.inf), INVALID),
        (dict(q=A + 4), INVALID), (dict(o=A + 64), INVALID), (dict(o=A + 0x300000), INVALID),
        (dict(workspace=None), INVALID), (dict(workspace=(1 << 30) + 128), INVALID),
        (dict(workspace_bytes=1000), INVALID), (dict(B=4097), UNSUPPORTED),
        (dict(weights=A + 0x20000, weights_stride=0), INVALID),
        (dict(weights=A + 0x300000, weights_stride=64), INVALID),
        (dict(weights=A + 0x20002, weights_stride=64), INVALID),
        (dict(weights=(1 << 30) + 4096, weights_stride=64), INVALID),
        (dict(B=4000, max_pages=1 << 26), INVALID),          # more work units than 32 bits
    ])
    n = ctypes.c_longlong(-1)
    size = tm.lib().tm_kv8_attn_workspace_size
    assert size(2, 1, 4, 2, 64, 4, 16, 0, None) == INVALID
    assert size(2, 1, 4, 3, 64, 4, 16, 0, ctypes.byref(n)) == INVALID
    assert size(2, 1, 4, 2, 80, 4, 16, 0, ctypes.byref(n)) == UNSUPPORTED
    plain = tm.tm_kv8_attn_workspace_size(2, 1, 4, 2, 64, 4, 16, False)
    scores = 2 * 2 * 4 * 64 * 4  # items, padded rows, tokens, fp32
    assert tm.tm_kv8_attn_workspace_size(2, 1, 4, 2, 64, 4, 16, True) >= plain + scores
    assert call("tm_kv8_attn_fwd", ATTN, workspace_bytes=plain - 1) == INVALID


WEIGHTS = dict(q=A, k=A + 0x100000, B=2, Hq=4, Hkv=2, N=64, D=64, scale=0.125, L=8, lens=None,
               weights=A + 0x200000, weights_stride=64, accumulate=0, workspace=1 << 30,
               workspace_bytes=1 << 28, stream=None)


def test_key_weights_refusals():
    refused("tm_key_weights_fwd", WEIGHTS, [
        (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(weights=None), INVALID),
        (dict(workspace=None), INVALID), (dict(B=0), INVALID), (dict(Hq=5), INVALID),
        (dict(N=0), INVALID), (dict(L=0), INVALID), (dict(D=32), UNSUPPORTED),
        (dict(Hq=258), UNSUPPORTED), (dict(scale=-1.0), INVALID), (dict(q=A + 2), INVALID),
        (dict(lens=A + 2), INVALID), (dict(weights_stride=63), INVALID),
        (dict(weights=A), INVALID), (dict(weights=A + 0x100000), INVALID),
        (dict(workspace=(1 << 30) + 8), INVALID), (dict(workspace_bytes=64), INVALID),
        (dict(workspace=A), INVALID), (dict(B=1 << 20, N=1 << 12), INVALID),
    ])
    n = ctypes.c_longlong(-1)
    assert tm.lib().tm_key_weights_workspace_size(2, 4, 2, 64, 64, 8, None) == INVALID
    assert tm.lib().tm_key_weights_workspace_size(2, 4, 2, 64, 64, 0, ctypes.byref(n)) == INVALID
    need = tm.tm_key_weights_workspace_size(2, 4, 2, 64, 64, 8)
    assert call("tm_key_weights_fwd", WEIGHTS, workspace_bytes=need - 1) == INVALID


SELECT = dict(weights=A, weights_stride=100, lens=None, B=2, H=2, n=100, keep=10, sinks=2, recent=4,
              index=A + 0x10000, kept=None, stream=None)


def test_select_refusals():
    refused("tm_kv_select", SELECT, [
        (dict(weights=None), INVALID), (dict(index=None), INVALID), (dict(B=0), INVALID),
        (dict(H=0), INVALID), (dict(n=0), INVALID), (dict(keep=0), INVALID),
        (dict(sinks=-1), INVALID), (dict(recent=-1), INVALID), (dict(recent=9), INVALID),
        (dict(weights_stride=99), INVALID), (dict(weights=A + 1), INVALID),
        (dict(lens=A + 1), INVALID), (dict(index=A + 16), INVALID), (dict(kept=A + 8), INVALID),
        (dict(kept=A + 0x10000), INVALID), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), INVALID),
    ])


def test_reference_rounding_is_the_formats():
    """The tests' own rounding against torch's e4m3 and numpy's integers, ties included."""
    import torch
    x = np.concatenate([np.arange(-448, 449) / 2.0, np.arange(0, 64) * 2.0 ** -11,
                        np.linspace(-30, 30, 1001)]).astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ref.nearest(x, ref.E4M3), got)
    assert ref.nearest(2.5, ref.INT8) == 2 and ref.nearest(3.5, ref.INT8) == 4


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """Before any CUDA call: a host tensor (a kernel would fault on it), other types and shapes."""
    import torch
    x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    i32 = torch.zeros((1,), dtype=torch.int32)
    table = torch.zeros((1, 2), dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    cache = tm.Kv8Cache.empty(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="current CUDA device"):
        tm.rope(x, x.clone(), f)
    with pytest.raises(ValueError, match="current CUDA device"):
        tm.kv8_append(cache, x, x, i32, table)
    with pytest.raises(ValueError, match="current CUDA device"):
        tm.kv8_attention(cache, x, i32, table)
    with pytest.raises(ValueError, match="current CUDA device"):
        tm.key_weights(x, x, 2)
    with pytest.raises(ValueError, match="current CUDA device"):
        tm.kv_select(torch.zeros((1, 2, 8)), 4)
    bad = [lambda: tm.rope(x, x, f.float()), lambda: tm.rope(x, x, f[:30]),
           lambda: tm.rope(x.float(), None, f), lambda: tm.rope(x, x[:, :3], f),
           lambda: tm.rope(x, x, f, positions=torch.zeros((1, 4))),
           lambda: tm.rope(x.transpose(2, 3), None, f[:1]),
           lambda: tm.kv8_append(cache, x, x, i32.long(), table),
           lambda: tm.kv8_append(cache, x[..., :32], x[..., :32], i32, table),
           lambda: tm.kv8_append(cache, x, x[:, :2], i32, table),
           lambda: tm.kv8_append(cache, x, x, i32, table[0]),
           lambda: tm.kv8_append(cache, x, x, i32, table, index=torch.zeros((1, 1, 4), dtype=torch.int32)),
           lambda: tm.kv8_append(cache, x, x, i32, table, counts=torch.zeros(2, dtype=torch.int32)),
           lambda: tm.kv8_append(cache._replace(k_range=i32), x, x, i32, table),
           lambda: tm.kv8_append(cache._replace(v8=cache.v8.float()), x, x, i32, table),
           lambda: tm.kv8_attention(cache, x.float(), i32, table),
           lambda: tm.kv8_attention(cache, x, i32, table, weights=torch.zeros((1, 1, 32))),
           lambda: tm.key_weights(x, x.float(), 2),
           lambda: tm.key_weights(x, x, 2, lens=torch.zeros(1)),
           lambda: tm.kv_select(torch.zeros((1, 2, 8)).double(), 4),
           lambda: tm.kv8_compact(cache, torch.zeros((1, 3, 4), dtype=torch.int32), i32, i32, table, table)]
    for n, call_ in enumerate(bad):
        with pytest.raises(ValueError) as e:
            call_()
        assert "current CUDA device" not in str(e.value), n
    one = torch.zeros((3, 1, 640), dtype=torch.bfloat16)[..., :128].unflatten(-1, (2, 64))
    assert tm._token_rows(one, "q") == 640      # a one-token slice of a packed projection
    assert tm._token_rows(x, "q") == 128
    with pytest.raises(ValueError, match="follow each other"):
        tm._token_rows(torch.zeros((2, 8, 2, 64), dtype=torch.bfloat16)[:, :4], "q")


def test_binding_takes_addresses_not_the_numbers_of_an_array():
    """A host array of one number is not the address it holds, nor is a float one."""
    for x in (np.array([4096], np.int32), np.array([4096.0], np.float32), 4096.0):
        with pytest.raises(TypeError):
            tm.tm_kv_select(A, 8, x, 1, 1, 8, 4, 0, 0, A)
        with pytest.raises(TypeError):
            tm.tm_kv8_attn_fwd(A, A, 1, 1, 1, 1, 64, 1.0, A, A, A, A, 1, 16, 0, x, 1, A, None, 0, 0,
                               A, 1 << 30)
