"""The strides that the raw calls pass on, without a GPU: a tensor [B, N, ...] whose
rows lie elsewhere than the number says is read where its rows are, or refused."""
import pytest

import long_context_prefill_trianglemix_b200 as tm


@pytest.fixture
def calls(monkeypatch):
    """Every call of the library as (name, arguments); tensors pass for addresses."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or tm.TM_OK

    monkeypatch.setattr(tm, "lib", lambda: Library())
    monkeypatch.setattr(tm, "_device_ptrs",
                        lambda *xs, **_: [x if x is None else x.data_ptr() for x in xs])
    monkeypatch.setattr(tm, "_stream", lambda s: 0)
    return made


def packed(B, N, Hq, Hkv, D):
    import torch
    x = torch.zeros((B, N, (Hq + 2 * Hkv) * D), dtype=torch.bfloat16)
    return [t.view(B, N, -1, D) for t in x.split([Hq * D, Hkv * D, Hkv * D], -1)]


def rope(q, k, q_stride, k_stride, qo=None, ko=None, strides=None):
    import torch
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    qo = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16) if qo is None else qo
    ko = torch.zeros((B, N, Hkv, D), dtype=torch.bfloat16) if ko is None else ko
    f = torch.zeros(D // 2, dtype=torch.float64)
    tm.tm_rope_fwd(q, qo, k, ko, B, N, Hq, Hkv, D, q_stride, *(strides or (Hq * D,)), k_stride,
                   *(strides or (Hkv * D,)), D, 0, 0, f, 1.0, None, 0)


def test_rope_of_one_token_passes_the_stride_between_sequences(calls):
    q, k, _ = packed(3, 1, 4, 2, 64)
    assert q.stride(1) != q.stride(0) == 512
    rope(q, k, q.stride(1), k.stride(1))
    rope(q, k, q.stride(0), 512)
    rope(q, k, q.stride(1), k.stride(1), q, k, (512,))
    for name, args in calls:
        assert name == "tm_rope_fwd" and args[9] == 512 and args[11] == 512
    assert [args[10] for _, args in calls] == [256, 256, 512]
    assert [args[12] for _, args in calls] == [128, 128, 512]


def test_rope_of_several_tokens_passes_its_numbers_on(calls):
    q, k, _ = packed(3, 5, 4, 2, 64)
    rope(q, k, 512, 512)
    flat = q[:1]
    rope(flat, k[:1], 512, 512)
    assert [(args[9], args[11]) for _, args in calls] == [(512, 512)] * 2


def test_rope_takes_a_buffer_of_another_shape_as_the_numbers_say(calls):
    """The first element of the rows, or the buffer that holds them."""
    import torch
    x = torch.zeros(3 * 512, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    for q, k in ((x, x[256:]), (x[0], x[256]), (x.view(3, 512), x.view(3, 512)[:, 256:])):
        tm.tm_rope_fwd(q, q, k, k, 3, 1, 4, 2, 64, 512, 512, 512, 512, 64, 0, 0, f, 1.0, None, 0)
    assert all(args[0] == x.data_ptr() and args[9:13] == (512,) * 4 for _, args in calls) and len(calls) == 3


def test_rope_refuses_rows_that_are_elsewhere(calls):
    q, k, _ = packed(3, 5, 4, 2, 64)
    for bad in [lambda: rope(q, k, 256, 512), lambda: rope(q, k, 512, 1024),
                lambda: rope(q[:, :4], k[:, :4], 512, 512),          # batches do not follow each other
                lambda: rope(q[:, :1], k[:, :1], 256, 512)]:
        with pytest.raises(ValueError, match="apart"):
            bad()
    rope(q[:, :1], k[:, :1], 512, 512)      # one row each: five packed rows apart
    assert [(args[9], args[11]) for _, args in calls] == [(2560, 2560)]


def append(k, v, k_stride, v_stride, n=None):
    import torch
    B, n_src, H, D = k.shape
    i32, page = torch.zeros(B, dtype=torch.int32), torch.zeros((4, H, 16, D), dtype=torch.int8)
    r = torch.zeros((4, H))
    tm.tm_kv8_append(k, v, k_stride, v_stride, B, n_src, n or n_src, H, D, None, None, i32,
                     i32.view(B, 1), 1, page, page, r, r, 4, 16, 0)


def test_append_of_one_token_passes_the_stride_between_sequences(calls):
    _, k, v = packed(3, 1, 4, 2, 64)
    append(k, v, k.stride(1), v.stride(1))
    append(k, v, 512, v.stride(0))
    _, k, v = packed(3, 5, 4, 2, 64)
    append(k, v, 512, 512, 4)
    append(k[:, 2:3], v[:, :1], 512, 2560)
    assert [args[2:4] for _, args in calls] == [(512, 512)] * 3 + [(2560, 2560)]


def test_append_refuses_rows_that_are_elsewhere(calls):
    _, k, v = packed(3, 5, 4, 2, 64)
    for bad in [lambda: append(k, v, 128, 512), lambda: append(k, v, 512, 128),
                lambda: append(k[:, :4], v[:, :4], 512, 512), lambda: append(k[:, :1], v[:, :1], 2560, 128)]:
        with pytest.raises(ValueError, match="apart"):
            bad()
    assert not calls


class Slice:
    """What the binding asks of a tensor on the current device, here of a host one."""

    def __init__(self, x):
        self.x = x

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.x, name)


def test_a_slice_that_no_stride_describes_is_refused(monkeypatch):
    """One token's positions out of a longer table, some columns of a page table, q of one token
    out of a packed projection: the library would read the rows between."""
    import torch
    made = []
    monkeypatch.setattr(tm, "_device", lambda: 0)
    monkeypatch.setattr(tm, "_stream", lambda s: 0)
    library = type("Library", (), {"__getattr__": lambda self, name: lambda *a: made.append(name) or 0})()
    monkeypatch.setattr(tm, "lib", lambda: library)
    q, k, v = (Slice(t) for t in packed(3, 1, 4, 2, 64))
    dense = [Slice(torch.zeros(t.x.shape, dtype=torch.bfloat16)) for t in (q, k)]
    f = Slice(torch.zeros(32, dtype=torch.float64))
    wide = torch.zeros((3, 8), dtype=torch.int32)
    i32, page = Slice(torch.zeros(3, dtype=torch.int32)), Slice(torch.zeros((4, 2, 16, 64), dtype=torch.int8))
    r, w = Slice(torch.zeros((4, 2))), Slice(torch.zeros((3, 2, 64)))

    def rope(positions):
        tm.tm_rope_fwd(q, dense[0], k, dense[1], 3, 1, 4, 2, 64, 512, 256, 512, 128, 64, 0, 0, f, 1.0,
                       positions, 0)

    def append(table):
        tm.tm_kv8_append(k, v, 512, 512, 3, 1, 1, 2, 64, None, None, i32, table, 4, page, page, r, r, 4,
                         16, 0)

    def attend(q, table):
        tm.tm_kv8_attn_fwd(q, dense[0], 3, 1, 4, 2, 64, 0.125, page, page, r, r, 4, 16, 0, table, 4, i32,
                           None, 0, 0, w, 1024)

    def select(weights):
        tm.tm_kv_select(weights, 32, None, 3, 2, 32, 4, 0, 0, w, None)

    few = Slice(wide[:, :4].contiguous())
    rope(Slice(wide[:, :1].contiguous()))
    append(few)
    attend(dense[0], few)
    select(Slice(w.x[..., :32].contiguous()))
    assert made == ["tm_rope_fwd", "tm_kv8_append", "tm_kv8_attn_fwd", "tm_kv_select"]
    for bad in [lambda: rope(Slice(wide[:, 2:3])), lambda: append(Slice(wide[:, :4])),
                lambda: attend(dense[0], Slice(wide[:, :4])), lambda: attend(q, few),
                lambda: select(Slice(w.x[..., :32])),
                lambda: tm.tm_key_weights_fwd(q, dense[1], 3, 4, 2, 1, 64, 0.125, 1, None, w, 64, 0, w, 1024)]:
        with pytest.raises(ValueError, match="contiguous"):
            bad()
    assert len(made) == 4
