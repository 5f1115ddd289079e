"""The operators around the attention in one graph with branches: kernels that start
early have several kernels ahead there, of their own stream and of others."""
import pytest

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


@pytest.mark.parametrize("captured", [False, True])
def test_branches_that_join(captured):
    """Two branches rotate and store, a third weighs a prompt's keys and selects; they join for the
    attention over both caches, again on two streams. Against the same calls one after the other."""
    import torch
    B, N, Hq, H, D, page, mp, L = 3, 200, 8, 2, 64, 16, 16, 20
    g = torch.Generator(device="cuda").manual_seed(7)

    def fresh(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)

    q, k, v = [fresh(B, N, h, D) for h in (Hq, H, H)]
    f = torch.from_numpy(tm.tm_rope_inv_freq(D, 1e4)).cuda()
    full = torch.tensor([200, 77, 1], dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(full)
    table = torch.arange(B * mp, dtype=torch.int32, device="cuda").view(B, mp)

    def run(streams):
        main = torch.cuda.current_stream()
        caches = [tm.Kv8Cache.empty(B * mp, H, page, D, fmt) for fmt in (0, 1)]
        out = {}
        for s in streams:
            s.wait_stream(main)

        def store(i):
            qr, kr = tm.rope(q, k, f, first=10 * i)
            tm.kv8_append(caches[i], kr, v, zero, table, counts=full)
            out["q", i] = qr[:, -2:].contiguous()

        def choose():
            out["w"] = tm.key_weights(q, k, L, lens=full)
            out["index"], out["kept"] = tm.kv_select(out["w"], 30, 2, 5, lens=full)

        for s, job in zip(streams, (lambda: store(0), lambda: store(1), choose)):
            with torch.cuda.stream(s):
                job()
        for s in streams:
            main.wait_stream(s)
        for i, s in enumerate(streams[:2]):   # each branch waits for all three
            s.wait_stream(main)
            with torch.cuda.stream(s):
                w = out["w"].clone()
                pad = torch.zeros((B, H, mp * page), device="cuda")
                pad[..., :N] = w
                out["o", i] = tm.kv8_attention(caches[i], out["q", i], full, table, weights=pad, accumulate=True)
                out["acc", i] = pad
        for s in streams[:2]:
            main.wait_stream(s)
        for i in range(2):
            out["codes", i] = caches[i].k8.view(torch.int8), caches[i].v_range
        return out

    def flat(out):
        return [t for key in sorted(out, key=str) for t in (out[key] if isinstance(out[key], tuple) else [out[key]])]

    streams = [torch.cuda.Stream() for _ in range(3)]
    run([torch.cuda.current_stream()] * 3)
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(streams)
    for round_ in range(3):
        for t in (q, k, v):
            t.copy_(fresh(*t.shape))
        if captured:
            for _ in range(3):
                graph.replay()
        else:
            got = run(streams)
        torch.cuda.synchronize()
        want = flat(run([torch.cuda.current_stream()] * 3))
        torch.cuda.synchronize()
        for a, b in zip(flat(got), want):
            assert torch.equal(a, b), round_
