"""block_norm, its gradient, MXFP4 rows and the MXFP4 product captured in one CUDA
graph and replayed on new inputs, and run from several threads on streams of
their own: the same bits as eager calls on the current stream."""
import threading

import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rand(seed, *shape, amp=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (amp * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def _inputs(T, d, h, S, seed):
    bt = BF if S == F32 else S
    return {"x": _rand(seed, T, d, dtype=S), "o": _rand(seed + 1, T, d, dtype=bt),
            "pre": 1 + _rand(seed + 2, d, amp=0.1), "post": 1 + _rand(seed + 3, d, amp=0.1),
            "gate": _rand(seed + 4, T), "mask": torch.arange(T, device="cuda") % 5 != seed % 5,
            "up": _rand(seed + 5, h, d, amp=0.05, dtype=BF),
            "down": _rand(seed + 6, d, h, amp=0.05, dtype=BF),
            "dxn": _rand(seed + 7, T, d, amp=1e-3, dtype=S),
            "dh": _rand(seed + 8, T, d, amp=1e-3, dtype=bt)}


def _run(s):
    """The operators as blocks one after another and a backward pass call them."""
    how = dict(pre=s["pre"], post=s["post"], gate=s["gate"], mask=s["mask"])
    n = B.block_norm(s["x"], s["o"], **how, gate_act="sigmoid", alpha=0.5, mxfp4=True)
    up, down = B.quantize_rows_mxfp4(s["up"]), B.quantize_rows_mxfp4(s["down"])
    hid = B.linear_mxfp4(n["mx"], up, act="gelu_tanh")
    y = B.linear_mxfp4(hid, down, residual=n["h"], out_dtype=n["h"].dtype)
    z = B.linear_mxfp4(n["mx"], up, out_dtype=F32)
    last = B.block_norm(n["xn"], y, post=s["post"], post_norm=False)["xn"]
    alone = B.block_norm(n["xn"], pre=s["pre"], h_dtype=y.dtype)["h"]
    g = B.block_norm_grad(n["xn"], s["o"], dxn=s["dxn"], dh=s["dh"], **how, gate_act="sigmoid",
                          alpha=0.5)
    back = B.dequantize_rows_mxfp4(n["mx"])
    return [n["xn"], n["h"], n["mx"].codes, n["mx"].scales, hid, y, z, last, alone, back,
            g["dx"], g["do"], g["dgate"], g["dpre"], g["dpost"]]


SHAPES = [(1, 128, 192, BF), (100, 256, 352, F16), (600, 544, 1056, F32), (2048, 1024, 2048, BF)]


@pytest.mark.parametrize("T,d,h,S", SHAPES)
def test_replays_match_eager_calls(T, d, h, S):
    sets = [_inputs(T, d, h, S, seed) for seed in (10, 20)]
    want = [[t.clone() for t in _run(s)] for s in sets]
    s = {n: t.clone() for n, t in sets[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first calls outside the capture
        _run(s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(s)
    for i in (1, 0, 1):
        for n, t in sets[i].items():
            s[n].copy_(t)
        for o in out:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(out, want[i])):
            assert torch.equal(a, b), (i, j)
    assert B.take_status() == 0


def test_threads_on_their_own_streams():
    sets = [_inputs(*shape, 30 + i) for i, shape in enumerate(SHAPES)]
    want = [[t.clone() for t in _run(s)] for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = _run(sets[i])
                stream.synchronize()
                wrong.extend((i, j) for j, (a, b) in enumerate(zip(got, want[i]))
                             if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(SHAPES))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and B.take_status() == 0


def test_large_sums_beside_the_16_bit_products_on_other_streams():
    """Kernels that take all of an SM's tensor memory or half of it, from two
    streams at once."""
    x, W = _rand(1, 100, 32768, dtype=BF), _rand(2, 256, 32768, amp=0.01, dtype=BF)
    q, w = B.quantize_rows_mxfp4(x), B.quantize_rows_mxfp4(W)
    a = lambda: B.linear_mxfp4(q, w, out_dtype=F32)  # noqa: E731
    b = lambda: B.linear(x, W, out_dtype=F32)  # noqa: E731
    want = a().clone(), b().clone()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        with torch.cuda.stream(one):
            got.append((a(), want[0]))
        with torch.cuda.stream(two):
            got.append((b(), want[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in got) and B.take_status() == 0
