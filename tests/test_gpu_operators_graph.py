"""linear, linear_grad, route and route_grad captured in one CUDA graph and
replayed on new inputs, and run from several threads on streams of their own:
the same bits as eager calls on the current stream."""
import threading

import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def _rand(seed, *shape, amp=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (amp * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def _inputs(T, d, E, h, dtype, seed):
    return {"x": _rand(seed, T, d, dtype=dtype), "Wr": _rand(seed + 1, E, d, amp=0.05, dtype=dtype),
            "up": _rand(seed + 2, h, d, amp=0.05, dtype=dtype),
            "down": _rand(seed + 3, d, h, amp=0.05, dtype=dtype),
            "bias": _rand(seed + 4, E, amp=0.1), "dy": _rand(seed + 5, T, d, amp=1e-3, dtype=dtype),
            "mask": torch.arange(T, device="cuda") % 5 != seed % 5}


def _run(s, k):
    """Every operator, as a block and its backward pass would call them."""
    logits = B.linear(s["x"], s["Wr"], out_dtype=F32)
    r = B.route(logits, k, bias=s["bias"], mask=s["mask"], score="sigmoid")
    lean = B.route(logits, k, stats=False)
    pre = torch.empty((s["x"].shape[0], s["up"].shape[0]), dtype=s["x"].dtype, device="cuda")
    hid = B.linear(s["x"], s["up"], act="gelu", pre=pre)
    y = B.linear(hid, s["down"], residual=s["x"])
    dh, ddown, _ = B.linear_grad(hid, s["down"], s["dy"], need=(True, True, False))
    dx, dup, db = B.linear_grad(s["x"], s["up"], dh, pre=pre, act="gelu")
    dl = B.route_grad(logits, r["ids"], r["counts"], dw=r["w"], dloss=r["loss"], mask=s["mask"],
                      score="sigmoid")
    gx, gW, gb = B.linear_grad(s["x"], s["Wr"], dl, dw_dtype=F32)
    return [logits, r["ids"], r["w"], r["counts"], r["prob"], r["loss"], lean["ids"], lean["w"],
            hid, y, dh, ddown, dx, dup, db, dl, gx, gW, gb]


SHAPES = [(1, 128, 16, 64, 2, BF), (100, 264, 72, 328, 6, F16), (600, 520, 200, 1032, 8, BF),
          (2048, 1024, 512, 2048, 10, BF)]


@pytest.mark.parametrize("T,d,E,h,k,dtype", SHAPES)
def test_replays_match_eager_calls(T, d, E, h, k, dtype):
    sets = [_inputs(T, d, E, h, dtype, seed) for seed in (10, 20)]
    want = [[t.clone() for t in _run(s, k)] for s in sets]
    s = {n: t.clone() for n, t in sets[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # first calls outside the capture
        _run(s, k)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _run(s, k)
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
    sets = [_inputs(*shape[:4], shape[5], 30 + i) for i, shape in enumerate(SHAPES)]
    want = [[t.clone() for t in _run(s, shape[4])] for s, shape in zip(sets, SHAPES)]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(10):
                got = _run(sets[i], SHAPES[i][4])
                stream.synchronize()
                wrong.extend((i, j) for j, (a, b) in enumerate(zip(got, want[i]))
                             if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(SHAPES))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and B.take_status() == 0
