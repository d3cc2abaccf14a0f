"""moe_linear and moe_linear_grad against the 64-bit definitions.

Bounds, element by element.  Products of two 16-bit values are exact in fp32
and a sum of R of them is kept in fp32: with S the sum of the magnitudes, a
chain of R/16 additions whose partial sums stay around S/sqrt(R) and lose at
most 2^-23 of themselves each is off by less than 2^-20 S up to R = 16384.
Activations and their gradients are computed in fp32 to a few units of
2^-22 of max(|z|, 1), and a slope of at most 1.13 carries z's error.  The
output's type adds half a unit: torch.finfo's eps / 2 (2^-8 of bf16's 8
significant bits, 2^-11 of fp16's 11, 2^-24 of fp32's) or, for subnormals,
half their spacing.  Where dP is rounded for the products,
each of its values is off by that half unit."""
import numpy as np
import pytest
import torch

from oracle import router as R

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
HALF = {t: (torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)
        for t in (torch.bfloat16, torch.float16, torch.float32)}


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return amp * torch.randn(*shape, generator=g)


def _wide(t, pad, dtype):
    """t on the GPU as the first columns of a wider tensor."""
    if not pad:
        return t.to("cuda", dtype)
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    w[:, :t.shape[1]] = t.to("cuda", dtype)
    return w[:, :t.shape[1]]


def _f64(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, tol, dtype):
    rel, small = HALF[dtype]
    err = np.abs(_f64(got) - ref)
    bound = tol + rel * (np.abs(ref) + tol) + small
    assert np.all(err <= bound), float(np.max(err / bound))


def _check_linear(T, K, N, act, dtype, out, bias=True, res=True, pre=True, pad=0, seed=0):
    x = _wide(_rand(seed, T, K), pad, dtype)
    W = _rand(seed + 1, N, K, amp=K ** -0.5).to("cuda", dtype)
    b = _rand(seed + 2, N).cuda() if bias else None
    r = _wide(_rand(seed + 3, T, N), pad, out) if res else None
    p = torch.full((T, N), float("nan"), dtype=dtype, device="cuda") if pre else None
    y = B.linear(x, W, bias=b, residual=r, act=act, out_dtype=out, pre=p)
    assert y.dtype == out and tuple(y.shape) == (T, N)
    xd, Wd = _f64(x), _f64(W)
    ref, z = R.linear(xd, Wd, None if b is None else _f64(b), None if r is None else _f64(r), act)
    tol = 2.0 ** -20 * (np.abs(xd) @ np.abs(Wd).T + (0 if b is None else np.abs(_f64(b))))
    if p is not None:
        _within(p, z, tol, dtype)
    _within(y, ref, 1.13 * tol + 2.0 ** -20 * np.maximum(np.abs(z), 1.0), out)


@pytest.mark.parametrize("T,K,N", [
    (1, 8, 1), (1, 2560, 512), (2, 64, 3), (7, 72, 16), (15, 136, 127), (16, 128, 128),
    (17, 1024, 130), (31, 40, 257), (33, 192, 129), (63, 520, 64), (65, 64, 8), (100, 4096, 96),
    (127, 200, 384), (129, 2560, 512), (300, 1032, 1001), (777, 264, 100)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear_shapes(T, K, N, dtype):
    _check_linear(T, K, N, "silu", dtype, dtype, pad=24)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear_epilogues(act, out):
    _check_linear(70, 512, 200, act, torch.bfloat16, out)
    _check_linear(9, 1536, 300, act, torch.bfloat16, out, bias=False, res=False, pre=False)


@pytest.mark.parametrize("act", ACTS)
def test_activation_values(act):
    # every bf16 value from 2^-20 to 2^6, of both signs, through an identity
    # product.  GELU's erf is a formula good to 1.5e-7, so its factor of z to
    # half of that; the others' factors to a few units of 2^-24
    bits = torch.arange(0x3580, 0x4280, dtype=torch.int32)
    z = torch.cat([bits, bits | 0x8000]).to(torch.int16).view(torch.bfloat16)
    z = z[:z.numel() // 16 * 16].reshape(-1, 16)
    y = B.linear(z.cuda(), torch.eye(16, dtype=torch.bfloat16, device="cuda"), act=act,
                 out_dtype=torch.float32)
    ref = R.act(_f64(z), act)
    assert np.all(np.abs(_f64(y) - ref) <= (0.75e-7 + 2.0 ** -21) * np.abs(_f64(z)))
    one = torch.ones(z.shape, dtype=torch.float32, device="cuda")
    _, _, db = B.linear_grad(z.cuda(), torch.eye(16, dtype=torch.bfloat16, device="cuda"), one[:1]
                             .expand(z.shape).contiguous(), pre=z.cuda(), act=act,
                             need=(False, False, True))
    want = R.act_grad(_f64(z), act).sum(0)
    assert np.all(np.abs(_f64(db) - want) <= (0.75e-7 + 2.0 ** -20) * np.maximum(
        1.0, np.abs(_f64(z))).sum(0))


def test_linear_large_tiles():
    # more tiles than CTAs fit at once, ragged in both directions
    _check_linear(2050, 256, 2600, "gelu_tanh", torch.bfloat16, torch.bfloat16)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", [torch.float16, torch.float32])
def test_linear_256_wide_tiles(act, out):
    # enough 256 x 256 tiles for pairs of CTAs, with odd edges and short reductions
    _check_linear(2321, 72, 2309, act, torch.float16, out, pad=40)


def test_linear_256_wide_tiles_long_reduction():
    _check_linear(2304, 4104, 2304, "none", torch.bfloat16, torch.bfloat16, bias=False, res=False)


@pytest.mark.parametrize("N,dtype,out", [
    (3000, torch.bfloat16, torch.bfloat16), (3001, torch.float16, torch.float32),
    (3001, torch.bfloat16, torch.bfloat16), (3000, torch.float16, torch.float32)])
def test_linear_tiles_of_two_widths(N, dtype, out):
    # just above a whole number of rounds of tiles: the last columns go to narrower ones
    _check_linear(2321, 1032, N, "silu", dtype, out, pad=8)
    _check_linear(2321, 1032, N, "none", dtype, out, bias=False, res=False, pre=False)


def test_linear_adds_into_its_output():
    x = _rand(1, 40, 320).to("cuda", torch.bfloat16)
    W = _rand(2, 90, 320, amp=0.05).to("cuda", torch.bfloat16)
    y = _rand(3, 40, 90).to("cuda", torch.bfloat16)
    want = B.linear(x, W, residual=y.clone())
    got = B.linear(x, W, residual=y, y=y)
    assert got.data_ptr() == y.data_ptr()
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_linear_keeps_nan_and_infinity_in_their_rows():
    x = _rand(1, 20, 128).to("cuda", torch.bfloat16)
    W = _rand(2, 150, 128, amp=0.1).to("cuda", torch.bfloat16)
    clean = B.linear(x, W, act="relu")
    x[3, 5] = float("nan")
    x[11, 100] = float("inf")
    y = B.linear(x, W, act="relu")
    other = [t for t in range(20) if t not in (3, 11)]
    assert torch.equal(y[other], clean[other])
    assert bool(y[3].isnan().all())
    inf = W[:, 100].float() > 0
    assert bool(y[11][inf].isinf().all()) and bool((y[11][~inf] == 0).all())


def test_linear_no_tokens():
    W = _rand(2, 30, 64).to("cuda", torch.bfloat16)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert tuple(B.linear(x, W).shape) == (0, 30)
    dx, dW, db = B.linear_grad(x, W, torch.empty((0, 30), dtype=torch.bfloat16, device="cuda"))
    assert tuple(dx.shape) == (0, 64) and bool((dW == 0).all()) and bool((db == 0).all())


def test_linear_output_beyond_31_bit_offsets():
    T, K, N = 70000, 8, 32768  # 2.29e9 outputs
    x = _rand(1, T, K).to("cuda", torch.bfloat16)
    W = _rand(2, N, K).to("cuda", torch.bfloat16)
    y = B.linear(x, W)
    for t in (0, 1, 65535, 65536, 69998, 69999):
        ref, _ = R.linear(_f64(x[t:t + 1]), _f64(W))
        tol = 2.0 ** -20 * (np.abs(_f64(x[t:t + 1])) @ np.abs(_f64(W)).T)
        _within(y[t:t + 1], ref, tol, torch.bfloat16)


def test_linear_on_another_stream_and_again():
    x = _rand(1, 500, 1024).to("cuda", torch.bfloat16)
    W = _rand(2, 512, 1024, amp=0.03).to("cuda", torch.bfloat16)
    want = B.linear(x, W, out_dtype=torch.float32)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [B.linear(x, W, out_dtype=torch.float32) for _ in range(5)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)  # one order of every sum


def _check_grad(T, K, N, act, dtype, dy_dtype, dw_dtype, pad=0, seed=0):
    x = _wide(_rand(seed, T, K), pad, dtype)
    W = _rand(seed + 1, N, K, amp=0.05).to("cuda", dtype)
    dy = _wide(_rand(seed + 2, T, N, amp=0.1), pad, dy_dtype)
    pre = None if act == "none" else _rand(seed + 3, T, N, amp=2.0).to("cuda", dtype)
    dx, dW, db = B.linear_grad(x, W, dy, pre=pre, act=act, dw_dtype=dw_dtype)
    xd, Wd, dyd = _f64(x), _f64(W), _f64(dy)
    pd = None if pre is None else _f64(pre)
    rx, rw, rb = R.linear_grad(xd, Wd, dyd, pd, act)
    slope = np.ones_like(dyd) if pd is None else R.act_grad(pd, act)
    adp = np.abs(dyd * slope)
    # dP itself: a few units of 2^-22 of dy max(|pre|, 1), then the rounding to dtype
    fp = np.zeros_like(adp) if act == "none" else 2.0 ** -20 * np.abs(dyd) * np.maximum(
        1.0, np.abs(pd))
    rel, small = HALF[dtype]
    rounded = act != "none" or dy_dtype != dtype
    op = fp + (rel * adp + small if rounded else 0.0)
    _within(dx, rx, op @ np.abs(Wd) + 2.0 ** -20 * (adp @ np.abs(Wd)), dtype)
    _within(dW, rw, op.T @ np.abs(xd) + 2.0 ** -20 * (adp.T @ np.abs(xd)), dw_dtype)
    _within(db, rb, fp.sum(0) + 2.0 ** -20 * adp.sum(0), torch.float32)


@pytest.mark.parametrize("T,K,N", [
    (1, 8, 1), (1, 256, 40), (5, 72, 3), (16, 64, 16), (31, 136, 127), (64, 64, 64),
    (65, 200, 129), (130, 1032, 33), (257, 128, 1001), (1000, 264, 70)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_linear_grad_shapes(T, K, N, dtype):
    _check_grad(T, K, N, "gelu_tanh", dtype, dtype, dtype, pad=8)
    _check_grad(T, K, N, "none", dtype, dtype, torch.float32, pad=8)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dy_dtype", [torch.bfloat16, torch.float32])
def test_linear_grad_epilogues(act, dy_dtype):
    _check_grad(90, 320, 150, act, torch.bfloat16, dy_dtype, torch.bfloat16)


def test_linear_grad_large_tiles():
    _check_grad(1500, 520, 1300, "silu", torch.bfloat16, torch.bfloat16, torch.bfloat16)


def test_linear_grad_256_wide_tiles():
    _check_grad(2300, 2312, 2201, "gelu", torch.bfloat16, torch.bfloat16, torch.bfloat16, pad=8)
    _check_grad(1000, 4104, 2600, "none", torch.float16, torch.float16, torch.float32)


def test_linear_grad_tiles_of_two_widths():
    T, K, N = 2100, 2600, 264
    x = _rand(0, T, K).to("cuda", torch.bfloat16)
    W = _rand(1, N, K, amp=0.05).to("cuda", torch.bfloat16)
    dy = _rand(2, T, N, amp=0.1).to("cuda", torch.bfloat16)
    dx, _, db = B.linear_grad(x, W, dy, need=(True, False, True))
    Wd, dyd = _f64(W), _f64(dy)
    _within(dx, dyd @ Wd, 2.0 ** -20 * (np.abs(dyd) @ np.abs(Wd)), torch.bfloat16)
    _within(db, dyd.sum(0), 2.0 ** -20 * np.abs(dyd).sum(0), torch.float32)


def test_linear_grad_computes_what_is_asked():
    x = _rand(1, 40, 64).to("cuda", torch.bfloat16)
    W = _rand(2, 24, 64).to("cuda", torch.bfloat16)
    dy = _rand(3, 40, 24).cuda()
    full = B.linear_grad(x, W, dy)
    for i in range(3):
        need = tuple(j == i for j in range(3))
        got = B.linear_grad(x, W, dy, need=need)
        assert [g is not None for g in got] == list(need)
        assert torch.equal(got[i], full[i])


def test_linear_against_differences_of_itself():
    # the directional derivative of sum(dy * y) along random dx, dW, db:
    # fp32 outputs of bf16 inputs moved by a bf16-exact step h = 2^-3 in each
    # of the three alone; the function is linear in each (act none), so the
    # difference has no truncation error and only fp32 sums' rounding
    T, K, N, h = 24, 96, 40, 2.0 ** -3
    q = lambda s, *shape: torch.round(_rand(s, *shape) * 16).clamp(-32, 32) / 16  # noqa: E731
    x, W = (q(s, *sh).to("cuda", torch.bfloat16) for s, sh in ((1, (T, K)), (2, (N, K))))
    dy = q(3, T, N).to("cuda", torch.bfloat16)
    dx, dW, db = B.linear_grad(x, W, dy, dw_dtype=torch.float32)
    vx, vW = (q(s, *sh).to("cuda", torch.bfloat16) for s, sh in ((4, (T, K)), (5, (N, K))))
    vb = q(6, N).cuda()
    y = lambda a, b, c: (B.linear(a, b, bias=c, out_dtype=torch.float32).double()  # noqa: E731
                         * dy.double()).sum()
    zero = torch.zeros(N, device="cuda")
    for up, down, grad, v in ((y(x + h * vx, W, zero), y(x - h * vx, W, zero), dx, vx),
                              (y(x, W + h * vW, zero), y(x, W - h * vW, zero), dW, vW),
                              (y(x, W, h * vb), y(x, W, -h * vb), db, vb)):
        want = float((up - down) / (2 * h))
        got = float((grad.double() * v.double()).sum())
        mag = float((grad.double().abs() * v.double().abs()).sum())
        assert abs(got - want) <= 2.0 ** -8 * mag  # dx comes in bf16


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.zeros((10, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        B.linear(x, W[:, :56])
    with pytest.raises(ValueError, match="contiguous"):
        B.linear(x, torch.zeros((64, 10), dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(ValueError, match="contiguous rows"):
        B.linear(torch.zeros((64, 4), dtype=torch.bfloat16, device="cuda").t(), W)
    with pytest.raises(ValueError, match="dtype"):
        B.linear(x, W.half())
    with pytest.raises(ValueError, match="residual"):
        B.linear(x, W, residual=torch.zeros((4, 10), device="cuda"))
    with pytest.raises(ValueError, match="act"):
        B.linear(x, W, act="tanh")
    with pytest.raises(B.MoeError) as e:  # rows that are no multiple of 16 bytes apart
        B.linear(torch.zeros((4, 68), dtype=torch.bfloat16, device="cuda")[:, :64], W)
    assert e.value.code == B.MOE_ERR_SHAPE
    with pytest.raises(B.MoeError) as e:
        B.linear(torch.zeros((4, 72), dtype=torch.bfloat16, device="cuda")[:, 1:65], W)
    assert e.value.code == B.MOE_ERR_ALIGN
    with pytest.raises(B.MoeError) as e:
        B.linear_grad(x, W, torch.zeros((4, 10), device="cuda"), act="silu")
    assert e.value.code == B.MOE_ERR_NULL
