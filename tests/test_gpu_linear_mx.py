"""moe_linear_mxfp4 against the 64-bit definition on the same MXFP4 values.

Bounds, element by element.  A product of two E2M1 values and their scales is
exact; sums are kept in fp32.  With S the sum of the magnitudes, K/64
instructions whose partial sums stay around S/sqrt(K) and lose at most 2^-23 of
themselves each are off by less than 2^-20 S up to K = 16384 (sums of one sign:
chains of at most 32 instructions, whose partial sums are S/2 on average, and a
few chains: 2^-18 S).  Activations as in test_gpu_linear.py: a few units of
2^-22 of max(|z|, 1), a slope of at most 1.13.  The output's type adds half a
unit (torch.finfo's eps / 2) or half the spacing of subnormals."""
import numpy as np
import pytest
import torch

from oracle import block as D

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
HALF = {t: (torch.finfo(t).eps / 2, torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2)
        for t in (BF, F16, F32)}


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return amp * torch.randn(*shape, generator=g)


def _wide(t, pad, dtype):
    if not pad:
        return t.to("cuda", dtype)
    w = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    w[:, :t.shape[1]] = t.to("cuda", dtype)
    return w[:, :t.shape[1]]


def _f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _rows(t):
    """MXFP4 rows of t, the scale bytes of rows past the last set to NaN."""
    R, K = t.shape
    q = B.quantize_rows_mxfp4(t.cuda())
    blocks = (K + 127) // 128 * 4
    used = torch.from_numpy(D.mx_pack(np.zeros((R, 32 * blocks), np.uint8),
                                      np.ones((R, blocks), np.uint8))[1]).cuda()
    q.scales[used == 0] = 255
    return q


def _values(q):
    return D.mx_values(*D.mx_unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy()))


def _within(got, ref, tol):
    rel, small = HALF[got.dtype]
    err = np.abs(_f64(got) - ref)
    bound = tol + rel * (np.abs(ref) + tol) + small
    assert np.all(err <= bound), float(np.max(err / bound))


def _check(T, K, N, act="none", out=BF, bias=True, res=True, pad=0, seed=0, sums=2.0 ** -20,
           one_sign=False):
    x, W = _rand(seed, T, K), _rand(seed + 1, N, K, amp=K ** -0.5)
    if one_sign:
        x, W = x.abs(), W.abs()
    x, W = _rows(x), _rows(W)
    b = _rand(seed + 2, N).cuda() if bias else None
    r = _wide(_rand(seed + 3, T, N), pad, out) if res else None
    y = _wide(torch.zeros(T, N), pad, out)
    assert B.linear_mxfp4(x, W, bias=b, residual=r, act=act, y=y) is y
    xd, Wd = _values(x), _values(W)
    ref, z = D.linear_mx(xd, Wd, _f64(b), _f64(r), act)
    tol = sums * (np.abs(xd) @ np.abs(Wd).T + (0 if b is None else np.abs(_f64(b))))
    _within(y, ref, 1.13 * tol + 2.0 ** -20 * np.maximum(np.abs(z), 1.0) * (act != "none")
            + 2.0 ** -23 * (0 if r is None else np.abs(_f64(r))))
    return y


@pytest.mark.parametrize("T,K,N", [
    (1, 32, 1), (1, 64, 8), (20, 96, 40), (31, 1024, 70), (40, 10240, 300), (64, 5376, 64), (1, 96, 130), (2, 128, 3), (7, 160, 16), (15, 256, 127), (16, 288, 128),
    (17, 512, 129), (32, 544, 100), (33, 1024, 300), (64, 1056, 64), (65, 2560, 200),
    (127, 800, 256), (128, 2560, 520), (1, 2560, 1024), (16, 10240, 256), (1, 11264, 40)])
@pytest.mark.parametrize("out", [BF, F32])
def test_few_rows(T, K, N, out):
    _check(T, K, N, out=out)


@pytest.mark.parametrize("T,K,N", [
    (129, 32, 1), (130, 96, 257), (200, 256, 100), (255, 288, 255), (256, 512, 256), (257, 1056, 300),
    (300, 2560, 64), (513, 544, 520), (777, 1056, 1001), (1024, 2560, 512), (600, 4096, 96)])
@pytest.mark.parametrize("out", [BF, F16, F32])
def test_many_rows(T, K, N, out):
    _check(T, K, N, out=out, pad=8 if N % 8 == 0 else 3)


@pytest.mark.parametrize("out", [BF, F16, F32])
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_wide_tiles_several_a_pair(out, act):
    """Three rounds of tiles of 256 columns: accumulators that share columns, in turn."""
    _check(2049, 512, 5900, act=act, out=out, res=False)


@pytest.mark.parametrize("K,out,pad", [(2560, BF, 8), (2560, F16, 3), (11264, F32, 0), (11264, F32, 1)])
def test_wide_tiles_with_a_residual(K, out, pad):
    _check(1000, K, 4850, out=out, pad=pad)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [5, 40, 300])
@pytest.mark.parametrize("out", [BF, F16, F32])
def test_activations(act, T, out):
    _check(T, 320, 200, act=act, out=out)


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("T", [20, 140])
def test_epilogues(bias, res, pad, T):
    _check(T, 256, 136, bias=bias, res=res, pad=pad)
    _check(T, 256, 136, bias=bias, res=res, pad=pad, out=F32)


@pytest.mark.parametrize("T", [3, 60, 128, 400])
@pytest.mark.parametrize("K", [2560, 11264, 16384])
def test_sums_of_one_sign(T, K):
    y = _check(T, K, 96, out=F32, bias=False, res=False, one_sign=True, sums=2.0 ** -18)
    assert torch.isfinite(y).all()


def test_every_block_has_its_own_scale():
    """A one in one place of x against W with a scale of its own in each block
    reads every scale and code of W back."""
    K, N = 416, 200
    g = torch.Generator().manual_seed(1)
    W = torch.randn(N, K, generator=g) * 2.0 ** torch.randint(-9, 9, (N, K // 32), generator=g
                                                              ).repeat_interleave(32, 1)
    W = _rows(W)
    for T in (K, 40):
        x = torch.zeros(T, K)
        at = torch.arange(T) * (K // T)
        x[torch.arange(T), at] = 2.0 ** (torch.arange(T) % 12 - 6).float()
        y = B.linear_mxfp4(_rows(x), W, out_dtype=F32)
        want = (_values(W)[:, at] * 2.0 ** (np.arange(T) % 12 - 6)).T
        assert np.array_equal(_f64(y), want)


@pytest.mark.parametrize("T", [1, 2, 7, 15, 16, 17, 40, 300])
@pytest.mark.parametrize("K", [32, 96, 640, 2560, 2816])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_rows_quantised_by_the_call(T, K, dtype):
    """Bit for bit what the product of the quantised rows is, whichever kernel
    quantises them, with NaN and infinite values too."""
    W = _rows(_rand(1, 300, K, amp=0.05))
    for pad in (0, 3, 8):
        x = _wide(_rand(2, T, K) * torch.exp(3 * _rand(3, T, K // 32)).repeat_interleave(32, 1), pad,
                  dtype)
        x[0, 5] = 0.0
        if T > 2:
            x[1, K - 1] = float("nan")
            x[2, 3] = float("inf")
        y = B.linear_mxfp4(x, W, act="relu", out_dtype=dtype)
        assert y.dtype == dtype
        q = B.quantize_rows_mxfp4(x)
        want = B.linear_mxfp4(q, W, act="relu", out_dtype=dtype)
        assert torch.equal(y.isnan(), want.isnan())
        assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))
        need = B.linear_rows_mxfp4_workspace_bytes(T, K, 300)
        assert (need == 0) == (T <= 16)
        if need:
            ws = torch.empty(need, dtype=torch.uint8, device="cuda")
            again = B.linear_mxfp4(x, W, act="relu", out_dtype=dtype, ws=ws)
            assert torch.equal(again.nan_to_num(7.0), want.nan_to_num(7.0))
            with pytest.raises(B.MoeError):
                B.linear_mxfp4(x, W, ws=ws[:-1])


@pytest.mark.parametrize("T,K,N", [(1, 2560, 10240), (16, 10240, 2560), (16, 11264, 11264),
                                   (3, 65536, 40), (16, 2048, 20000), (1, 11264, 2816)])
def test_few_rows_of_large_products(T, K, N):
    """Among them products whose rows are too long for the kernel to quantise."""
    x = _rand(1, T, K).to("cuda", BF)
    W = B.quantize_rows_mxfp4((_rand(2, 64, K, amp=K ** -0.5)).cuda())
    many = B.Mxfp4Rows(W.codes.repeat((N + 63) // 64, 1)[:N].contiguous(), None)
    scales = W.scales.view(1, -1, 32, 4, 4)[:, :, :, :2].repeat(1, 1, 1, 2, 1)  # rows 64 ... are 0 ...
    scales = scales.reshape(1, -1, 512).repeat((N + 127) // 128, 1, 1).contiguous()
    many = B.Mxfp4Rows(many.codes, scales)
    res = _rand(3, T, N).cuda()
    y = B.linear_mxfp4(x, many, residual=res, out_dtype=F32)
    q = B.quantize_rows_mxfp4(x)
    assert torch.equal(y, B.linear_mxfp4(q, many, residual=res, out_dtype=F32))
    xd, Wd = _values(q), _values(W)
    ref = np.tile(xd @ Wd.T, (1, (N + 63) // 64))[:, :N] + _f64(res)
    size = np.tile(np.abs(xd) @ np.abs(Wd).T, (1, (N + 63) // 64))[:, :N]
    _within(y, ref, 2.0 ** -19 * size + 2.0 ** -23 * np.abs(_f64(res)))


def test_extreme_scales():
    x, W = torch.zeros(40, 64), torch.zeros(50, 64)
    x[:, 0], W[:, 0] = 2.0 ** 100, 2.0 ** -126
    x[:, 40], W[:, 40] = 2.0 ** -126, 2.0 ** 100
    x[0] = 0
    y = B.linear_mxfp4(_rows(x), _rows(W), out_dtype=F32)
    assert not y[0].any() and (y[1:] == 2.0 ** -25).all()


def test_a_nan_block_stays_in_its_row():
    x, W = _rand(1, 200, 320), _rand(2, 70, 320)
    for T in (5, 200):
        clean = B.linear_mxfp4(_rows(x[:T]), _rows(W), out_dtype=F32)
        bad = x[:T].clone()
        bad[3, 100] = float("nan")
        bad[4, 319] = float("inf")
        y = B.linear_mxfp4(_rows(bad), _rows(W), out_dtype=F32)
        assert torch.isnan(y[3:5]).all()
        keep = [t for t in range(T) if t not in (3, 4)]
        assert torch.equal(y[keep], clean[keep])


def test_a_nan_block_of_a_weight_stays_in_its_column():
    x, W = _rand(1, 300, 320), _rand(2, 300, 320)
    bad = W.clone()
    bad[7, 300] = float("nan")
    bad[250, 0] = -float("inf")
    keep = [n for n in range(300) if n not in (7, 250)]
    for T in (5, 100, 300):
        clean = B.linear_mxfp4(_rows(x[:T]), _rows(W), out_dtype=F32)
        y = B.linear_mxfp4(_rows(x[:T]), _rows(bad), out_dtype=F32)
        assert torch.isnan(y[:, [7, 250]]).all() and torch.equal(y[:, keep], clean[:, keep])


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("out", [BF, F32])
def test_many_chains(T, out):
    """More of K than one accumulator sums of an fp32 output."""
    _check(T, 16640, 130, out=out)
    _check(T, 40000, 20, out=out, bias=False, res=False)


@pytest.mark.parametrize("T", [9, 200])
@pytest.mark.parametrize("out", [BF, F32])
def test_rows_that_start_anywhere(T, out):
    x = _rand(1, T, 321).to("cuda", BF)[:, 1:]
    W = _rows(_rand(2, 72, 320))
    r, y = _rand(3, T, 75).to("cuda", out)[:, 1:73], torch.zeros(T, 75, dtype=out, device="cuda")
    B.linear_mxfp4(x, W, residual=r, y=y[:, 3:])
    want = B.linear_mxfp4(x.contiguous(), W, residual=r.contiguous(), out_dtype=out)
    assert torch.equal(y[:, 3:], want) and not y[:, :3].any()


def test_residual_in_place_and_rows_left_alone():
    x, W = _rand(1, 200, 320), _rows(_rand(2, 72, 320))
    for T in (5, 200):
        for dtype in (BF, F32):
            r = _rand(3, T + 4, 80).to("cuda", dtype)
            want = B.linear_mxfp4(_rows(x[:T]), W, residual=r[:T, :72].clone(), out_dtype=dtype)
            keep = r.clone()
            y = r[:T, :72]
            B.linear_mxfp4(_rows(x[:T]), W, residual=y, y=y)
            assert torch.equal(y, want)
            assert torch.equal(r[T:], keep[T:]) and torch.equal(r[:, 72:], keep[:, 72:])


@pytest.mark.parametrize("T", [129, 143, 144, 145, 271, 272])
@pytest.mark.parametrize("out", [BF, F32])
def test_residual_of_a_few_rows_of_a_tile(T, out):
    """Warps whose 32 rows end in their first or second half."""
    _check(T, 128, 200, out=out, bias=False)


def test_the_same_bits_every_time():
    x, W = _rows(_rand(1, 1000, 2560)), _rows(_rand(2, 700, 2560))
    y = B.linear_mxfp4(x, W, out_dtype=F32)
    few = B.linear_mxfp4(_rows(_rand(1, 1000, 2560)[:9]), W, out_dtype=F32)
    for _ in range(5):
        assert torch.equal(B.linear_mxfp4(x, W, out_dtype=F32), y)
        assert torch.equal(B.linear_mxfp4(_rows(_rand(1, 1000, 2560)[:9]), W, out_dtype=F32), few)
    assert B.take_status() == 0


def test_no_rows_and_refusals():
    W = _rows(_rand(2, 70, 320))
    assert B.linear_mxfp4(torch.empty(0, 320, dtype=BF, device="cuda"), W).shape == (0, 70)
    x = _rand(1, 4, 320).to("cuda", BF)
    for bad in (dict(x=x[:, :288]), dict(x=x.double()), dict(x=x.cpu()), dict(act="tanh"),
                dict(bias=torch.zeros(69, device="cuda")), dict(out_dtype=torch.int32),
                dict(residual=torch.zeros(4, 70, device="cuda")), dict(y=x[:, :69]),
                dict(x=B.Mxfp4Rows(W.codes[:4], W.scales[:0]))):
        with pytest.raises(ValueError):
            B.linear_mxfp4(**{**dict(x=x, W=W), **bad})
