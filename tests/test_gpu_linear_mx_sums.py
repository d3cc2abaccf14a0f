"""fp32 sums of one sign in moe_linear_mxfp4, whatever their length.

The tensor core truncates: an MMA loses half a unit of the sum so far on average, at
most 2^-24 of it.  An fp32 output's reduction is cut into chains of 64 MMAs (16 stages
of 256), whose sum so far is at most their own: 2^-18 of it, and of the whole.  Chains
and the parts of a reduction that is split over CTAs (eight at most) are added to the
nearest in fp32, and the last addition is the output: 2^-24 of the sum each."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

DRIFT = 2.0 ** -18


def _rows(seed, R, K, spread):
    """Positive values, blocks of 32 of scales up to 2^spread apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn(R, K, generator=g, device="cuda").abs()
    s = torch.randint(0, spread + 1, (R, K // 32), generator=g, device="cuda")
    return B.quantize_rows_mxfp4(v * torch.exp2(-s.float()).repeat_interleave(32, 1))


# chains of a CTA, and CTAs that share a reduction: one chain each, several, pairs of
# CTAs with chains of one tile and of several
@pytest.mark.parametrize("T,K,N,chains,parts", [
    (3, 16384, 96, 1, 8), (400, 16384, 96, 4, 1), (20, 131328, 4096, 5, 8),
    (400, 32768, 12800, 8, 1), (400, 65536, 4096, 16, 1), (70, 65536 + 96, 4224, 17, 1),
    (16, 11264, 40000, 3, 1), (50, 34816, 96, 2, 8), (2000, 4096, 3000, 1, 1),
    (2000, 4128, 3000, 2, 1)])
@pytest.mark.parametrize("spread", [0, 12])
def test_sums_of_one_sign(T, K, N, chains, parts, spread):
    x, W = _rows(1, T, K, spread), _rows(2, N, K, spread)
    y = B.linear_mxfp4(x, W, out_dtype=torch.float32)
    xd = B.dequantize_rows_mxfp4(x, torch.float32).double()
    worst = 0.0
    for n in range(0, N, 1024):
        w = B.Mxfp4Rows(W.codes[n:n + 1024], W.scales[n // 128:(n + 1024) // 128])
        ref = xd @ B.dequantize_rows_mxfp4(w, torch.float32).double().t()
        worst = max(worst, float(((y[:, n:n + 1024].double() - ref).abs() / ref).max()))
    assert worst <= DRIFT + (chains + parts + 1) * 2.0 ** -24, worst
