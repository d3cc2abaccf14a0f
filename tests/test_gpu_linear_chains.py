"""Long reductions of numbers of one sign, where the tensor core's truncating
additions drift by at most 2^-23 of the sum per MMA of 16 products.  fp32
outputs are summed in chains of 32 MMAs, which are added in fp32 to the
nearest: a few hundred roundings of 2^-25 whose signs vary (2e-7, doubled for
the largest of some 10^4 elements).  16-bit outputs: chains of 1024 (fp16) or
8192 (bf16) MMAs, a quarter of half a unit, and half a unit of the type."""
import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _abs(seed, *shape, dtype, amp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (amp * torch.randn(*shape, generator=g, device="cuda").abs()).to(dtype)


def _off(got, a, b):
    """Largest relative error of a b, in 64 bits."""
    ref = a.double() @ b.double()
    return float(((got.double() - ref).abs() / ref).max())


@pytest.mark.parametrize("N,T", [(64, 65536), (9, 131072), (30, 131072), (64, 131072),
                                 (100, 100001), (300, 70000)])
def test_fp32_dw_of_many_tokens(N, T):
    x = _abs(1, T, 136, dtype=torch.bfloat16)
    dy = _abs(2, T, N, dtype=torch.bfloat16)
    W = torch.zeros((N, 136), dtype=torch.bfloat16, device="cuda")
    _, dW, _ = B.linear_grad(x, W, dy, need=(False, True, False), dw_dtype=torch.float32)
    assert _off(dW, dy.t(), x) < 32 * 2.0 ** -23 + 4e-7


@pytest.mark.parametrize("T,dtype", [(1, torch.bfloat16), (40, torch.float16), (120, torch.bfloat16)])
def test_fp32_output_of_a_long_row(T, dtype):
    K, N = 131072 + 72, 100
    x, W = _abs(3, T, K, dtype=dtype), _abs(4, N, K, dtype=dtype)
    y = B.linear(x, W, out_dtype=torch.float32)
    assert _off(y, x, W.t()) < 32 * 2.0 ** -23 + 4e-7


@pytest.mark.parametrize("N,T,dtype,chain", [(256, 1 << 20, torch.float16, 1024),
                                             (64, 1 << 20, torch.float16, 1024),
                                             (200, 1 << 21, torch.bfloat16, 8192)])
def test_16_bit_dw_of_a_million_tokens(N, T, dtype, chain):
    x = _abs(5, T, 64, dtype=dtype)
    dy = _abs(6, T, N, dtype=dtype, amp=2.0 ** -6)
    W = torch.zeros((N, 64), dtype=dtype, device="cuda")
    _, dW, _ = B.linear_grad(x, W, dy, need=(False, True, False))
    half = torch.finfo(dtype).eps / 2
    tol = chain * 2.0 ** -23 + 1e-6
    assert _off(dW, dy.t(), x) < tol + half * (1 + tol)
