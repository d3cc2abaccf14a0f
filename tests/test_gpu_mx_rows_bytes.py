"""Every code with every scale byte, read back: exactly its value in the type asked for,
infinite where that is past the type's largest (4 and 6 times 2^126, 2 and more times
2^127), NaN for the byte 255."""
import numpy as np
import pytest
import torch

from oracle import block as D

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_code_with_every_scale(dtype):
    K = 256 * 32
    code = np.tile(np.arange(16, dtype=np.uint8), (3, K // 16))
    scale = np.tile(np.arange(256, dtype=np.uint8), (3, 1))
    codes, tiles = D.mx_pack(code, scale)
    q = B.Mxfp4Rows(torch.from_numpy(codes).cuda(), torch.from_numpy(tiles).cuda())
    got = B.dequantize_rows_mxfp4(q, dtype).double().cpu().numpy()
    want = D.mx_values(code, scale)
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.array_equal(got, want, equal_nan=True)
    zeros = got == 0
    assert np.array_equal(np.signbit(got[zeros]), np.signbit(want[zeros]))
