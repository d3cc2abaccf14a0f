"""The MXFP4 rows that moe_block_norm writes: codes and scale tiles, byte by byte, are
those of its h as rounded."""
import numpy as np
import pytest

from oracle import block as D
from test_gpu_block_norm import BF, F16, F32, _f64, _inputs

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [32, 96, 160, 416, 4128])
@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, F16)])
@pytest.mark.parametrize("pad", [0, 3])
def test_scale_bytes_past_a_row_of_nan_are_0(d, S, Bt, pad):
    v = _inputs(130, d, S, Bt, pad=pad)
    v["x"][1, d // 2] = float("nan")
    v["o"][127, 0] = float("inf")
    v["x"][129, d - 1] = float("inf")
    r = B.block_norm(**v, mxfp4=True)
    code, scale = D.mx_encode(_f64(r["h"]))
    assert (scale[1] == 255).all() and (scale[129, -1] == 255)
    codes, tiles = D.mx_pack(code, scale)
    assert np.array_equal(r["mx"].codes.cpu().numpy(), codes)
    assert np.array_equal(r["mx"].scales.cpu().numpy(), tiles)
