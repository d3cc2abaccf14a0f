"""The MXFP4 rows that moe_block_norm writes: codes and scale tiles, byte by byte, are
those of its h as rounded."""
import numpy as np
import pytest
import torch

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


def _at(t):
    return None if t is None else t.data_ptr()


@pytest.mark.parametrize("S,Bt", [(BF, BF), (F32, F16), (F32, F32)])
@pytest.mark.parametrize("T,d,pad", [(1, 2560, 0), (130, 96, 0), (130, 416, 3), (300, 2592, 0),
                                     (50, 4128, 1), (9, 8224, 0)])
@pytest.mark.parametrize("o", [True, False])
def test_codes_without_h(T, d, pad, S, Bt, o):
    """h NULL: its codes and scales alone are written (the C interface; the binding
    always writes h)."""
    v = _inputs(T, d, S, Bt, o=o, pad=pad, mask=True)
    want = B.block_norm(**v, h_dtype=Bt, mxfp4=True)
    mx = B.Mxfp4Rows.empty(T, d, "cuda")
    mx.scales.fill_(7)
    xn = torch.empty(T, d, dtype=S, device="cuda") if o else None
    code = {BF: B.DT_BF16, F16: B.DT_F16, F32: B.DT_F32}
    rc = B.lib().moe_block_norm(
        _at(v["x"]), max(v["x"].stride(0), d), code[S], _at(v["o"]),
        max(v["o"].stride(0), d) if o else 0, code[Bt], _at(v["pre"]), _at(v["post"]),
        _at(v["gate"]), _at(v["mask"]), T, d, 1, 0, 1.0, 1e-6, _at(xn), d, None, 0, _at(mx.codes),
        _at(mx.scales), torch.cuda.current_stream().cuda_stream)
    assert rc == B.MOE_OK
    assert torch.equal(mx.codes, want["mx"].codes) and torch.equal(mx.scales, want["mx"].scales)
    assert not o or torch.equal(xn, want["xn"])
