"""The choice of tiles of moe_linear and moe_linear_grad on the CPU, over the
range of sizes, types and SM counts: what a launch asks of an SM has to fit."""
import random

import pytest

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300 import build as build_mod

SMEM = 227 * 1024  # of a CTA on sm_103a, its static shared memory included


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


SIZES = [(2048, 2560, 512), (1024, 2560, 256), (512, 5120, 512), (4096, 2560, 1024),
         (2048, 5120, 512), (4096, 5120, 512), (8192, 5120, 512), (1089, 3032, 875),
         (2048, 7168, 256), (21, 912, 7602)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("what", [("y",), ("dx",), ("dW",), ("dx", "dW")])
def test_every_launch_fits_shared_memory(lib, what, f32):
    rng = random.Random(7)
    span = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    sizes = SIZES + [(span(1, 200000), 8 * span(1, 4096), span(1, 40000)) for _ in range(4000)]
    for sms in (132, 148, 152, 160):
        for T, K, N in sizes:
            p = B.selftest_linear_plan(T, K, N, what, f32, sms)
            assert 1 <= p["launches"] <= 2
            assert p["smem"] + 1024 <= SMEM, (T, K, N, sms, p)


@pytest.mark.parametrize("what", [("dW", "dy fp32"), ("dx", "dW", "dy fp32")])
def test_every_launch_of_a_dw_from_two_pieces_fits(lib, what):
    rng = random.Random(8)
    span = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    sizes = SIZES + [(span(1, 200000), 8 * span(1, 4096), span(1, 40000)) for _ in range(4000)]
    for T, K, N in sizes:
        p = B.selftest_linear_plan(T, K, N, what, True, 152)
        assert 1 <= p["launches"] <= 2 and p["smem"] + 1024 <= SMEM, (T, K, N, p)


def test_status_calls_refuse(lib):
    fake = 0x10000
    assert lib.moe_take_status(None, None) == B.MOE_ERR_NULL
    assert lib.moe_selftest_linear_wait_limit(fake, fake, 4, 64, 8, fake, None, -1, None) == (
        B.MOE_ERR_SHAPE)
    assert lib.moe_selftest_linear_wait_limit(fake, fake, 4, 60, 8, fake, None, 0, None) == (
        B.MOE_ERR_SHAPE)
    assert lib.moe_selftest_linear_plan(4, 64, 8, 1, 0, 152, None) == B.MOE_ERR_NULL
    for what in (0, 3, 5, 7, 9, 16):
        with pytest.raises(B.MoeError):
            B._check("plan", lib.moe_selftest_linear_plan(4, 64, 8, what, 1, 152,
                                                          (B.C.c_int64 * 3)()))
