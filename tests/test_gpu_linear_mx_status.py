"""The stop of an MXFP4 product whose wait runs out: no GPU fault, a CTA's first stage
expects 16 bytes that never arrive, so its bounded waits run out (about 2 s) and it
stops; the status word says so, and the next call is right."""
import time

import pytest
import torch

from moe_prefill_routing_gb300 import binding as B

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rand(seed, *shape, amp=1.0):
    g = torch.Generator().manual_seed(seed)
    return (amp * torch.randn(*shape, generator=g)).to("cuda", BF)


# few rows, one CTA a tile; split over a cluster; a sum cut into chains; rows that the
# kernel quantises, in one CTA and in a cluster; pairs of CTAs, whose tiles of 64 - 192
# columns and of 256 are kernels of their own.  `lost`: rows and columns of the stopped tile
@pytest.mark.parametrize("T,K,N,cta,rows,out,lost", [
    (16, 480, 512, 1, False, BF, (slice(0, 16), slice(128, 256))),
    (30, 4096, 512, 8, False, BF, None),
    (20, 131328, 256, 3, False, F32, None),
    (4, 512, 512, 2, True, BF, (slice(0, 4), slice(256, 384))),
    (16, 2560, 512, 5, True, F32, None),
    (300, 2560, 512, 2, False, BF, None),
    (2049, 512, 5900, 4, False, BF, None),
    (2049, 512, 5900, 0, False, F32, None)])
@pytest.mark.parametrize("own", [True, False])
def test_a_wait_that_runs_out_is_reported(T, K, N, cta, rows, out, lost, own):
    x, W = _rand(1, T, K), B.quantize_rows_mxfp4(_rand(2, N, K, amp=K ** -0.5))
    if not rows:
        x = B.quantize_rows_mxfp4(x)
    want = B.linear_mxfp4(x, W, out_dtype=out)
    torch.cuda.synchronize()
    assert B.take_status() == 0
    word = torch.zeros(1, dtype=torch.int32, device="cuda") if own else None
    t0 = time.time()
    y = B.selftest_linear_mxfp4_wait_limit(x, W, cta, out, word)
    torch.cuda.synchronize()
    assert 1.0 < time.time() - t0 < 60.0
    taken = B.take_status()
    if own:
        assert int(word.item()) == B.STATUS_TIMEOUT and taken == 0
    else:
        assert taken == B.STATUS_TIMEOUT and B.take_status() == 0  # cleared
    if lost:  # the other tiles are what they should be
        keep = torch.ones((T, N), dtype=torch.bool, device="cuda")
        keep[lost] = False
        assert torch.equal(y[keep], want[keep])
    assert torch.equal(B.linear_mxfp4(x, W, out_dtype=out), want) and B.take_status() == 0


def test_calls_with_a_status_word_leave_it_alone():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    W = B.quantize_rows_mxfp4(_rand(2, 96, 128))
    for T in (3, 40, 300):
        x = _rand(1, T, 128)
        assert torch.equal(B.linear_mxfp4(x, W, status=word), B.linear_mxfp4(x, W))
    assert int(word.item()) == 0 and B.take_status() == 0
