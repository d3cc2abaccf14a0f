"""What the MXFP4 product's self-test refuses.  No call here reaches a GPU."""
import pytest

from moe_prefill_routing_gb300 import binding as B
from moe_prefill_routing_gb300 import build as build_mod

FAKE = 0x10000
NAMES = "x xs W Ws T K N y y_dtype status cta stream".split()
OK = dict(x=FAKE, xs=FAKE, W=FAKE, Ws=FAKE, T=4, K=64, N=10, y=FAKE, y_dtype=0, status=None, cta=0,
          stream=None)


@pytest.mark.parametrize("kw,rc", [
    (dict(cta=-1), "SHAPE"), (dict(cta=(1 << 31) - 1), "SHAPE"), (dict(T=0), "SHAPE"),
    (dict(K=48), "SHAPE"), (dict(N=0), "SHAPE"), (dict(y_dtype=3), "DTYPE"), (dict(x=None), "NULL"),
    (dict(W=None), "NULL"), (dict(x=FAKE + 8), "ALIGN"), (dict(xs=FAKE + 8), "ALIGN"),
    (dict(y=FAKE + 1), "ALIGN"), (dict(status=FAKE + 2), "ALIGN"),
    (dict(xs=None, x=FAKE + 1), "ALIGN"),
    (dict(xs=None, T=17), "SHAPE")])  # more rows than the kernel quantises
def test_wait_limit(kw, rc):
    build_mod.build()
    a = {**OK, **kw}
    got = B.lib().moe_selftest_linear_mxfp4_wait_limit(*[a[n] for n in NAMES])
    assert got == getattr(B, "MOE_ERR_" + rc)
