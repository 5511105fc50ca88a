"""The causal forward over many units a CTA, with odd numbers of query tiles (units of one query
tile among units of two: the two MMA issuers then use different key tiles of the ring): every
element within the bounds of tests/window_ref.py, the same bits from run to run, no wait run out."""
import pytest
import torch

from bwd_xattn_fwd_gb300 import workloads as W
from window_ref import check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(64, 384, 8, 2, 64), (60, 300, 8, 2, 32), (50, 384, 8, 8, 64), (80, 257, 8, 8, 32),
                                   (160, 128, 8, 2, 64), (60, 256, 8, 4, 64), (30, 640, 8, 2, 64), (40, 384, 8, 2, 128),
                                   (20, 600, 6, 6, 128)], ids=str)
def test_many_units_a_cta(shape):
    from bwd_xattn_fwd_gb300 import xattn
    B, S, nh, nkv, hd = shape
    w = W.Workload("units", B, S, nh, nkv, hd, "bf16", qkv_scale=0.5)
    x = {n: t.cuda() for n, t in W.make_inputs(w, seed=S).items()}
    o, lse = xattn.attention_fwd(x["q"], x["k"], x["v"])
    for _ in range(20):
        again = xattn.attention_fwd(x["q"], x["k"], x["v"])
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    check({"o": o, "lse": lse}, reference(x, S, 0, hd ** -0.5, True), str(shape))
