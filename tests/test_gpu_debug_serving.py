"""The window kernels and the paged cache's kernels in the debug build (on-device bounds checks
that record XATTN_ERR_DEVICE_BOUNDS), in a child process that loads it in place of the release
library: every check passes on edge shapes, and the results stay within their bounds."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, "tests")
sys.path.insert(0, ".")
import torch
from bwd_xattn_fwd_gb300 import workloads as W, xattn
from paged_ref import check_tree, paged_state, random_words, signed, tree_reference
from window_ref import check, reference

assert xattn.xattn_build_flags() & xattn.BUILD_DEVICE_CHECKS
for shape, det in [((2, 700, 4, 2, 64, 130, 4), False), ((24, 300, 8, 2, 32, 70, 140), False),
                   ((1, 1500, 4, 4, 64, 200, 3), False), ((1, 2500, 4, 2, 64, 128, 4), True),
                   ((1, 900, 4, 2, 128, 300, 130), False)]:
    B, S, nh, nkv, hd, window, sinks = shape
    w = W.Workload("debug", B, S, nh, nkv, hd, "bf16", qkv_scale=0.5)
    x = {n: t.cuda() for n, t in W.make_inputs(w, seed=5).items()}
    o, lse = xattn.attention_window_fwd(x["q"], x["k"], x["v"], window, sinks)
    dq, dk, dv = xattn.attention_window_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, window, sinks, deterministic=det)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0, shape
    check({"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, reference(x, window, sinks, hd ** -0.5, True), str(shape))
i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
for B, n, nh, nkv, hd, page, lens, window, sinks in [
        (3, 5, 8, 2, 64, 16, [0, 333, 1200], 2**31 - 1, 0), (2, 64, 4, 2, 64, 64, [700, 90], 2**31 - 1, 0),
        (2, 1, 8, 2, 128, 32, [2000, 17], 300, 4), (3, 9, 14, 2, 32, 256, [600, 1, 2500], 200, 130),
        (40, 1, 4, 4, 64, 16, [100 + 37 * i for i in range(40)], 2**31 - 1, 0)]:
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=3, device="cuda")
    words = random_words(B, n, 1)
    q = (torch.randn(B, n, nh, hd, generator=torch.Generator().manual_seed(1)) * 0.5).to(torch.bfloat16).cuda()
    o, lse = xattn.attention_tree_decode(q, k, v, i32(table), i32(lens), tree=torch.tensor(signed(words), device="cuda"),
                                         window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0, (B, n, hd)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, words, window, sinks, hd ** -0.5), str((B, n, hd)))
print("debug build ok")
"""


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def test_debug_build_checks_pass():
    from bwd_xattn_fwd_gb300 import build
    env = dict(os.environ, XATTN_LIBRARY=build.build(debug=True))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "debug build ok" in r.stdout
