"""CUDA contexts of the caller's: one that is current stays current and is the one that a call runs in; a thread whose context
has been popped gets the device's primary one."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def test_a_popped_context_is_bound_again():
    from bwd_xattn_fwd_gb300 import xattn
    cu = ctypes.CDLL("libcuda.so.1")
    q = torch.randn(2, 70, 2, 64, device="cuda").bfloat16()
    rope = torch.randn(2, 70, 16, device="cuda").bfloat16()
    out = [[torch.empty_like(q), torch.empty(2, 70, 2, device="cuda"), torch.empty(2, 70, 2, 16, device="cuda").bfloat16()]
           for _ in range(2)]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    seen = []

    def current():
        c = ctypes.c_void_p(1)
        assert cu.cuCtxGetCurrent(ctypes.byref(c)) == 0
        return c.value

    def calls(o, lse, o2):
        xattn.xattn_fwd(q, q, q, 2, 70, 2, 2, 64, 0.1, o, lse, stream)
        xattn.xattn_latent_fwd(q, q, rope, 2, 70, 2, 48, 16, 16, 0.1, o2, lse, stream)

    def work():
        calls(*out[0])
        seen.append(current())
        assert cu.cuCtxPopCurrent_v2(ctypes.byref(ctypes.c_void_p())) == 0
        seen.append(current())
        calls(*out[1])
        seen.append(current())

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert len(seen) == 3 and seen[0] and seen[1] is None and seen[2] == seen[0]
    assert all(torch.equal(a, b) for a, b in zip(*out)) and xattn.xattn_check_device_status() == 0


# The process works in a context that it has made, with memory of that context; torch is on the CPU only.
OWN_CONTEXT = r"""
import ctypes, sys
sys.path.insert(0, "tests")
sys.path.insert(0, ".")
import torch
from bwd_xattn_fwd_gb300 import xattn
from latent_ref import latent_inputs, latent_reference
from window_ref import check
cu = ctypes.CDLL("libcuda.so.1")
V, sz = ctypes.c_void_p, ctypes.c_size_t
def ok(code): assert code == 0, code
dev, ctx, stream = ctypes.c_int(), V(), V()
ok(cu.cuInit(0))
ok(cu.cuDeviceGet(ctypes.byref(dev), 0))
ok(cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, dev))
ok(cu.cuStreamCreate(ctypes.byref(stream), 0))
def current():
    c = V()
    ok(cu.cuCtxGetCurrent(ctypes.byref(c)))
    return c.value
def room(t):
    p = V()
    ok(cu.cuMemAlloc_v2(ctypes.byref(p), sz(t.numel() * t.element_size())))
    ok(cu.cuMemcpyHtoD_v2(p, V(t.data_ptr()), sz(t.numel() * t.element_size())))
    return p
def back(p, t):
    ok(cu.cuMemcpyDtoH_v2(V(t.data_ptr()), p, sz(t.numel() * t.element_size())))
    return t
assert current() == ctx.value
B, S, nh, dn, dr, dv = 2, 300, 2, 64, 32, 64
x = latent_inputs(B, S, nh, dn, dr, dv, seed=1, device="cpu")
o, lse = torch.zeros(B, S, nh, dv).bfloat16(), torch.zeros(B, S, nh)
q, kv, rope, od, ld = (room(t) for t in (x["q"], x["kv"], x["k_rope"], o, lse))
xattn.xattn_latent_fwd(q.value, kv.value, rope.value, B, S, nh, dn, dr, dv, 0.1, od.value, ld.value, stream.value)
assert current() == ctx.value
ok(cu.cuStreamSynchronize(stream))
ref = latent_reference(x, 0.1)
check({"o": back(od, o), "lse": back(ld, lse)}, ref, "own context")
k = torch.randn(1, 1, 2, 64).bfloat16()                     # one position: the output is its value
kd, o1, l1 = room(k), room(torch.zeros_like(k)), room(torch.zeros(2))
xattn.xattn_fwd(kd.value, kd.value, kd.value, 1, 1, 2, 2, 64, 0.1, o1.value, l1.value, stream.value)
assert current() == ctx.value
ok(cu.cuStreamSynchronize(stream))
assert torch.equal(back(o1, torch.zeros_like(k)), k)
assert xattn.xattn_check_device_status(stream.value) == 0 and current() == ctx.value
print("kept")
"""


def test_a_context_of_the_caller_s_stays_current():
    run = subprocess.run([sys.executable, "-c", OWN_CONTEXT], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert run.returncode == 0 and run.stdout.strip() == "kept", run.stdout[-1000:] + run.stderr[-3000:]
