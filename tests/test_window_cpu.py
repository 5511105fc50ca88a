"""Window attention's argument checks, and its 64-bit reference against differences, without a GPU."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

from window_ref import reference


@pytest.fixture(scope="module")
def lib():
    from bwd_xattn_fwd_gb300 import build
    return ctypes.CDLL(build.build())


P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float


def _fwd(lib, name="xattn_window_fwd", q=16, k=32, v=48, B=1, S=4, nh=2, nkv=1, hd=64, window=2, sinks=0,
         scale=0.125, o=64, lse=80):
    f = getattr(lib, name)
    f.restype, f.argtypes = I, [P] * 3 + [I] * 7 + [F] + [P] * 3
    return f(q, k, v, B, S, nh, nkv, hd, window, sinks, scale, o, lse, None)


def _bwd(lib, name="xattn_window_bwd", q=16, hd=64, S=4, nh=2, nkv=1, window=2, sinks=0, scale=0.125, lse=96, dq=112):
    f = getattr(lib, name)
    f.restype = I
    f.argtypes = [P] * 6 + [I] * 7 + [F] + ([I] if name == "xattn_window_bwd" else []) + [P] * 4
    det = (0,) if name == "xattn_window_bwd" else ()
    return f(q, 32, 48, 64, 80, lse, 1, S, nh, nkv, hd, window, sinks, scale, *det, dq, 128, 144, None)


@pytest.mark.parametrize("name", ["xattn_window_fwd", "xattn_window_fwd_f32"])
def test_forward_checks(lib, name):
    assert _fwd(lib, name, q=None) == 1
    assert _fwd(lib, name, lse=None) == 1
    assert _fwd(lib, name, B=0) == 2
    assert _fwd(lib, name, S=0) == 2
    assert _fwd(lib, name, S=(1 << 30) + 1) == 2
    assert _fwd(lib, name, nh=3, nkv=2) == 3
    assert _fwd(lib, name, scale=float("nan")) == 9
    assert _fwd(lib, name, window=0) == 13
    assert _fwd(lib, name, window=-5) == 13
    assert _fwd(lib, name, sinks=-1) == 13
    assert _fwd(lib, name, hd=129) == 4
    if name == "xattn_window_fwd":
        assert _fwd(lib, hd=48) == 4
        assert _fwd(lib, q=18) == 5
        assert _fwd(lib, lse=82) == 5


@pytest.mark.parametrize("name", ["xattn_window_bwd", "xattn_window_bwd_f32"])
def test_backward_checks(lib, name):
    assert _bwd(lib, name, q=None) == 1
    assert _bwd(lib, name, S=-1) == 2
    assert _bwd(lib, name, nh=3, nkv=2) == 3
    assert _bwd(lib, name, window=0) == 13
    assert _bwd(lib, name, sinks=-1) == 13
    assert _bwd(lib, name, hd=130) == 4
    assert _bwd(lib, name, scale=float("inf")) == 9
    if name == "xattn_window_bwd":
        assert _bwd(lib, scale=1e-30) == 9
        assert _bwd(lib, dq=120) == 5
        assert _bwd(lib, lse=98) == 5


def test_status_strings_of_the_new_codes(lib):
    lib.xattn_status_string.restype = ctypes.c_char_p
    texts = {lib.xattn_status_string(code).decode() for code in (0, 12, 13, 14)}
    assert len(texts) == 4 and "unknown xattn status" not in texts


def test_accepted_sizes_reach_the_device(lib):
    if not torch.cuda.is_available():
        assert _fwd(lib, window=0x7FFFFFFF, sinks=0x7FFFFFFF) == 6
        assert _bwd(lib, hd=128, window=0x7FFFFFFF, sinks=0x7FFFFFFF) == 6


def test_helpers_refuse_what_they_cannot_read():
    from bwd_xattn_fwd_gb300 import xattn
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                   # not on a GPU
        xattn.attention_window_fwd(q, q, q, 2)
    with pytest.raises(TypeError):
        xattn.attention_window_fwd(q.half(), q.half(), q.half(), 2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (20, 0), (4, 20)])
def test_reference_gradients_against_differences(window, sinks):
    g = torch.Generator().manual_seed(0)
    x = {n: torch.randn(1, 12, h, 8, generator=g, dtype=torch.float64)
         for n, h in (("q", 4), ("k", 2), ("v", 2), ("dO", 4))}
    ref = reference(x, window, sinks, 0.3, False)

    def loss(y):
        return float((x["dO"] * reference({**x, **y}, window, sinks, 0.3, False)["o"][0]).sum())

    for name in ("q", "k", "v"):
        d = torch.randn(x[name].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        slope = (loss({name: x[name] + h * d}) - loss({name: x[name] - h * d})) / (2 * h)
        assert abs(float((ref["d" + name][0] * d).sum()) - slope) <= 1e-7 * (1 + abs(slope))


WITHOUT_EXTENSION = """
import sys
from bwd_xattn_fwd_gb300 import build
build.torch_lib = lambda: "/nonexistent/xattn_torch.so"
from bwd_xattn_fwd_gb300 import xattn
assert "torch" not in sys.modules
try:
    xattn.xattn_window_fwd(0, 32, 48, 1, 4, 2, 1, 64, 2, 0, 0.1, 64, 80, stream=0)
except xattn.XattnError as err:
    assert err.status == xattn.Status.ERR_NULL_PTR
import torch
q = torch.zeros(1, 4, 2, 64)
try:
    xattn.attention_window_fwd(q, q, q, 2)
except ImportError as err:
    print("needs", err)
"""


def test_the_c_entry_points_need_neither_torch_nor_the_extension(lib):
    """The binding imports, and its C-level functions run, before torch and without the native
    part of the tensor-level calls; the first of those says what is missing."""
    run = subprocess.run([sys.executable, "-c", WITHOUT_EXTENSION], capture_output=True, text=True,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and "/nonexistent/xattn_torch.so is not built" in run.stdout, run.stderr


def test_the_extension_is_one_python_s(monkeypatch):
    """A Python extension belongs to an ABI as well as to a torch version: its file names both."""
    import importlib.metadata
    import sysconfig
    from bwd_xattn_fwd_gb300 import build
    here = build.torch_lib()
    assert importlib.metadata.version("torch") in here and sysconfig.get_config_var("SOABI") in here
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert build.torch_lib() != here


def test_a_torch_without_cuda_has_no_extension(monkeypatch, tmp_path):
    """There is nothing to build then, the library is built all the same, and the tensor-level calls
    say what they lack."""
    from bwd_xattn_fwd_gb300 import build, xattn
    (tmp_path / "lib").mkdir()
    monkeypatch.setattr(build, "torch_dir", lambda: str(tmp_path))
    assert build.torch_lib() == "" and build._torch_current()
    assert build.build() == build.LIB
    with pytest.raises(ImportError, match="CUDA"):
        xattn._load_calls()


def test_trimming_the_scratch_needs_a_device(lib):
    from bwd_xattn_fwd_gb300 import xattn
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    with pytest.raises(xattn.XattnError) as err:
        xattn.xattn_trim_scratch(1 << 20)
    assert err.value.status == xattn.Status.ERR_CUDA


def _causal(lib, name, bad):
    """A causal entry point with pointer number `bad` two bytes off."""
    f = getattr(lib, name)
    n_in, n_out = (3, 2) if "fwd" in name else (6, 3)
    f.restype, f.argtypes = I, [P] * n_in + [I] * 5 + [F] + [P] * n_out + [P]
    at = [16 * (i + 1) + (2 if i == bad else 0) for i in range(n_in + n_out)]
    return f(*at[:n_in], 1, 4, 2, 1, 64, 0.125, *at[n_in:], None)


def _window_f32(lib, name, bad):
    f = getattr(lib, name)
    n_in, n_out = (3, 2) if "fwd" in name else (6, 3)
    f.restype, f.argtypes = I, [P] * n_in + [I] * 7 + [F] + [P] * n_out + [P]
    at = [16 * (i + 1) + (2 if i == bad else 0) for i in range(n_in + n_out)]
    return f(*at[:n_in], 1, 4, 2, 1, 64, 2, 0, 0.125, *at[n_in:], None)


def test_misaligned_floats_are_refused(lib):
    """A float tensor or lse that is not 4-byte aligned would fault on the device."""
    for name in ("xattn_window_fwd_f32", "xattn_window_bwd_f32"):
        for bad in range(5 if "fwd" in name else 9):
            assert _window_f32(lib, name, bad) == 5, (name, bad)
    for name in ("xattn_fwd_f32", "xattn_bwd_f32", "xattn_fwd", "xattn_bwd", "xattn_bwd_deterministic",
                 "xattn_bwd_noalloc"):
        for bad in range(5 if "fwd" in name else 9):
            assert _causal(lib, name, bad) == 5, (name, bad)
    f = lib.xattn_bwd_preprocess
    f.restype, f.argtypes = I, [P] * 3 + [I] * 4 + [F, P, ctypes.c_size_t, P]
    assert f(16, 32, 50, 1, 4, 2, 64, 0.125, 256, 1 << 20, None) == 5


def test_scales_too_large_for_base_2(lib):
    assert _fwd(lib, scale=2.5e38) == 9 and _bwd(lib, scale=2.5e38) == 9
    if not torch.cuda.is_available():
        assert _fwd(lib, "xattn_window_fwd_f32", scale=2.5e38) == 6
