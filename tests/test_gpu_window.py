"""Window attention with sinks through the binding, against its definition in 64 bits (every
element within a bound derived from the roundings, tests/window_ref.py), on windows and sinks
that end inside, at and across tiles; against the causal op; gradients against differences;
graphs, streams and run-to-run reproducibility."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from bwd_xattn_fwd_gb300 import workloads as W
from window_ref import check, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn  # noqa: F401  (fails loudly if not built)


def _inputs(B, S, nh, nkv, hd, dtype, seed=0):
    w = W.Workload("window", B, S, nh, nkv, hd, dtype, qkv_scale=0.5)
    return {n: t.cuda() for n, t in W.make_inputs(w, seed=seed).items()}


def _run(x, window, sinks, scale, deterministic=False):
    from bwd_xattn_fwd_gb300 import xattn
    q, k, v, dO = (x[n] for n in ("q", "k", "v", "dO"))
    o, lse = xattn.attention_window_fwd(q, k, v, window, sinks, scale)
    dq, dk, dv = xattn.attention_window_bwd(q, k, v, o, dO, lse, window, sinks, scale, deterministic=deterministic)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# (B, S, nh, nkv, hd, window, sinks): lengths 1, below, at and past tiles; windows of one key,
# ending inside and at tiles, spanning several, and beyond the sequence; no sinks, a few, a
# tile's worth, more than one tile, all keys; query groups and one head per kv head
SHAPES = [
    (1, 1, 1, 1, 64, 1, 0),
    (2, 5, 2, 1, 32, 2, 1),
    (1, 128, 2, 2, 64, 1, 0),
    (1, 129, 2, 2, 64, 128, 0),
    (1, 300, 4, 2, 64, 1, 1),
    (2, 300, 4, 2, 64, 7, 3),
    (1, 640, 4, 4, 64, 129, 0),
    (1, 700, 4, 1, 64, 128, 4),
    (2, 1000, 4, 2, 64, 130, 4),
    (1, 1100, 8, 2, 64, 257, 128),
    (1, 1500, 4, 2, 64, 64, 129),
    (1, 1500, 4, 2, 64, 300, 260),
    (1, 900, 4, 2, 64, 2000, 3),
    (1, 900, 4, 2, 64, 100, 2000),
    (1, 900, 2, 1, 64, 899, 0),
    (2, 515, 6, 3, 32, 60, 4),
    (1, 1300, 4, 4, 32, 200, 17),
    (1, 257, 2, 1, 128, 100, 0),
    (1, 1290, 4, 2, 128, 300, 4),
    (1, 1290, 2, 2, 128, 33, 140),
    (24, 520, 8, 2, 64, 140, 4),       # several units per CTA
    (3, 2100, 12, 12, 32, 500, 4),
    (2, 4000, 4, 1, 64, 256, 4),       # sink tiles cut into many parts
    (1, 3500, 8, 2, 128, 150, 130),
    (1, 5000, 2, 1, 64, 40, 1500),     # many sink tiles
    (40, 700, 8, 8, 32, 30, 200),      # many heads: sink tiles uncut
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("deterministic", [False, True])
def test_bf16(shape, deterministic):
    B, S, nh, nkv, hd, window, sinks = shape
    x = _inputs(B, S, nh, nkv, hd, "bf16", seed=S)
    scale = hd ** -0.5
    check(_run(x, window, sinks, scale, deterministic), reference(x, window, sinks, scale, True), str(shape))


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 1, 0), (2, 70, 4, 2, 24, 9, 0), (1, 130, 2, 2, 64, 33, 5),
                                   (1, 260, 2, 1, 128, 64, 70), (1, 90, 3, 3, 33, 500, 0), (1, 90, 3, 1, 5, 1, 200),
                                   (2, 499, 4, 2, 64, 100, 3), (3, 333, 4, 2, 128, 40, 33), (9, 70, 3, 3, 20, 9, 0)],
                         ids=str)
def test_f32(shape):
    B, S, nh, nkv, hd, window, sinks = shape
    x = _inputs(B, S, nh, nkv, hd, "f32", seed=S)
    scale = hd ** -0.5
    check(_run(x, window, sinks, scale), reference(x, window, sinks, scale, False), str(shape))


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_scales(scale):
    x = _inputs(1, 700, 4, 2, 64, "bf16", seed=3)
    check(_run(x, 200, 4, scale), reference(x, 200, 4, scale, True), f"scale {scale}")


@pytest.mark.parametrize("hd", [32, 64, 128])
def test_a_window_of_everything_is_the_causal_op(hd):
    """The forward does the causal op's arithmetic in its order: bit for bit the same."""
    from bwd_xattn_fwd_gb300 import xattn
    x = _inputs(2, 700, 4, 2, hd, "bf16", seed=1)
    q, k, v = (x[n] for n in ("q", "k", "v"))
    o, lse = xattn.attention_window_fwd(q, k, v, xattn.NO_WINDOW)
    ro, rl = xattn.attention_fwd(q, k, v)
    assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_gradients_against_differences():
    """Directional differences of L = sum(dO * o) in fp32 mode, taken in 64 bits of the
    definition: (L(x + h d) - L(x - h d)) / 2h against <grad, d>. With h = 1e-4 the difference's
    own error is O(h^2) ~ 1e-8 of the third derivative (unit-size inputs), far below 1e-4."""
    shape = (1, 150, 4, 2, 32)
    x = _inputs(*shape, "f32", seed=9)
    window, sinks, scale = 40, 3, 32 ** -0.5
    got = _run(x, window, sinks, scale)
    g = torch.Generator("cuda").manual_seed(1)

    def loss(y):
        o = reference({**x, **y}, window, sinks, scale, False)["o"][0]
        return float((x["dO"].double() * o).sum())

    for name in ("q", "k", "v"):
        d = torch.randn(x[name].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        slope = (loss({name: x[name].double() + h * d}) - loss({name: x[name].double() - h * d})) / (2 * h)
        dot = float((got["d" + name].double() * d).sum())
        assert abs(dot - slope) <= 1e-4 * float((got["d" + name].double() * d).abs().sum()), (name, dot, slope)


def test_reproducible():
    """o, lse, dk and dv are bit for bit the same from run to run, dq too when asked for."""
    x = _inputs(2, 2000, 8, 2, 64, "bf16", seed=4)
    a, b = (_run(x, 300, 5, 0.125) for _ in range(2))
    c, d = (_run(x, 300, 5, 0.125, deterministic=True) for _ in range(2))
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n
    for n in c:
        assert torch.equal(c[n], d[n]), n


@pytest.mark.parametrize("shape", [(4, 4096, 16, 4, 64, 1024, 0), (3, 4000, 16, 4, 64, 512, 0),
                                   (2, 3970, 16, 4, 128, 1024, 4), (40, 640, 8, 2, 64, 256, 0),
                                   (30, 1000, 8, 8, 32, 128, 0)], ids=str)
def test_many_units_in_a_row(shape):
    """Many units per CTA, windows that end at tile borders (the two query tiles of a unit then
    differ in one key tile at each end), again and again: no wait runs out, and every run gives
    the same bits. With an odd number of query tiles some units have one tile only."""
    from bwd_xattn_fwd_gb300 import xattn
    B, S, nh, nkv, hd, window, sinks = shape
    x = _inputs(B, S, nh, nkv, hd, "bf16", seed=8)
    first = xattn.attention_window_fwd(x["q"], x["k"], x["v"], window, sinks)
    for _ in range(15):
        again = xattn.attention_window_fwd(x["q"], x["k"], x["v"], window, sinks)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert xattn.xattn_check_device_status() == 0


def test_graph_replay_and_streams():
    """Forward and backward captured on a side stream, replayed on new inputs."""
    from bwd_xattn_fwd_gb300 import xattn
    x = _inputs(2, 600, 4, 2, 64, "bf16", seed=5)
    scale = 0.125
    _run(x, 100, 4, scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    q, k, v, dO = (x[n] for n in ("q", "k", "v", "dO"))
    with torch.cuda.graph(graph, stream=side):
        o, lse = xattn.attention_window_fwd(q, k, v, 100, 4, scale)
        dq, dk, dv = xattn.attention_window_bwd(q, k, v, o, dO, lse, 100, 4, scale)
    y = _inputs(2, 600, 4, 2, 64, "bf16", seed=6)
    for n in x:
        x[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    check({"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}, reference(y, 100, 4, scale, True), "replay")
    # an explicit stream, its outputs allocated for it
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o2, lse2 = xattn.attention_window_fwd(q, k, v, 100, 4, scale, stream=other)
    other.synchronize()
    assert torch.equal(o2, o) and torch.equal(lse2, lse)


FIRST_IN_CAPTURE = """
import torch
from bwd_xattn_fwd_gb300 import xattn
g = torch.Generator(device="cuda").manual_seed(0)
q, k, v, dO = (torch.randn(2, 200, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(4))
table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
lens = torch.tensor([50, 7], device="cuda", dtype=torch.int32)
pages = torch.randn(8, 128, 2, 64, generator=g, device="cuda").bfloat16()
def calls():
    o, lse = xattn.attention_window_fwd(q, k, v, 70, 3)
    grads = xattn.attention_window_bwd(q, k, v, o, dO, lse, 70, 3, deterministic=True)
    t, _ = xattn.attention_tree_decode(q[:, :4].contiguous(), pages, pages, table, lens)
    return o, *grads, t
side = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
eager = calls()
torch.cuda.synchronize()
assert xattn.xattn_check_device_status() == 0
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
print("same")
"""


def test_first_calls_of_a_process_captured():
    """The library's first calls in a process (which set up its state for the device) may be
    captured ones."""
    run = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]


def test_two_threads_at_once():
    """Calls from two host threads on streams of their own give what they give alone."""
    cases = [(_inputs(2, 400, 4, 2, 64, "bf16", seed=1), 100, 4), (_inputs(1, 700, 2, 2, 128, "bf16", seed=2), 33, 140)]
    alone = [_run(x, w, s, 0.125, deterministic=True) for x, w, s in cases]
    got = [None, None]

    def work(i):
        x, w, s = cases[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                from bwd_xattn_fwd_gb300 import xattn
                o, lse = xattn.attention_window_fwd(x["q"], x["k"], x["v"], w, s, 0.125)
                dq, dk, dv = xattn.attention_window_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, w, s, 0.125,
                                                        deterministic=True)
            torch.cuda.current_stream().synchronize()
            got[i] = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert all(torch.equal(a[n], b[n]) for n in a)


def test_the_scratch_can_be_given_back():
    """A backward's scratch (its fp32 dQ accumulator alone is 4 B S nh hd bytes) stays with the
    library until it is trimmed; the next call takes new scratch and gives the same bits."""
    from bwd_xattn_fwd_gb300 import xattn
    B, S, nh, nkv, hd = 4, 4096, 16, 4, 64
    x = _inputs(B, S, nh, nkv, hd, "bf16", seed=2)
    a = _run(x, 700, 4, 0.125)
    used = 4 * B * S * nh * hd
    xattn.xattn_trim_scratch(1 << 40)                      # beyond what there is: nothing to give back
    held = torch.cuda.mem_get_info()[0]
    xattn.xattn_trim_scratch()
    assert torch.cuda.mem_get_info()[0] - held >= used
    b = _run(x, 700, 4, 0.125)
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(a[n], b[n]), n
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = xattn.attention_window_fwd(x["q"], x["k"], x["v"], 700, 4, 0.125)
        xattn.xattn_trim_scratch()                         # takes no part in the capture
        c = xattn.attention_window_bwd(x["q"], x["k"], x["v"], o, x["dO"], lse, 700, 4, 0.125)
    for _ in range(2):                                     # the graph's scratch is its own
        graph.replay()
        torch.cuda.synchronize()
        xattn.xattn_trim_scratch()
        assert torch.equal(o, a["o"]) and torch.equal(c[1], a["dk"]) and torch.equal(c[2], a["dv"])


EVERY_CALL_FIRST_IN_CAPTURE = """
import torch
from bwd_xattn_fwd_gb300 import xattn
g = torch.Generator(device="cuda").manual_seed(0)
rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
q, k, v, dO, o = (rnd(2, 200, 2, 64) for _ in range(5))
qf, kf, vf, dOf, of = (t.float() for t in (q, k, v, dO, o))
lse = torch.full((2, 200, 2), 5.0, device="cuda")
one, new = rnd(2, 2, 64), rnd(2, 4, 2, 64)
i32 = lambda x: torch.tensor(x, device="cuda", dtype=torch.int32)
table, lens, path = i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([50, 7]), i32([[0, 2, 3, 0]] * 2)
pools = rnd(8, 16, 2, 64), rnd(8, 16, 2, 64)
def calls():
    out = [*xattn.attention_fwd(q, k, v), *xattn.attention_bwd(q, k, v, o, dO, lse)[1:],
           *xattn.attention_bwd(q, k, v, o, dO, lse, deterministic=True), *xattn.attention_decode(one, k, v),
           *xattn.attention_fwd(qf, kf, vf), *xattn.attention_bwd(qf, kf, vf, of, dOf, lse),
           *xattn.attention_window_fwd(qf, kf, vf, 70, 3), *xattn.attention_window_bwd(qf, kf, vf, of, dOf, lse, 70, 3)]
    xattn.cache_append(new, new, *pools, table, lens)
    xattn.cache_compact(*pools, table, lens, path, i)
    return *out, pools[0].clone(), pools[1].clone()
i = i32([3, 2])
side = torch.cuda.Stream()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=side):
    captured = calls()
graph.replay()
torch.cuda.synchronize()
eager = calls()
torch.cuda.synchronize()
assert xattn.xattn_check_device_status() == 0
assert all(torch.equal(a, b) for a, b in zip(captured, eager))
print("same")
"""


def test_the_other_calls_as_a_process_s_first_captured():
    """The same of the causal calls, the decode step, the fp32 forms and the page calls."""
    run = subprocess.run([sys.executable, "-c", EVERY_CALL_FIRST_IN_CAPTURE], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]
