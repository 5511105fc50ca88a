"""Latent attention through the binding against its definition in 64 bits (every element within a bound derived
from the roundings, tests/latent_ref.py): the expanded form and its gradients at lengths 1, below, at and past
tiles and at every kind of head size; the absorbed form over ragged, empty and long paged caches whose other rows
hold NaN; the two forms against each other; graphs, streams, threads and run-to-run reproducibility."""
import math
import os
import random
import subprocess
import sys
import threading

import pytest
import torch

from latent_ref import latent_decode_reference, latent_inputs, latent_reference, latent_state
from paged_ref import check_tree
from window_ref import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn  # noqa: F401  (fails loudly if not built)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _run(x, scale):
    from bwd_xattn_fwd_gb300 import xattn
    q, kv, rope, dO = (x[n] for n in ("q", "kv", "k_rope", "dO"))
    o, lse = xattn.attention_latent_fwd(q, kv, rope, scale)
    dq, dkv, drope = xattn.attention_latent_bwd(q, kv, rope, o, dO, lse, scale)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    return {"o": o, "lse": lse, "dq": dq, "dkv": dkv, "dk_rope": drope}


# (B, S, nh, dn, dr, dv)
SHAPES = [
    (1, 1, 1, 128, 64, 128),
    (1, 1, 3, 16, 16, 16),
    (2, 5, 2, 64, 32, 64),
    (1, 63, 1, 128, 64, 128),
    (1, 64, 2, 128, 64, 128),
    (2, 65, 2, 64, 64, 128),
    (1, 127, 2, 128, 32, 64),
    (1, 128, 2, 128, 64, 128),
    (3, 129, 2, 64, 32, 64),
    (1, 192, 2, 80, 48, 112),
    (1, 255, 5, 48, 16, 96),
    (2, 256, 2, 128, 64, 128),
    (1, 257, 3, 112, 64, 16),
    (1, 385, 2, 16, 64, 128),
    (2, 513, 3, 64, 32, 64),
    (1, 700, 4, 128, 64, 128),
    (1, 1030, 16, 96, 32, 64),
    (2, 1500, 2, 128, 64, 128),
    (40, 200, 8, 64, 32, 64),          # several units a CTA
    (9, 300, 12, 128, 64, 128),
    (1, 3001, 2, 128, 64, 128),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_expanded(shape):
    B, S, nh, dn, dr, dv = shape
    x = latent_inputs(*shape, seed=S)
    scale = (dn + dr) ** -0.5
    check(_run(x, scale), latent_reference(x, scale), str(shape))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5, 1e-30])
def test_scales(scale):
    x = latent_inputs(1, 300, 2, 128, 64, 128, seed=3)
    check(_run(x, scale), latent_reference(x, scale), f"scale {scale}")


def test_the_default_scale():
    from bwd_xattn_fwd_gb300 import xattn
    x = latent_inputs(1, 70, 2, 64, 32, 64, seed=4)
    q, kv, rope = x["q"], x["kv"], x["k_rope"]
    o, lse = xattn.attention_latent_fwd(q, kv, rope)
    o2, lse2 = xattn.attention_latent_fwd(q, kv, rope, 96 ** -0.5)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    a = xattn.attention_latent_bwd(q, kv, rope, o, x["dO"], lse)
    b = xattn.attention_latent_bwd(q, kv, rope, o, x["dO"], lse, 96 ** -0.5)
    assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_growing_scores():
    """Row maxima that grow by more than 2^8 from tile to tile, and ones that the first tile holds."""
    x = latent_inputs(1, 900, 2, 128, 64, 128, seed=5)
    up = torch.linspace(0.05, 1.0, 900, device="cuda")
    for ramp in (up, up.flip(0)):
        y = dict(x)
        y["kv"] = x["kv"].clone()
        y["kv"][..., :128] = (x["kv"][..., :128].float() * ramp[None, :, None, None] * 4).bfloat16()
        y["q"] = (x["q"].float() * 4).bfloat16()
        check(_run(y, 0.3), latent_reference(y, 0.3), "ramp")


def test_rows_of_one_sequence_do_not_reach_another():
    """A batch gives each sequence the bits that it has alone."""
    x = latent_inputs(3, 333, 4, 128, 64, 128, seed=6)
    got = _run(x, 0.07)
    for b in range(3):
        alone = _run({n: t[b:b + 1].contiguous() for n, t in x.items()}, 0.07)
        for n in got:
            assert torch.equal(got[n][b:b + 1], alone[n]), (n, b)


def test_gradients_against_differences():
    """Directional differences of L = sum(dO * o), in 64 bits of the definition, against <grad, d> of the
    computed gradients, each element of which is within its bound of the exact one: the two differ by at most
    sum(bound |d|), and by the difference's own O(h^2) error, some 1e-8 of the sum of |grad d|."""
    x = latent_inputs(1, 150, 3, 64, 32, 64, seed=9)
    scale = 96 ** -0.5
    got, ref = _run(x, scale), latent_reference(x, scale)
    g = torch.Generator("cuda").manual_seed(1)

    def loss(y):
        return float((x["dO"].double() * latent_reference({**x, **y}, scale)["o"][0]).sum())

    for name in ("q", "kv", "k_rope"):
        d = torch.randn(x[name].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        slope = (loss({name: x[name].double() + h * d}) - loss({name: x[name].double() - h * d})) / (2 * h)
        grad = got["d" + name].double()
        room = float((ref["d" + name][1] * d.abs()).sum()) + 1e-6 * float((grad * d).abs().sum())
        assert abs(float((grad * d).sum()) - slope) <= room, name


def test_training_step_as_autograd():
    """The two calls as a torch.autograd.Function over the projections of a layer: gradients of the latents
    and weights that reach them through kv against the same layer written out in 64 bits. The products around
    the attention round to bf16 (kv, its gradient): each gradient within 3 % of the largest."""
    from bwd_xattn_fwd_gb300 import xattn

    class Latent(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, kv, rope):
            o, lse = xattn.attention_latent_fwd(q, kv, rope)
            ctx.save_for_backward(q, kv, rope, o, lse)
            return o

        @staticmethod
        def backward(ctx, dO):
            q, kv, rope, o, lse = ctx.saved_tensors
            return xattn.attention_latent_bwd(q, kv, rope, o, dO.contiguous(), lse)

    g = torch.Generator().manual_seed(2)
    B, S, nh, dc, dn, dr, dv = 2, 200, 4, 128, 64, 32, 64
    rnd = lambda *s, t=1.0: (torch.randn(*s, generator=g) * t).bfloat16().cuda()
    leaf = [rnd(B, S, dc, t=0.5), rnd(dc, nh * (dn + dv), t=dc ** -0.5), rnd(B, S, nh, dn + dr, t=0.5), rnd(B, S, dr, t=0.5)]
    dO = rnd(B, S, nh, dv)
    own = [t.clone().requires_grad_() for t in leaf]
    Latent.apply(own[2], (own[0] @ own[1]).view(B, S, nh, dn + dv), own[3]).backward(dO)
    exact = [t.double().requires_grad_() for t in leaf]
    kv = (exact[0] @ exact[1]).view(B, S, nh, dn + dv)
    k = torch.cat([kv[..., :dn], exact[3][:, :, None].expand(-1, -1, nh, -1)], 3)
    s = torch.einsum("bihd,bjhd->bhij", exact[2], k) * (dn + dr) ** -0.5
    s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device="cuda").triu(1), -math.inf)
    torch.einsum("bhij,bjhd->bihd", torch.softmax(s, 3), kv[..., dn:]).backward(dO.double())
    for a, b in zip(own, exact):
        assert float((a.grad.double() - b.grad).abs().max() / b.grad.abs().max()) <= 0.03


def test_reproducible_and_many_units():
    """Bit for bit the same, again and again, with many units a CTA."""
    for shape in ((4, 1100, 16, 128, 64, 128), (30, 385, 8, 64, 32, 64)):
        x = latent_inputs(*shape, seed=7)
        first = _run(x, 0.07)
        for _ in range(8):
            again = _run(x, 0.07)
            assert all(torch.equal(first[n], again[n]) for n in first)


# ---- absorbed form ------------------------------------------------------------------------

def _decode(q, pages, table, lens, dc, scale):
    from bwd_xattn_fwd_gb300 import xattn
    o, lse = xattn.attention_latent_decode(q, pages, _i32(table), _i32(lens), dc, scale)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    return o, lse


def _q(B, n, nh, width, seed, times=0.5):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn(B, n, nh, width, generator=g) * times).to(torch.bfloat16).cuda()


def _lens(B, top, seed):
    rng = random.Random(seed)
    return [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(B)]


# (B, n, nh, dc, dr, page, longest cache)
CASES = [
    (1, 1, 1, 512, 64, 16, 0),
    (1, 1, 16, 512, 64, 16, 5),
    (2, 1, 16, 512, 64, 64, 63),
    (2, 1, 16, 512, 64, 64, 64),
    (3, 1, 16, 512, 64, 64, 300),
    (2, 2, 16, 512, 64, 32, 200),
    (2, 4, 16, 512, 64, 16, 500),      # 64 rows
    (2, 1, 128, 512, 64, 128, 700),    # two row tiles
    (2, 3, 40, 512, 64, 16, 333),      # 120 rows: the second tile not full
    (2, 7, 5, 512, 64, 256, 600),      # pages wider than a tile
    (1, 64, 3, 512, 64, 384, 1000),
    (2, 64, 4, 256, 32, 16, 100),
    (3, 1, 8, 256, 64, 32, 900),
    (3, 5, 12, 256, 32, 64, 450),
    (2, 1, 16, 128, 16, 16, 700),
    (2, 9, 2, 128, 64, 64, 129),
    (2, 1, 24, 384, 48, 64, 800),
    (1, 1, 1, 128, 16, 16, 40),
    (70, 1, 16, 256, 32, 16, 400),     # more sequences than a warp scans at once
    (200, 1, 8, 512, 64, 64, 700),
    (300, 2, 4, 128, 16, 64, 1900),
    (1, 1, 16, 512, 64, 64, 30000),    # one long cache over every CTA
    (1, 4, 32, 512, 64, 128, 9000),
    (5, 1, 128, 512, 64, 64, 9000),    # few units over many CTAs, some short
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_absorbed(case):
    B, n, nh, dc, dr, page, top = case
    lens = _lens(B, top, B + top)
    lens[-1] = top
    pages, table = latent_state(B, n, dc + dr, page, lens, seed=top, device="cuda")
    q = _q(B, n, nh, dc + dr, top)
    o, lse = _decode(q, pages, table, lens, dc, 0.07)
    check_tree(o, lse, latent_decode_reference(q, pages, table, lens, dc, 0.07), str(case))


@pytest.mark.parametrize("scale", [0.0, -0.05, 0.6])
def test_absorbed_scales(scale):
    pages, table = latent_state(2, 2, 576, 16, [300, 77], seed=1, device="cuda")
    q = _q(2, 2, 16, 576, 1)
    o, lse = _decode(q, pages, table, [300, 77], 512, scale)
    check_tree(o, lse, latent_decode_reference(q, pages, table, [300, 77], 512, scale), f"scale {scale}")


def test_absorbed_growing_scores():
    """Maxima that grow by more than 2^8 from tile to tile, for some heads only, and ones that shrink."""
    lens = [1000, 1000]
    pages, table = latent_state(2, 1, 576, 16, lens, seed=2, device="cuda")
    flat = pages.view(-1, 576)
    q = _q(2, 1, 16, 576, 2, times=2.0)
    for b, flip in ((0, False), (1, True)):
        at = torch.tensor([table[b][p // 16] * 16 + p % 16 for p in range(1001)], device="cuda")
        ramp = torch.linspace(0.02, 2.0, 1001, device="cuda")
        flat[at] = (flat[at].float() * (ramp.flip(0) if flip else ramp)[:, None]).bfloat16()
    q[:, :, 8:] *= 0.01
    o, lse = _decode(q, pages, table, lens, 512, 0.4)
    check_tree(o, lse, latent_decode_reference(q, pages, table, lens, 512, 0.4), "ramp")


def test_absorbed_missing_pages():
    """Entries that are no page hide their positions; a token that sees none gives 0 and -inf."""
    lens = [200, 90, 40, 500]
    pages, table = latent_state(4, 2, 576, 16, lens, seed=3, device="cuda", table_width=34)
    num_pages = pages.shape[0]
    table[0][0], table[0][5], table[0][12] = -1, num_pages, -7
    table[1] = [-1] * 34
    table[2] = [2**30] * 34
    table[3][4:12] = [-1] * 8                              # a tile of 128 positions
    q = _q(4, 2, 16, 576, 3)
    o, lse = _decode(q, pages, table, lens, 512, 0.07)
    check_tree(o, lse, latent_decode_reference(q, pages, table, lens, 512, 0.07), "missing")
    assert not o[1].any() and not o[2].any()


def test_absorbed_lengths_beyond_the_table():
    """Lengths are taken within what the table holds."""
    pages, table = latent_state(3, 2, 144, 16, [30, 30, 0], seed=4, device="cuda")
    q = _q(3, 2, 4, 144, 4)
    o, lse = _decode(q, pages, table, [30, 10**9, -5], 128, 0.1)
    check_tree(o, lse, latent_decode_reference(q, pages, table, [30, 10**9, -5], 128, 0.1), "lengths")


def test_a_sequence_s_bits_do_not_depend_on_the_others_values():
    """The other sequences' rows and queries may be anything, NaN included."""
    lens = [300, 1200, 64, 700]
    pages, table = latent_state(4, 1, 576, 64, lens, seed=5, device="cuda")
    q = _q(4, 1, 16, 576, 5)
    o, lse = _decode(q, pages, table, lens, 512, 0.07)
    for b in (0, 2):
        other = 1 if b != 1 else 0
        rows = [e for e in table[other] if e >= 0]
        dirty, dq = pages.clone(), q.clone()
        dirty[rows] = math.nan
        dq[other] = math.nan
        o2, lse2 = _decode(dq, dirty, table, lens, 512, 0.07)
        assert torch.equal(o2[b], o[b]) and torch.equal(lse2[b], lse[b])
        assert bool(torch.isnan(o2[other]).all())


def test_the_two_forms_agree():
    """The last rows of the expanded form over projected latents, and the absorbed form over the same latents in
    pages. Between them lie roundings of bf16 values that the two take at other places (kv and the absorbed query to
    2^-8 each, P, o and the projection of o): six, each 2^-8 of the values' size, some 2.4 %."""
    from bwd_xattn_fwd_gb300 import xattn
    g = torch.Generator().manual_seed(3)
    B, T, nh, dc, dn, dr, dv, page, n = 2, 300, 16, 256, 64, 32, 64, 16, 4
    rnd = lambda *s, t=0.5: (torch.randn(*s, generator=g) * t).bfloat16().cuda()
    c, rope, q = rnd(B, T, dc), rnd(B, T, dr), rnd(B, T, nh, dn + dr)
    w_k, w_v = rnd(nh, dc, dn, t=dc ** -0.5), rnd(nh, dc, dv, t=dc ** -0.5)
    kv = torch.cat([torch.einsum("bjc,hcd->bjhd", c, w) for w in (w_k, w_v)], 3).contiguous()
    o, lse = xattn.attention_latent_fwd(q, kv, rope)
    width = (T + page - 1) // page
    table = torch.randperm(B * width, generator=g).int().view(B, width).cuda()
    pages = torch.zeros(B * width, page, dc + dr, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(T, device="cuda")
    slots = (table[:, pos // page].long() * page + pos % page).view(-1)
    xattn.latent_write(c.view(-1, dc), rope.view(-1, dr), pages, slots)
    last = q[:, -n:]
    absorbed = torch.cat([torch.einsum("bihd,hcd->bihc", last[..., :dn], w_k), last[..., dn:]], 3).contiguous()
    lat, lse2 = xattn.attention_latent_decode(absorbed, pages, table, _i32([T - n] * B), dc, (dn + dr) ** -0.5)
    out = torch.einsum("bihc,hcd->bihd", lat.float(), w_v.float())
    assert float((out - o[:, -n:].float()).abs().max()) <= 0.024 * float(o.abs().max())
    assert float((lse2 - lse[:, -n:]).abs().max()) <= 0.024
    assert xattn.xattn_check_device_status() == 0


def test_graph_replay_and_streams():
    """Forward, backward and decode captured on a side stream while eager gradients of the same leaves live,
    replayed on new inputs and lengths; an explicit stream."""
    from bwd_xattn_fwd_gb300 import xattn
    x = latent_inputs(2, 300, 3, 64, 32, 64, seed=5)
    eager = _run(x, 0.1)
    lens = _i32([100, 400])
    pages, table = latent_state(2, 1, 576, 16, [500, 500], seed=6, device="cuda")
    table_t, dq_ = _i32(table), _q(2, 1, 16, 576, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = xattn.attention_latent_fwd(x["q"], x["kv"], x["k_rope"], 0.1)
        dq, dkv, drope = xattn.attention_latent_bwd(x["q"], x["kv"], x["k_rope"], o, x["dO"], lse, 0.1)
        od, ld = xattn.attention_latent_decode(dq_, pages, table_t, lens, 512, 0.07)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager["o"]) and torch.equal(dq, eager["dq"]) and torch.equal(drope, eager["dk_rope"])
    y = latent_inputs(2, 300, 3, 64, 32, 64, seed=6)
    for n in x:
        x[n].copy_(y[n])
    lens.copy_(_i32([0, 499]))
    graph.replay()
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    check({"o": o, "lse": lse, "dq": dq, "dkv": dkv, "dk_rope": drope}, latent_reference(y, 0.1), "replay")
    check_tree(od, ld, latent_decode_reference(dq_, pages, table, [0, 499], 512, 0.07), "replayed decode")
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o2, _ = xattn.attention_latent_fwd(x["q"], x["kv"], x["k_rope"], 0.1, stream=other)
    g2 = xattn.attention_latent_bwd(x["q"], x["kv"], x["k_rope"], o, x["dO"], lse, 0.1, stream=other)
    od2, _ = xattn.attention_latent_decode(dq_, pages, table_t, lens, 512, 0.07, stream=other)
    other.synchronize()
    assert torch.equal(o2, o) and torch.equal(g2[1], dkv) and torch.equal(od2, od)


def test_two_graphs_and_two_threads():
    """Two captured graphs in turn and at once, and calls of two host threads on their own streams: scratch is
    each call's own."""
    from bwd_xattn_fwd_gb300 import xattn
    cases = [latent_inputs(2, 400, 4, 128, 64, 128, seed=1), latent_inputs(1, 700, 2, 64, 32, 64, seed=2)]
    dec = []
    for seed in (1, 2):
        pages, table = latent_state(3, 1, 576, 16, [700, 20, 333], seed=seed, device="cuda")
        dec.append((_q(3, 1, 16, 576, seed), pages, _i32(table), _i32([700, 20, 333]), 512, 0.07))

    def work(i):
        x = cases[i]
        o, lse = xattn.attention_latent_fwd(x["q"], x["kv"], x["k_rope"], 0.1)
        return (o, *xattn.attention_latent_bwd(x["q"], x["kv"], x["k_rope"], o, x["dO"], lse, 0.1),
                *xattn.attention_latent_decode(*dec[i]))

    alone = [work(i) for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            outs.append(work(i))
        graphs.append(g)
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    got = [None, None]

    def thread(i):
        with torch.cuda.stream(streams[i]):
            for _ in range(10):
                got[i] = work(i)
            streams[i].synchronize()

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(alone[i], outs[i]))
        assert all(torch.equal(a, b) for a, b in zip(alone[i], got[i]))
    assert xattn.xattn_check_device_status() == 0


def test_a_thread_whose_first_cuda_call_is_the_library_s():
    """A host thread may call without having used CUDA before."""
    from bwd_xattn_fwd_gb300 import xattn
    x = latent_inputs(1, 100, 2, 64, 32, 64, seed=1)
    q, kv, rope = x["q"], x["kv"], x["k_rope"]
    k = torch.randn(1, 100, 2, 64, device="cuda").bfloat16()
    calls = [lambda: xattn.attention_latent_fwd(q, kv, rope, 0.1), lambda: xattn.attention_fwd(k, k, k),
             lambda: xattn.attention_window_fwd(k, k, k, 9)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    for c, (o, lse) in zip(calls, want):
        got = []
        t = threading.Thread(target=lambda: got.append(c()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert got and torch.equal(got[0][0], o) and torch.equal(got[0][1], lse)


FIRST_IN_CAPTURE = """
import torch
from bwd_xattn_fwd_gb300 import xattn
g = torch.Generator(device="cuda").manual_seed(0)
rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
i32 = lambda x: torch.tensor(x, device="cuda", dtype=torch.int32)
q, kv, rope, dO = rnd(2, 200, 2, 96), rnd(2, 200, 2, 128), rnd(2, 200, 32), rnd(2, 200, 2, 64)
table, lens, one = i32([[0, 1, -1, -1], [2, -1, -1, -1]]), i32([17, 5]), i32([1, 1])
free, count = i32([3, 4, 5, -1, -1, -1]), i32([3])
pages, c, r, qd = rnd(6, 16, 144), rnd(2, 128), rnd(2, 16), rnd(2, 1, 4, 144)
pools, new = (rnd(6, 16, 2, 64), rnd(6, 16, 2, 64)), rnd(2, 2, 64)
def calls():
    o, lse = xattn.attention_latent_fwd(q, kv, rope)
    out = [o, lse, *xattn.attention_latent_bwd(q, kv, rope, o, dO, lse)]
    slots, offsets, granted = xattn.cache_reserve(table, lens, one, free, count, 16, 2)
    xattn.latent_write(c, r, pages, slots)
    xattn.cache_write(new, new, *pools, slots)
    out += [slots, offsets, granted, pages.clone(), pools[0].clone(), *xattn.attention_latent_decode(qd, pages, table, lens, 128, 0.1)]
    xattn.cache_release(table, lens + granted, lens, free, count, 16)
    return *out, table.clone(), free.clone(), count.clone()
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
    """The library's first calls in a process may be captured ones."""
    run = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], capture_output=True, text=True, timeout=300,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]


def test_refusals():
    from bwd_xattn_fwd_gb300 import xattn
    x = latent_inputs(1, 20, 2, 64, 32, 64)
    q, kv, rope = x["q"], x["kv"], x["k_rope"]
    with pytest.raises(xattn.XattnError):
        xattn.attention_latent_fwd(q, kv, rope[..., :24].contiguous())      # dr 24, dn 72
    with pytest.raises(TypeError):
        xattn.attention_latent_fwd(q.half(), kv, rope)
    with pytest.raises(ValueError):
        xattn.attention_latent_fwd(q, kv, rope[:, :, ::2])
    with pytest.raises(ValueError):
        xattn.attention_latent_fwd(q.transpose(1, 2), kv, rope)
    with pytest.raises(ValueError):
        xattn.attention_latent_fwd(q, kv[:, :10].contiguous(), rope)
    pages, table = latent_state(1, 1, 576, 16, [30], device="cuda")
    qd = _q(1, 1, 16, 576, 0)
    with pytest.raises(TypeError):
        xattn.attention_latent_decode(qd, pages, _i32(table).long(), _i32([30]), 512, 0.1)
    with pytest.raises(ValueError):
        xattn.attention_latent_decode(qd, pages, _i32(table), _i32([30, 3]), 512, 0.1)
    with pytest.raises(xattn.XattnError):
        xattn.attention_latent_decode(qd, pages, _i32(table), _i32([30]), 500, 0.1)
    with pytest.raises(xattn.XattnError):
        xattn.attention_latent_decode(qd, pages, _i32(table), _i32([30]), 512, math.inf)
