"""The paged cache's tables, slot maps and writes through the binding against plain Python (tests/latent_ref.py):
empty and ragged requests, full pages, too few pages or slots, tables that end, entries that are no page; turns
of a server as a program runs them, eager and captured, with both kinds of cache."""
import random

import pytest
import torch

from latent_ref import latent_decode_reference, release_reference, reserve_reference
from paged_ref import check_tree, tree_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn  # noqa: F401  (fails loudly if not built)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _state(B, width, page, ctx, spare, seed):
    rng = random.Random(seed)
    need = [min((max(c, 0) + page - 1) // page, width) for c in ctx]
    num_pages = sum(need) + spare + 5
    ids = list(range(num_pages))
    rng.shuffle(ids)
    table = [[ids.pop() if j < n else -1 for j in range(width)] for n in need]
    free = [ids.pop() for _ in range(spare)]
    return table, free + [-1] * (num_pages - spare), num_pages


# (B, table width, page, longest context, longest new, spare pages, slot map's length over the tokens)
CASES = [
    (1, 1, 16, 0, 1, 1, 0),
    (1, 3, 16, 20, 0, 2, 3),
    (1, 4, 16, 5, 60, 3, 0),
    (3, 5, 32, 100, 1, 5, 7),
    (64, 66, 64, 4096, 1, 64, 3),
    (65, 9, 16, 100, 40, 30, 0),        # too few pages
    (33, 9, 16, 100, 90, 400, -50),     # the slot map ends inside
    (70, 4, 16, 64, 40, 400, 5),        # tables that end inside the request
    (5, 70, 128, 3000, 5000, 200, 1),
    (1000, 10, 16, 80, 5, 700, 11),
    (1025, 6, 16, 40, 50, 9000, 0),     # more sequences than a block plans at once
    (5000, 4, 16, 30, 3, 1500, 9),
    (20000, 2, 16, 20, 2, 3000, 100),
    (7, 300, 16, 0, 4700, 2500, 2),     # long prompts
    (2, 3, 256, 300, 400, 0, 4),        # no page at all
    (64, 20, 16, 200, 80, 3000, 0),     # a plan and a fill, a release by one block
    (700, 10, 16, 80, 2, 700, 4),       # the other way round
    (9, 40, 16, 300, 40, 100, 2),
    (64, 300, 16, 40, 30, 500, 1),      # few sequences, wide tables
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_reserve_and_release(case):
    from bwd_xattn_fwd_gb300 import xattn
    B, width, page, top, most, spare, over = case
    rng = random.Random(B * 7 + top)
    ctx = [rng.choice([0, top, rng.randint(0, top)]) for _ in range(B)]
    new = [rng.choice([0, most, rng.randint(0, most)]) for _ in range(B)]
    table, free, num_pages = _state(B, width, page, ctx, spare, B)
    tokens = max(sum(new) + over, 0)
    t, f, c = _i32(table), _i32(free), _i32([spare])
    slots, offsets, granted = xattn.cache_reserve(t, _i32(ctx), _i32(new), f, c, page, tokens)
    rt, rc, rs, ro, rg = reserve_reference(table, ctx, new, free, spare, page, tokens, num_pages)
    assert slots.dtype == torch.int64 and slots.tolist() == rs
    assert offsets.tolist() == ro and granted.tolist() == rg
    assert t.tolist() == rt and c.tolist() == [rc] and f.tolist() == free
    # Some of it given back, then all.
    held = [a + g for a, g in zip(ctx, rg)]
    keep = [rng.choice([0, h, rng.randint(0, h + 20)]) for h in held]
    xattn.cache_release(t, _i32(held), _i32(keep), f, c, page)
    bt, bf, bc = release_reference(rt, held, keep, free, rc, page, num_pages)
    assert t.tolist() == bt and f.tolist() == bf and c.tolist() == [bc]
    xattn.cache_release(t, _i32(keep), _i32([0] * B), f, c, page)
    bt, bf, bc = release_reference(bt, keep, [0] * B, bf, bc, page, num_pages)
    assert t.tolist() == bt and f.tolist() == bf and c.tolist() == [bc]


def test_a_release_undoes_a_reserve():
    from bwd_xattn_fwd_gb300 import xattn
    ctx, new = [3, 40, 0, 16], [30, 1, 100, 16]
    table, free, _ = _state(4, 9, 16, ctx, 20, 1)
    t, f, c = _i32(table), _i32(free), _i32([20])
    _, _, granted = xattn.cache_reserve(t, _i32(ctx), _i32(new), f, c, 16, 147)
    assert granted.tolist() == new
    xattn.cache_release(t, _i32(ctx) + granted, _i32(ctx), f, c, 16)
    assert t.tolist() == table and f.tolist() == free and c.tolist() == [20]


def test_odd_lengths_counts_and_entries():
    """Negative lengths, lengths past the table, counts past the stack, entries that are no page, a page given back
    twice: as the plain form."""
    from bwd_xattn_fwd_gb300 import xattn
    table, free, num_pages = _state(4, 3, 16, [48, 20, 0, 10], 12, 2)
    ctx, new = [10**9, -7, 0, 10], [5, 2**31 - 1, -3, 20]
    for count in (-4, 10**6, 3):
        t, f, c = _i32(table), _i32(free), _i32([count])
        slots, offsets, granted = xattn.cache_reserve(t, _i32(ctx), _i32(new), f, c, 16, 100)
        rt, rc, rs, ro, rg = reserve_reference(table, ctx, new, free, count, 16, 100, num_pages)
        assert slots.tolist() == rs and granted.tolist() == rg and t.tolist() == rt and c.tolist() == [rc]
        assert offsets.tolist() == [min(x, 2**31 - 1) for x in ro]
    table[0][1], table[1][0] = num_pages, 2**31 - 1
    held, keep = [10**9, 30, 5, 17], [0, -1, 9, 0]
    for count in (2, num_pages - 2):
        t, f, c = _i32(table), _i32(free), _i32([count])
        xattn.cache_release(t, _i32(held), _i32(keep), f, c, 16)
        bt, bf, bc = release_reference(table, held, keep, free, count, 16, num_pages)
        assert t.tolist() == bt and f.tolist() == bf and c.tolist() == [bc]


@pytest.mark.parametrize("rows,width", [(1, (8, 8)), (3, (512, 64)), (67, (512, 64)), (5000, (128, 16)), (300, (24, 40)),
                                        (40000, (256, 32))], ids=str)
def test_latent_write(rows, width):
    """Rows side by side into their slots; rows without a place are dropped, no other row is touched."""
    from bwd_xattn_fwd_gb300 import xattn
    dc, dr = width
    g = torch.Generator("cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    num_pages, page = rows // 16 + 5, 16
    pages, c, rope = rnd(num_pages, page, dc + dr), rnd(rows, dc), rnd(rows, dr)
    slots = torch.randperm(num_pages * page, generator=torch.Generator().manual_seed(rows))[:rows].cuda()
    slots[rows // 2] = -1
    slots[rows // 3] = num_pages * page
    slots[rows // 5] = 2**62
    want = pages.clone()
    ok = (slots >= 0) & (slots < num_pages * page)
    want.view(-1, dc + dr)[slots[ok]] = torch.cat([c, rope], 1)[ok]
    version = pages._version
    xattn.latent_write(c, rope, pages, slots)
    assert torch.equal(pages, want) and pages._version > version


@pytest.mark.parametrize("rows,nkv,hd", [(1, 1, 8), (5, 2, 64), (70, 3, 24), (4096, 4, 128), (30000, 1, 32)], ids=str)
def test_cache_write(rows, nkv, hd):
    from bwd_xattn_fwd_gb300 import xattn
    g = torch.Generator("cuda").manual_seed(rows)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    num_pages, page = rows // 32 + 5, 32
    kp, vp, k, v = rnd(num_pages, page, nkv, hd), rnd(num_pages, page, nkv, hd), rnd(rows, nkv, hd), rnd(rows, nkv, hd)
    slots = torch.randperm(num_pages * page, generator=torch.Generator().manual_seed(rows))[:rows].cuda()
    slots[rows // 2] = -1
    ok = slots >= 0
    want = kp.clone(), vp.clone()
    want[0].view(-1, nkv, hd)[slots[ok]] = k[ok]
    want[1].view(-1, nkv, hd)[slots[ok]] = v[ok]
    xattn.cache_write(k, v, kp, vp, slots)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


def test_nothing_to_write():
    from bwd_xattn_fwd_gb300 import xattn
    pages = torch.ones(3, 16, 144, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    xattn.latent_write(pages.new_empty(0, 128), pages.new_empty(0, 16), pages, none)
    assert bool((pages == 1).all())
    slots, offsets, granted = xattn.cache_reserve(_i32([[-1]]), _i32([0]), _i32([0]), _i32([0, 1]), _i32([2]), 16, 0)
    assert slots.numel() == 0 and offsets.tolist() == [0, 0] and granted.tolist() == [0]


def test_refusals():
    from bwd_xattn_fwd_gb300 import xattn
    t, x, f, c = _i32([[-1, -1]]), _i32([0]), _i32([0, 1]), _i32([2])
    with pytest.raises(xattn.XattnError):
        xattn.cache_reserve(t, x, x, f, c, 17, 4)
    with pytest.raises(xattn.XattnError):
        xattn.cache_reserve(t, x, x, f, c, 16, -1)
    with pytest.raises(ValueError):
        xattn.cache_reserve(t, x, f, f, c, 16, 4)
    with pytest.raises(ValueError):
        xattn.cache_release(t, x, x, f, f, 16)
    with pytest.raises(ValueError):
        xattn.cache_release(t.T, x, x, f, c, 16)
    with pytest.raises(TypeError):
        xattn.cache_reserve(t, x.long(), x, f, c, 16, 4)
    with pytest.raises(xattn.XattnError):
        xattn.latent_write(torch.zeros(1, 12, device="cuda").bfloat16(), torch.zeros(1, 4, device="cuda").bfloat16(),
                           torch.zeros(1, 16, 16, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int64, device="cuda"))


def _rows(table, b, T, page):
    return torch.tensor([table[b][p // page] * page + p % page for p in range(T)], device="cuda")


@pytest.mark.parametrize("captured", [False, True])
def test_a_server_s_turns(captured):
    """Ragged prompts reserved and written, then decode turns (reserve, write, attend), one request ended and
    another begun: attention over a latent cache and over a K/V cache with one table, against the plain forms
    over what was written. The turns may be one captured graph, replayed."""
    from bwd_xattn_fwd_gb300 import xattn
    B, page, width, num_pages, dc, dr, nh, nkv, hd = 3, 16, 8, 20, 128, 16, 8, 2, 64
    g = torch.Generator("cuda").manual_seed(0)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.5).bfloat16()
    table, free, count = _i32([[-1] * width] * B), torch.arange(num_pages, dtype=torch.int32, device="cuda"), _i32([num_pages])
    lens = _i32([0] * B)
    pages = torch.full((num_pages, page, dc + dr), float("nan"), device="cuda").bfloat16()
    kp, vp = (torch.full((num_pages, page, nkv, hd), float("nan"), device="cuda").bfloat16() for _ in range(2))
    history = [{"lat": [], "k": [], "v": []} for _ in range(B)]

    def remember(lat, rope, k, v, counts):
        at = 0
        for b, n in enumerate(counts):
            history[b]["lat"].append(torch.cat([lat, rope], 1)[at:at + n].clone())
            history[b]["k"].append(k[at:at + n].clone())
            history[b]["v"].append(v[at:at + n].clone())
            at += n

    def prompt(new):
        total = sum(new)
        c, rope, k, v = rnd(total, dc), rnd(total, dr), rnd(total, nkv, hd), rnd(total, nkv, hd)
        slots, _, granted = xattn.cache_reserve(table, lens, _i32(new), free, count, page, total)
        xattn.latent_write(c, rope, pages, slots)
        xattn.cache_write(k, v, kp, vp, slots)
        lens.add_(granted)
        assert granted.tolist() == new
        remember(c, rope, k, v, new)

    prompt([40, 0, 17])
    c, rope, k, v = rnd(B, dc), rnd(B, dr), rnd(B, nkv, hd), rnd(B, nkv, hd)
    q, qk = rnd(B, 1, nh, dc + dr), rnd(B, 1, nh, hd)
    one = _i32([1] * B)

    def turn():
        slots, _, granted = xattn.cache_reserve(table, lens, one, free, count, page, B)
        xattn.latent_write(c, rope, pages, slots)
        xattn.cache_write(k, v, kp, vp, slots)
        out = (*xattn.attention_latent_decode(q, pages, table, lens, dc, 0.1),
               *xattn.attention_tree_decode(qk, kp, vp, table, lens))
        lens.add_(granted)
        return out

    graph, out = None, None
    if captured:
        saved = [x.clone() for x in (table, free, count, lens, pages, kp, vp)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = turn()
        for x, s in zip((table, free, count, lens, pages, kp, vp), saved):
            assert torch.equal(x.view(torch.int16) if x.is_floating_point() else x,
                               s.view(torch.int16) if s.is_floating_point() else s)     # a capture runs nothing
    for step in range(20):
        for x in (c, rope, k, v, q, qk):
            x.copy_(rnd(*x.shape))
        remember(c, rope, k, v, [1] * B)
        if captured:
            graph.replay()
        else:
            out = turn()
        if step == 9:                                       # the first request ends, another takes its place
            xattn.cache_release(table, lens, lens * _i32([0, 1, 1]), free, count, page)
            lens.mul_(_i32([0, 1, 1]))
            history[0] = {"lat": [], "k": [], "v": []}
            prompt([50, 0, 0])
            continue
        if step not in (0, 8, 10, 19):
            continue
        tl, before = table.tolist(), (lens - 1).tolist()
        for b in range(B):
            T = lens[b].item()
            at = _rows(tl, b, T, page)
            assert torch.equal(pages.view(-1, dc + dr)[at], torch.cat(history[b]["lat"]))
            assert torch.equal(kp.view(-1, nkv, hd)[at], torch.cat(history[b]["k"]))
            assert torch.equal(vp.view(-1, nkv, hd)[at], torch.cat(history[b]["v"]))
        check_tree(out[0], out[1], latent_decode_reference(q, pages, tl, before, dc, 0.1), f"latent, step {step}")
        check_tree(out[2], out[3], tree_reference(qk, kp, vp, tl, before, None, 10**6, 0, hd ** -0.5), f"K/V, step {step}")
    used = sum((n + page - 1) // page for n in lens.tolist())
    assert count.item() == num_pages - used
    held = [e for r in table.tolist() for e in r if e >= 0] + free.tolist()[:count.item()]
    assert sorted(held) == list(range(num_pages))           # every page once
    assert xattn.xattn_check_device_status() == 0
