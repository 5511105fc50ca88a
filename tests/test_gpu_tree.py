"""Tree attention over a paged cache and the cache's page operations through the binding,
against plain forms (tests/paged_ref.py): ragged and empty caches, pages that end inside tiles,
rows that hold NaN wherever no token looks, freed pages, windows and sinks, words that see
nothing, odd groups; a turn of drafted decoding as a program runs it; graphs and streams."""
import math
import random

import pytest
import torch

from paged_ref import (append_reference, check_tree, compact_reference, paged_state, random_words, signed,
                       tree_reference)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn  # noqa: F401  (fails loudly if not built)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _q(B, n, nh, hd, seed):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn(B, n, nh, hd, generator=g) * 0.5).to(torch.bfloat16).cuda()


def _attend(q, k, v, table, lens, words, window, sinks, scale=None):
    from bwd_xattn_fwd_gb300 import xattn
    tree = None if words is None else torch.tensor(signed(words), device="cuda")
    o, lse = xattn.attention_tree_decode(q, k, v, _i32(table), _i32(lens), tree=tree, window=window, sinks=sinks,
                                         scale=scale)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    return o, lse


def _lens(B, top, seed):
    rng = random.Random(seed)
    return [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(B)]


BIG = 2**31 - 1
# (B, n, nh, nkv, hd, page, longest cache, window, sinks)
CASES = [
    (1, 1, 1, 1, 64, 16, 0, BIG, 0),
    (1, 1, 4, 1, 64, 16, 5, BIG, 0),
    (3, 1, 8, 2, 64, 64, 300, BIG, 0),
    (2, 5, 8, 2, 64, 16, 127, BIG, 0),
    (2, 3, 4, 4, 32, 32, 128, BIG, 0),
    (4, 8, 16, 4, 64, 128, 700, BIG, 0),
    (2, 7, 6, 2, 128, 16, 500, BIG, 0),
    (2, 64, 4, 4, 64, 16, 333, BIG, 0),
    (2, 64, 16, 2, 64, 64, 600, BIG, 0),       # 512 rows a kv head: four row tiles
    (2, 27, 14, 2, 32, 16, 450, BIG, 0),       # a group of 7: rows end inside a tile
    (2, 61, 8, 1, 128, 256, 700, BIG, 0),      # pages wider than a tile
    (1, 2, 2, 1, 64, 384, 1000, BIG, 0),
    (3, 1, 8, 2, 64, 16, 900, 1, 0),           # a window of the token alone
    (3, 4, 8, 2, 64, 16, 900, 4, 3),
    (3, 1, 8, 2, 128, 16, 1500, 129, 4),
    (2, 16, 8, 2, 64, 32, 2000, 300, 130),
    (2, 9, 4, 2, 32, 64, 1200, 128, 128),
    (3, 5, 4, 2, 64, 16, 600, 200, 5000),      # more sinks than positions
    (70, 2, 8, 2, 64, 16, 400, BIG, 0),        # more sequences than a warp scans at once
    (200, 1, 4, 4, 32, 32, 900, 256, 4),
    (300, 2, 2, 1, 64, 64, 1900, BIG, 0),      # more sequences than a warp's lanes hold at once
    (300, 2, 2, 1, 32, 64, 9000, BIG, 0),      # the same with some far longer than most: units cut
    (1, 4, 4, 1, 64, 64, 30000, BIG, 0),       # one long cache over every CTA
    (5, 16, 8, 2, 64, 64, 9000, BIG, 0),       # few units over many CTAs, some short
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("shape", ["tree", "run"])
def test_tree_attention(case, shape):
    B, n, nh, nkv, hd, page, top, window, sinks = case
    lens = _lens(B, top, seed=top + n)
    lens[0] = top
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=7, device="cuda")
    words = random_words(B, n, seed=3) if shape == "tree" else None
    q = _q(B, n, nh, hd, seed=n)
    o, lse = _attend(q, k, v, table, lens, words, window, sinks)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, words, window, sinks, hd ** -0.5), f"{case} {shape}")


def test_words_that_see_nothing():
    """With an empty cache a word of zero sees nothing: o = 0, lse = -inf; arbitrary words
    (without the token's own bit, with bits past n) mean what their bits say."""
    B, n, nh, nkv, hd, page = 4, 6, 8, 2, 64, 16
    lens = [0, 0, 50, 200]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=1, device="cuda")
    words = [[0, 0, 0, 0, 0, 0], [0, 1, 0, 0b100000, 0b111, ~0 & (2**64 - 1)], [0] * 6, [2, 1, 0, 5 << 40, 63, 8]]
    q = _q(B, n, nh, hd, seed=2)
    o, lse = _attend(q, k, v, table, lens, words, BIG, 0)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, words, BIG, 0, hd ** -0.5), "words")
    assert bool((o[0] == 0).all()) and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("hd,page", [(64, 16), (128, 32), (32, 128)])
def test_missing_pages_and_lengths_out_of_range(hd, page):
    """Entries outside the pool hold no positions (-1, the pool's size, the extremes of int32);
    lengths are taken within what the table holds."""
    B, n, nh, nkv = 5, 3, 4, 2
    lens = [400, 130, 390, 64, 256]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=5, device="cuda")
    num_pages = k.shape[0]
    table[0][1] = -1
    table[1][0] = num_pages
    table[2] = [-(2**31)] * len(table[2])
    table[3][0] = 2**31 - 1
    q = _q(B, n, nh, hd, seed=8)
    for words in (None, random_words(B, n, 1)):
        o, lse = _attend(q, k, v, table, lens, words, BIG, 0)
        check_tree(o, lse, tree_reference(q, k, v, table, lens, words, BIG, 0, hd ** -0.5), "missing pages")
    k, v, table = paged_state(2, n, nkv, hd, page, [200, 300], seed=5, device="cuda")
    cap = len(table[0]) * page
    k.nan_to_num_(nan=0.25)
    v.nan_to_num_(nan=0.25)
    q = _q(2, n, nh, hd, seed=8)
    wild = [-5, cap + 1000]
    o, lse = _attend(q, k, v, table, wild, None, BIG, 0)
    check_tree(o, lse, tree_reference(q, k, v, table, wild, None, BIG, 0, hd ** -0.5), "lengths")


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("sinks", [0, 4])
def test_pages_behind_the_window_may_be_freed(n, sinks):
    """The answer does not change when pages that no token sees are freed (-1) or point at a page
    that now holds NaN."""
    B, nh, nkv, hd, page, window = 3, 8, 2, 64, 16, 200
    lens = [1000, 450, 777]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=4, device="cuda")
    q = _q(B, n, nh, hd, seed=4)
    o, lse = _attend(q, k, v, table, lens, None, window, sinks)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, None, window, sinks, hd ** -0.5), "kept")
    stale = k.shape[0]
    k2 = torch.cat([k, torch.full_like(k[:1], math.nan)])
    v2 = torch.cat([v, torch.full_like(v[:1], math.nan)])
    for b in range(B):
        for e in range(len(table[b])):
            if e * page >= sinks and (e + 1) * page <= lens[b] - window + 1:
                table[b][e] = -1 if e % 2 else stale
    o2, lse2 = _attend(q, k2, v2, table, lens, None, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("scale", [0.0, -0.5, 3.0])
def test_scales(scale):
    B, n, nh, nkv, hd, page, lens = 2, 4, 4, 2, 64, 32, [300, 90]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=2, device="cuda")
    q, words = _q(B, n, nh, hd, 1), random_words(B, n, 2)
    o, lse = _attend(q, k, v, table, lens, words, BIG, 0, scale=scale)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, words, BIG, 0, scale), f"scale {scale}")


def test_shared_pages_and_the_contiguous_decode():
    """Sequences that share their prefix's pages; and a cache laid out in order agrees with
    xattn_decode within both bounds (bf16 rounding of o and of P: 2^-7 of sum p |v| <= max |v|)."""
    from bwd_xattn_fwd_gb300 import xattn
    B, nh, nkv, hd, page, T = 4, 8, 2, 64, 64, 640
    k, v, table = paged_state(B, 1, nkv, hd, page, [T - 1] * B, seed=6, device="cuda", spare=0)
    for b in range(1, B):
        table[b][:4] = table[0][:4]
    q = _q(B, 1, nh, hd, 3)
    lens = [T - 1] * B
    o, lse = _attend(q, k, v, table, lens, None, BIG, 0)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, None, BIG, 0, hd ** -0.5), "shared")
    idx = torch.tensor(table, device="cuda")
    kc, vc = (p[idx].view(B, T, nkv, hd).contiguous() for p in (k, v))
    oc, lc = xattn.attention_decode(q[:, 0].contiguous(), kc, vc)
    assert float((oc.float() - o[:, 0].float()).abs().max()) <= 2 * 2.0 ** -7 * float(vc.float().abs().max())
    assert float((lc - lse[:, 0]).abs().max()) <= 2.0 ** -8


def test_reproducible_and_rows_of_other_sequences_do_not_matter():
    B, n, nh, nkv, hd, page = 9, 4, 8, 2, 64, 16
    lens = _lens(B, 800, 5)
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=9, device="cuda")
    q, words = _q(B, n, nh, hd, 5), random_words(B, n, 5)
    a = _attend(q, k, v, table, lens, words, 300, 4)
    b = _attend(q, k, v, table, lens, words, 300, 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


PAGE_CASES = [(1, 1, 1, 8, 16, [0]), (3, 1, 2, 64, 16, [5, 0, 31]), (2, 37, 4, 32, 32, [0, 63]),
              (5, 16, 1, 128, 64, [1, 64, 100, 7, 0]), (2, 300, 3, 24, 128, [17, 250]), (4, 64, 8, 128, 16, [9, 0, 3, 200])]


@pytest.mark.parametrize("case", PAGE_CASES, ids=str)
def test_append(case):
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nkv, hd, page, lens = case
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=n, device="cuda")
    k.nan_to_num_(nan=7.0)
    v.nan_to_num_(nan=9.0)
    if B > 2:
        table[1][lens[1] // page] = -1               # rows without a page are dropped
        table[2][lens[2] // page] = k.shape[0]
    g = torch.Generator().manual_seed(n)
    kn, vn = (torch.randn(B, n, nkv, hd, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    rk, rv = append_reference(kn, vn, k, v, table, lens)
    xattn.cache_append(kn, vn, k, v, _i32(table), _i32(lens))
    assert torch.equal(k, rk) and torch.equal(v, rv)
    # past the table's end, and before position 0: the rows that have no place are dropped
    far = [len(table[0]) * page - (n + 1) // 2] * B
    far[-1] = -(n // 2)
    rk, rv = append_reference(vn, kn, k, v, table, far)
    xattn.cache_append(vn, kn, k, v, _i32(table), _i32(far))
    assert torch.equal(k, rk) and torch.equal(v, rv)


@pytest.mark.parametrize("case", [c for c in PAGE_CASES if c[1] <= 64], ids=str)
def test_compact(case):
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nkv, hd, page, lens = case
    rng = random.Random(n)
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=n, device="cuda")
    k.nan_to_num_(nan=7.0)
    v.nan_to_num_(nan=9.0)
    for accepted in ([n] * B, [min(n, rng.randint(0, 12)) for _ in range(B)], [0] * B, [n + 5] + [-3] * (B - 1)):
        path = [sorted(rng.sample(range(n), min(max(a, 0), n))) + [0] * (n - min(max(a, 0), n)) for a in accepted]
        rk, rv = compact_reference(k, v, table, lens, path, accepted)
        xattn.cache_compact(k, v, _i32(table), _i32(lens), _i32(path), _i32(accepted))
        assert torch.equal(k, rk) and torch.equal(v, rv), accepted
    # a path that skips far ahead, an entry past n, one below its place
    path = [[min(n - 1, i + n // 2) for i in range(n)] for _ in range(B)]
    path[0] = [n + 3] * n
    accepted = [min(n, n // 2 + 1)] * B
    if B > 2:
        table[2][lens[2] // page] = -1
    rk, rv = compact_reference(k, v, table, lens, path, accepted)
    xattn.cache_compact(k, v, _i32(table), _i32(lens), _i32(path), _i32(accepted))
    assert torch.equal(k, rk) and torch.equal(v, rv)


def test_a_turn_of_drafted_decoding():
    """A windowed model's program: a prompt through the window forward and into the pages, a tree
    drafted and attended, its accepted path kept, then one more token; each token's output equals
    the window forward's of the sequence that was accepted (both within bf16's bounds of the
    definition, which the reference is)."""
    from bwd_xattn_fwd_gb300 import xattn
    from window_ref import reference
    B, P, n, nh, nkv, hd, page, window, sinks = 2, 150, 6, 8, 2, 64, 16, 70, 3
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: (torch.randn(*s, generator=g) * 0.5).to(torch.bfloat16).cuda()  # noqa: E731
    k, v, table = paged_state(B, 20, nkv, hd, page, [P] * B, seed=1, device="cuda")
    k.fill_(math.nan)
    v.fill_(math.nan)
    tb, zero = _i32(table), _i32([0] * B)
    qp, kp, vp = rnd(B, P, nh, hd), rnd(B, P, nkv, hd), rnd(B, P, nkv, hd)
    xattn.attention_window_fwd(qp, kp, vp, window, sinks)
    xattn.cache_append(kp, vp, k, v, tb, zero)
    # tree: 0 -> {1, 2}, 2 -> {3, 4}, 4 -> 5; accepted: 0, 2, 4
    words = [[0b1, 0b11, 0b101, 0b1101, 0b10101, 0b110101]] * B
    path = [0, 2, 4]
    lens = _i32([P] * B)
    qd, kd, vd = rnd(B, n, nh, hd), rnd(B, n, nkv, hd), rnd(B, n, nkv, hd)
    xattn.cache_append(kd, vd, k, v, tb, lens)
    o, lse = xattn.attention_tree_decode(qd, k, v, tb, lens, tree=torch.tensor(words, device="cuda"), window=window,
                                         sinks=sinks)
    xattn.cache_compact(k, v, tb, lens, _i32([path + [0] * 3] * B), _i32([3] * B))
    lens = lens + 3
    q1, k1, v1 = rnd(B, 1, nh, hd), rnd(B, 1, nkv, hd), rnd(B, 1, nkv, hd)
    xattn.cache_append(k1, v1, k, v, tb, lens)
    o1, lse1 = xattn.attention_tree_decode(q1, k, v, tb, lens, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    seq = {"q": torch.cat([qp, qd[:, path], q1], 1), "k": torch.cat([kp, kd[:, path], k1], 1),
           "v": torch.cat([vp, vd[:, path], v1], 1)}
    seq["dO"] = torch.zeros_like(seq["q"])
    ref = reference(seq, window, sinks, hd ** -0.5, True)
    got_o, got_l = torch.cat([o[:, path], o1], 1).double(), torch.cat([lse[:, path], lse1], 1).double()
    val, err = ref["o"]
    assert float(((got_o - val[:, P:]).abs() / err[:, P:]).max()) <= 1.0
    assert float((got_l - ref["lse"][0][:, P:]).abs().max()) <= float(ref["lse"][1].max())


def test_graphs_follow_lengths_and_two_graphs_do_not_meet():
    """Two captured turns on two streams replayed together, after the lengths and the table have
    changed under them."""
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nh, nkv, hd, page = 3, 4, 8, 2, 64, 16
    states = []
    for seed in (1, 2):
        k, v, table = paged_state(B, n, nkv, hd, page, [900, 50, 400], seed=seed, device="cuda")
        words = random_words(B, n, seed)
        s = dict(k=k, v=v, table=table, tb=_i32(table), lens=_i32([5, 50, 100]), q=_q(B, n, nh, hd, seed), words=words,
                 tree=torch.tensor(signed(words), device="cuda"), stream=torch.cuda.Stream(),
                 graph=torch.cuda.CUDAGraph())
        states.append(s)
    call = lambda s: xattn.attention_tree_decode(s["q"], s["k"], s["v"], s["tb"], s["lens"], tree=s["tree"])  # noqa: E731
    call(states[0])
    torch.cuda.synchronize()
    for s in states:
        with torch.cuda.graph(s["graph"], stream=s["stream"]):
            s["o"], s["lse"] = call(s)
    new = [900, 50, 400]
    for s in states:
        s["lens"].copy_(_i32(new))
    torch.cuda.synchronize()
    for _ in range(3):
        for s in states:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    for s in states:
        check_tree(s["o"], s["lse"], tree_reference(s["q"], s["k"], s["v"], s["table"], new, s["words"], BIG, 0,
                                                    hd ** -0.5), "graph")


def test_a_graph_whose_lengths_even_out():
    """200 units of (sequence, kv head): a few long caches among short ones are cut into runs, even
    ones are not; one captured call takes both, in either order."""
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nh, nkv, hd, page = 50, 2, 4, 4, 64, 64
    even, uneven = [2000 - b for b in range(B)], [6000 if b % 20 == 3 else b for b in range(B)]
    k, v, table = paged_state(B, n, nkv, hd, page, [max(x) for x in zip(even, uneven)], seed=5, device="cuda")
    width = max(len(r) for r in table)
    table = [r + [-1] * (width - len(r)) for r in table]
    q, tb, lens = _q(B, n, nh, hd, 3), _i32(table), _i32(even)
    graph = torch.cuda.CUDAGraph()
    xattn.attention_tree_decode(q, k, v, tb, lens)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        o, lse = xattn.attention_tree_decode(q, k, v, tb, lens)
    for now in (even, uneven, even):
        lens.copy_(_i32(now))
        graph.replay()
        torch.cuda.synchronize()
        assert xattn.xattn_check_device_status() == 0
        check_tree(o, lse, tree_reference(q, k, v, table, now, None, BIG, 0, hd ** -0.5), "even" if now is even else "uneven")


def test_explicit_streams_by_object_and_handle():
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nh, nkv, hd, page, lens = 2, 4, 4, 2, 64, 16, [100, 60]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=2, device="cuda")
    q, tb, ln = _q(B, n, nh, hd, 1), _i32(table), _i32(lens)
    ref, rl = xattn.attention_tree_decode(q, k, v, tb, ln)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        o, lse = xattn.attention_tree_decode(q, k, v, tb, ln, stream=stream)
        side.synchronize()
        assert torch.equal(o, ref) and torch.equal(lse, rl)


def test_tensors_that_do_not_fit_are_refused_and_nothing_is_written():
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nh, nkv, hd, page, lens = 2, 4, 4, 2, 64, 16, [100, 60]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=2, device="cuda")
    q, tb, ln = _q(B, n, nh, hd, 1), _i32(table), _i32(lens)
    words = torch.ones(B, n, dtype=torch.int64, device="cuda")
    call = xattn.attention_tree_decode
    for bad in ((q.float(), k, v, tb, ln), (q, k.half(), v, tb, ln), (q, k, v, tb.long(), ln), (q, k, v, tb, ln.float()),
                ("q", k, v, tb, ln)):
        with pytest.raises((TypeError, ValueError)):
            call(*bad)
    for bad in ((q[:1], k, v, tb, ln), (q, k, v[:-1], tb, ln), (q, k, v, tb, ln[:1]), (q.cpu(), k, v, tb, ln),
                (q, k, v, tb.cpu(), ln), (q[..., ::2], k, v, tb, ln), (q.transpose(1, 2), k, v, tb, ln),
                (q, k, v, tb[:, ::2], ln), (q[0], k, v, tb, ln), (q, k[0], v, tb, ln)):
        with pytest.raises(ValueError):
            call(*bad)
    with pytest.raises(ValueError):
        call(q, k, v, tb, ln, tree=words[:, :2])
    with pytest.raises(TypeError):
        call(q, k, v, tb, ln, tree=words.int())
    with pytest.raises(xattn.XattnError) as err:
        call(q, k, v, tb, ln, window=3)                               # a window that ends inside the tree
    assert err.value.status == xattn.Status.ERR_WINDOW
    with pytest.raises(xattn.XattnError) as err:
        call(q[:, :, :3].contiguous(), k, v, tb, ln)
    assert err.value.status == xattn.Status.ERR_GROUP
    with pytest.raises(xattn.XattnError) as err:
        call(q, k, v, tb, ln, scale=float("nan"))
    assert err.value.status == xattn.Status.ERR_BAD_SCALE
    before = k.clone(), v.clone()
    new = torch.zeros(B, n, nkv, hd, dtype=torch.bfloat16, device="cuda")
    for bad in ((new.float(), new), (new, new[:, :2]), (new[..., :32], new[..., :32]), (new.cpu(), new)):
        with pytest.raises((TypeError, ValueError)):
            xattn.cache_append(*bad, k, v, tb, ln)
    path, acc = _i32([[0, 1, 2, 3]] * B), _i32([1, 1])
    for bad in ((path.long(), acc), (path, acc[:1]), (path[:, ::2], acc), (path[0], acc), (path.cpu(), acc)):
        with pytest.raises((TypeError, ValueError)):
            xattn.cache_compact(k, v, tb, ln, *bad)
    with pytest.raises(xattn.XattnError) as err:                      # more rows than the table holds
        xattn.cache_append(*(torch.zeros(B, 500, nkv, hd, dtype=torch.bfloat16, device="cuda"),) * 2, k, v, tb, ln)
    assert err.value.status == xattn.Status.ERR_PAGES
    torch.cuda.synchronize()
    assert torch.equal(k.view(torch.int16), before[0].view(torch.int16))
    assert torch.equal(v.view(torch.int16), before[1].view(torch.int16))


def _hide(k, v, table, lens, words, window, sinks, page, n):
    """NaN in K and V of every position of the sequences that no token sees."""
    hidden = 0
    for b, ctx in enumerate(lens):
        seen = 0
        for w in words[b]:
            w &= (1 << n) - 1
            near = max(ctx + max(bin(w).count("1") - 1, 0) - window + 1, 0)
            seen |= ((1 << ctx) - 1) & ~((1 << min(near, ctx)) - 1) | (1 << min(sinks, ctx)) - 1 | w << ctx
        rows = [table[b][p // page] * page + p % page for p in range(ctx + n) if not (seen >> p) & 1]
        hidden += len(rows)
        for pool in (k, v):
            pool.view(-1, *pool.shape[2:])[rows] = math.nan
    return hidden


# (B, n, nh, nkv, hd, page, longest cache, window, sinks): tiles of 32, 64 and 128 rows, and several;
# whole units (short tables), cut ones, and calls that choose
UNSEEN_CASES = [
    (3, 8, 4, 1, 64, 16, 500, BIG, 0),
    (3, 6, 4, 1, 32, 32, 700, 90, 3),
    (5, 16, 16, 4, 64, 64, 3000, BIG, 0),
    (5, 16, 16, 4, 128, 16, 2500, 300, 4),
    (4, 9, 14, 2, 32, 16, 900, 70, 0),
    (4, 30, 16, 4, 64, 16, 1500, 200, 100),
    (3, 64, 8, 2, 64, 128, 600, BIG, 0),
    (3, 61, 16, 2, 128, 64, 3000, 500, 4),
    (60, 8, 16, 4, 64, 64, 1800, BIG, 0),
    (60, 12, 16, 4, 64, 16, 1800, 128, 4),
]


@pytest.mark.parametrize("case", UNSEEN_CASES, ids=str)
def test_positions_that_no_token_sees_may_hold_nan(case):
    """A batch of trees of different sizes: spare tokens have words of 0 and rows that nobody wrote;
    tokens that no word names; and trees without a token of depth 0, whose windows all end before
    the first token's would."""
    B, n, nh, nkv, hd, page, top, window, sinks = case
    rng = random.Random(n)
    lens = [top - 37 * b % (top // 2) for b in range(B)]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=n, device="cuda")
    words = random_words(B, n, seed=5)
    for b in range(B):
        if b % 3 == 0:                                   # a smaller tree
            words[b][rng.randint(1, n - 1):] = [0] * n
            del words[b][n:]
        elif b % 3 == 1:                                 # token n - 2 named by nobody, not by itself
            words[b] = [w & ~(1 << (n - 2)) for w in words[b]]
        else:                                            # every token has at least three ancestors
            words[b] = [w | 0b1111 for w in words[b]]
    assert _hide(k, v, table, lens, words, window, sinks, page, n) >= 2
    q = _q(B, n, nh, hd, seed=n)
    o, lse = _attend(q, k, v, table, lens, words, window, sinks)
    check_tree(o, lse, tree_reference(q, k, v, table, lens, words, window, sinks, hd ** -0.5), str(case))


@pytest.mark.parametrize("n,nh,hd,top", [(4, 4, 64, 600), (4, 4, 64, 20000), (12, 4, 32, 9000), (40, 4, 128, 9000),
                                         (40, 4, 64, 700)])
def test_scores_that_are_no_numbers_are_not_rows_that_see_nothing(n, nh, hd, top):
    """A query that holds NaN, and one whose scores overflow: o and lse of those rows are NaN, as a
    softmax in fp32 gives them, and not the 0 and -inf of a row that sees nothing; other rows are
    as right as without them."""
    B, nkv, page, lens = 2, 1, 64, [top, top // 3]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=6, device="cuda")
    q = _q(B, n, nh, hd, seed=6)
    bad = torch.zeros(B, n, nh, dtype=torch.bool, device="cuda")
    bad[0, 1, 2] = bad[1, n - 1, 0] = True
    q[0, 1, 2, 5] = math.nan
    q[1, n - 1, 0] = 3e38
    k.masked_fill_(k.isnan(), 0.0)
    for b in range(B):                                   # one key of large numbers: q . k is +inf for that query
        k.view(-1, nkv, hd)[table[b][0] * page + 3] = 2.0
    o, lse = _attend(q, k, v, table, lens, None, BIG, 0)
    assert bool(o[bad].isnan().all()) and bool(lse[bad].isnan().all())
    q[bad] = 0.0
    ref = tree_reference(q, k, v, table, lens, None, BIG, 0, hd ** -0.5)
    o[bad], lse[bad] = ref[0][0][bad].to(o.dtype), ref[1][0][bad].float()
    check_tree(o, lse, ref, "the other rows")


@pytest.mark.parametrize("case", [(6, 4, 4, 1, 64, 16, 700), (6, 4, 16, 4, 128, 64, 4000), (5, 16, 16, 4, 64, 64, 5000),
                                  (9, 14, 8, 2, 32, 32, 3000), (5, 48, 16, 2, 64, 16, 2500), (4, 64, 4, 2, 128, 64, 900),
                                  (70, 8, 8, 2, 64, 64, 1700)], ids=str)
def test_a_sequence_does_not_depend_on_the_others(case):
    """Units of different sequences share a CTA's tiles and the records of cut ones: with the lengths
    as they were, new K, V and queries of all other sequences leave a sequence's bits alone."""
    B, n, nh, nkv, hd, page, top = case
    lens = [top - 61 * b % (top // 2) for b in range(B)]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=3, device="cuda")
    q, words = _q(B, n, nh, hd, 3), random_words(B, n, 3)
    o, lse = _attend(q, k, v, table, lens, words, BIG, 0)
    g = torch.Generator("cuda").manual_seed(1)
    for kept in (0, B // 2, B - 1):
        pages = torch.tensor([e for e in table[kept] if e >= 0], device="cuda")
        k2, v2, q2 = (torch.randn(t.shape, generator=g, device="cuda").to(t.dtype) for t in (k, v, q))
        k2[pages], v2[pages], q2[kept] = k[pages], v[pages], q[kept]
        o2, lse2 = _attend(q2, k2, v2, table, lens, words, BIG, 0)
        assert torch.equal(o2[kept], o[kept]) and torch.equal(lse2[kept], lse[kept])
        assert not torch.equal(o2[kept - 1], o[kept - 1])


def test_page_calls_tell_autograd_that_they_write():
    """append and compact raise the pools' version counters as in-place operations do; a refused call
    does not, and inference tensors (which have none) are taken."""
    from bwd_xattn_fwd_gb300 import xattn
    B, n, nkv, hd, page, lens = 2, 4, 2, 64, 16, [10, 0]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=2, device="cuda")
    new = torch.zeros(B, n, nkv, hd, dtype=torch.bfloat16, device="cuda")
    tb, ln, path, acc = _i32(table), _i32(lens), _i32([[0, 2, 3, 0]] * B), _i32([3, 1])
    weight = torch.ones(hd, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    product = weight * k.nan_to_num_(0.0)                          # saves k for its backward
    at = k._version, v._version
    with pytest.raises(ValueError):
        xattn.cache_append(new, new[:, :2], k, v, tb, ln)
    assert (k._version, v._version) == at
    xattn.cache_append(new, new, k, v, tb, ln)
    assert k._version > at[0] and v._version > at[1]
    at = k._version, v._version
    xattn.cache_compact(k, v, tb, ln, path, acc)
    assert k._version > at[0] and v._version > at[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        product.sum().backward()
    with torch.inference_mode():
        ki, vi = k.clone(), v.clone()
        xattn.cache_append(new, new, ki, vi, tb, ln)
        xattn.cache_compact(ki, vi, tb, ln, path, acc)
    torch.cuda.synchronize()
