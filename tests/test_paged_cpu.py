"""The paged cache's calls without a GPU: argument checks of the C entry points and of the
binding, and the plain forms that the GPU tests compare with."""
import ctypes

import pytest
import torch

from paged_ref import append_reference, compact_reference, paged_state, random_words, tree_reference

P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    from bwd_xattn_fwd_gb300 import build
    return ctypes.CDLL(build.build())


def _tree(lib, q=16, k=32, table=64, lens=68, tree=72, B=1, n=4, nh=4, nkv=2, hd=64, num_pages=3, page=16, width=2,
          window=4, sinks=0, scale=0.1, o=80, lse=96):
    f = lib.xattn_tree_decode
    f.restype, f.argtypes = I, [P] * 6 + [I] * 10 + [F] + [P] * 3
    return f(q, k, 48, table, lens, tree, B, n, nh, nkv, hd, num_pages, page, width, window, sinks, scale, o, lse, None)


def test_tree_checks(lib):
    assert _tree(lib, q=None) == 1
    assert _tree(lib, lens=None) == 1
    assert _tree(lib, B=0) == 2
    assert _tree(lib, n=0) == 2
    assert _tree(lib, n=65, width=9, window=65) == 2
    assert _tree(lib, num_pages=0) == 2
    assert _tree(lib, nh=3) == 3
    assert _tree(lib, hd=48) == 4
    assert _tree(lib, q=18) == 5
    assert _tree(lib, table=66) == 5
    assert _tree(lib, tree=76) == 5
    assert _tree(lib, lse=98) == 5
    assert _tree(lib, scale=float("inf")) == 9
    assert _tree(lib, window=3) == 13
    assert _tree(lib, sinks=-1) == 13
    for page in (-16, 0, 1, 8, 24, 48, 96, 100, 130, 200):
        assert _tree(lib, page=page) == 14, page
    assert _tree(lib, width=1, n=17, window=17) == 14             # the table cannot hold the new tokens
    assert _tree(lib, page=128, width=(1 << 23) + 1) == 14
    assert _tree(lib, page=128, width=1 << 23, B=128) == 2        # 128 sequences x 2 kv heads x 2^23 tiles
    if not torch.cuda.is_available():
        for page in (16, 32, 64, 128, 256, 384):
            assert _tree(lib, page=page, tree=None) == 6          # accepted; fails only for want of a GPU


def _append(lib, k_new=16, table=64, B=1, n=4, nkv=2, hd=64, num_pages=3, page=16, width=2):
    f = lib.xattn_cache_append
    f.restype, f.argtypes = I, [P] * 6 + [I] * 7 + [P]
    return f(k_new, 32, 48, 64, table, 68, B, n, nkv, hd, num_pages, page, width, None)


def _compact(lib, k=16, path=64, B=1, n=4, nkv=2, hd=64, num_pages=3, page=16, width=2):
    f = lib.xattn_cache_compact
    f.restype, f.argtypes = I, [P] * 6 + [I] * 7 + [P]
    return f(k, 32, 60, 64, path, 68, B, n, nkv, hd, num_pages, page, width, None)


@pytest.mark.parametrize("call,first,array", [(_append, "k_new", "table"), (_compact, "k", "path")])
def test_page_checks(lib, call, first, array):
    assert call(lib, **{first: None}) == 1
    assert call(lib, **{array: None}) == 1
    assert call(lib, n=0) == 2
    assert call(lib, nkv=-1) == 2
    assert call(lib, hd=12) == 4
    assert call(lib, **{first: 24}) == 5
    assert call(lib, **{array: 66}) == 5
    assert call(lib, page=17) == 14
    assert call(lib, n=33) == 14
    if not torch.cuda.is_available():
        assert call(lib, hd=8) == 6


def test_binding_checks():
    from bwd_xattn_fwd_gb300 import xattn
    k = torch.zeros(2, 16, 1, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 2, 2, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        xattn.attention_tree_decode(q, k, k, table, lens)             # not on a GPU
    with pytest.raises(ValueError):
        xattn.attention_tree_decode(q[0], k, k, table, lens)
    with pytest.raises(ValueError):
        xattn.cache_append(k, k, k, k, table[0], lens)
    with pytest.raises(ValueError):
        xattn.cache_compact(k, k, table, lens, lens, lens)


def test_a_compaction_beyond_the_largest_grid(lib):
    assert _compact(lib, B=2**30, n=1, nkv=1, hd=8) == 2             # two blocks a sequence


def test_a_stream_of_another_device():
    from types import SimpleNamespace
    from bwd_xattn_fwd_gb300 import xattn
    t, s = SimpleNamespace(device=torch.device("cuda:0")), SimpleNamespace(device=torch.device("cuda:1"))
    with pytest.raises(ValueError):
        xattn._Elsewhere(t, s)


def test_the_plain_tree_of_a_run_is_causal_attention():
    """A run of new tokens (no words, or the words 2^(i+1) - 1) over a cache is the last rows of
    causal attention: against a softmax written out over the whole sequence."""
    B, n, nkv, hd, page, lens = 2, 4, 2, 8, 16, [20, 33]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=1, dtype=torch.float64)
    q = torch.randn(B, n, 4, hd, dtype=torch.float64, generator=torch.Generator().manual_seed(0))
    (o, _), (lse, _) = tree_reference(q, k, v, table, lens, None, 10**6, 0, 0.3)
    words = [[(2 << i) - 1 for i in range(n)]] * B
    (o2, _), _ = tree_reference(q, k, v, table, lens, words, 10**6, 0, 0.3)
    assert torch.equal(o, o2)
    for b in range(B):
        T = lens[b] + n
        rows = torch.tensor([table[b][p // page] * page + p % page for p in range(T)])
        kb, vb = (x.view(-1, nkv, hd)[rows].repeat_interleave(2, 1) for x in (k, v))
        s = torch.einsum("ihd,phd->hip", q[b], kb) * 0.3
        hidden = torch.arange(T)[None, :] > torch.arange(n)[:, None] + lens[b]
        w = torch.softmax(s.masked_fill(hidden, float("-inf")), 2)
        assert float((torch.einsum("hip,phd->ihd", w, vb) - o[b]).abs().max()) <= 1e-12


def test_the_plain_window_equals_hiding_positions():
    """A window with sinks equals the unwindowed form with the hidden positions' pages missing
    (window and sinks at page boundaries, one token)."""
    B, n, nkv, hd, page, lens = 1, 1, 1, 8, 16, [63]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=2, dtype=torch.float64)
    q = torch.randn(B, n, 2, hd, dtype=torch.float64, generator=torch.Generator().manual_seed(0))
    (a, _), _ = tree_reference(q, k, v, table, lens, None, 32, 16, 0.3)
    gone = [[table[0][0], -1, table[0][2], table[0][3]]]
    (b, _), _ = tree_reference(q, k, v, gone, lens, None, 10**6, 0, 0.3)
    assert float((a - b).abs().max()) <= 1e-14


def test_plain_append_then_compact():
    B, n, nkv, hd, page, lens = 1, 4, 1, 8, 16, [14]
    k, v, table = paged_state(B, n, nkv, hd, page, lens, seed=3, dtype=torch.float64)
    new = torch.arange(4 * 8, dtype=torch.float64).view(1, 4, 1, 8)
    k, v = append_reference(new, -new, k, v, table, lens)
    k, v = compact_reference(k, v, table, lens, [[0, 2, 3, 0]], [3])
    at = [table[0][p // page] * page + p % page for p in range(14, 18)]
    assert torch.equal(k.view(-1, 1, 8)[at][:, 0], new[0, [0, 2, 3, 3], 0])
    assert torch.equal(v.view(-1, 1, 8)[at][:, 0], -new[0, [0, 2, 3, 3], 0])


def test_random_words_are_trees():
    for row in random_words(3, 64, 1):
        for i, w in enumerate(row):
            assert w >> i == 1                                       # itself, and no later token


def test_a_scale_too_large_for_base_2(lib):
    assert _tree(lib, scale=-2.5e38) == 9
