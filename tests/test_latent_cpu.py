"""Latent attention's and the page tables' calls without a GPU: argument checks of the C entry points and of
the binding, and the plain forms that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

from latent_ref import (latent_decode_reference, latent_inputs, latent_reference, latent_state, release_reference,
                        reserve_reference)

P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
NO_GPU = 6


@pytest.fixture(scope="module")
def lib():
    from bwd_xattn_fwd_gb300 import build
    return ctypes.CDLL(build.build())


def _fwd(lib, q=16, kv=32, rope=48, B=1, S=5, nh=3, dn=64, dr=32, dv=64, scale=0.1, o=64, lse=80):
    f = lib.xattn_latent_fwd
    f.restype, f.argtypes = I, [P] * 3 + [I] * 6 + [F] + [P] * 3
    return f(q, kv, rope, B, S, nh, dn, dr, dv, scale, o, lse, None)


def _bwd(lib, q=16, kv=32, rope=48, o=64, dO=80, lse=96, B=1, S=5, nh=3, dn=64, dr=32, dv=64, scale=0.1, dq=128,
         dkv=160, drope=144):
    f = lib.xattn_latent_bwd
    f.restype, f.argtypes = I, [P] * 6 + [I] * 6 + [F] + [P] * 4
    return f(q, kv, rope, o, dO, lse, B, S, nh, dn, dr, dv, scale, dq, dkv, drope, None)


@pytest.mark.parametrize("call,more", [(_fwd, ("o",)), (_bwd, ("o", "dO", "dq", "dkv", "drope"))])
def test_expanded_checks(lib, call, more):
    for name in ("q", "kv", "rope", "lse", *more):
        assert call(lib, **{name: None}) == 1, name
    for name in ("q", "kv", "rope", *more):
        assert call(lib, **{name: 24}) == 5, name
    for name in ("o",) if call is _fwd else ("dq", "dkv"):
        assert call(lib, **{name: 48}) == 5, name                         # written by whole 32-byte sectors
    assert call(lib, lse=98) == 5
    for name in ("B", "S", "nh", "dn", "dr", "dv"):
        assert call(lib, **{name: 0}) == 2, name
        assert call(lib, **{name: -16}) == 2, name
    assert call(lib, B=2**20, S=2**20, nh=2**10) == 2
    assert call(lib, S=2**30 + 1) == 2
    for bad in (dict(dn=8), dict(dn=144), dict(dn=100), dict(dr=8), dict(dr=80), dict(dr=24), dict(dv=136), dict(dv=120)):
        assert call(lib, **bad) == 4, bad
    assert call(lib, scale=math.nan) == 9
    assert call(lib, scale=2.5e38) == 9
    if not torch.cuda.is_available():
        for good in (dict(), dict(scale=0.0), dict(scale=-1e-30), dict(dn=128, dr=64, dv=128), dict(dn=16, dr=16, dv=48)):
            assert call(lib, **good) == NO_GPU, good


def _decode(lib, q=16, pages=32, table=64, lens=68, B=1, n=1, nh=16, dc=512, dr=64, num_pages=3, page=16, width=2,
            scale=0.1, o=80, lse=96):
    f = lib.xattn_latent_decode
    f.restype, f.argtypes = I, [P] * 4 + [I] * 8 + [F] + [P] * 3
    return f(q, pages, table, lens, B, n, nh, dc, dr, num_pages, page, width, scale, o, lse, None)


def test_decode_checks(lib):
    for name in ("q", "pages", "table", "lens", "o", "lse"):
        assert _decode(lib, **{name: None}) == 1, name
    for name in ("q", "pages", "o"):
        assert _decode(lib, **{name: 24}) == 5, name
    for name in ("table", "lens", "lse"):
        assert _decode(lib, **{name: 66}) == 5, name
    for name in ("B", "n", "nh", "dc", "dr", "num_pages", "width"):
        assert _decode(lib, **{name: 0}) == 2, name
    assert _decode(lib, n=65, width=9) == 2
    assert _decode(lib, B=2**16, n=2, nh=2**13) == 2
    for bad in (dict(dc=64), dict(dc=576), dict(dc=640), dict(dc=200), dict(dr=8), dict(dr=80)):
        assert _decode(lib, **bad) == 4, bad
    assert _decode(lib, scale=math.inf) == 9
    assert _decode(lib, scale=-2.5e38) == 9
    for page in (-16, 0, 1, 8, 24, 48, 96, 100, 200):
        assert _decode(lib, page=page) == 14, page
    assert _decode(lib, n=33) == 14                                   # the table cannot hold the new tokens
    if not torch.cuda.is_available():
        for good in (dict(), dict(dc=128, dr=16), dict(n=32), dict(page=256), dict(nh=1), dict(nh=200)):
            assert _decode(lib, **good) == NO_GPU, good


def _reserve(lib, table=16, ctx=20, new=24, free=28, count=32, B=2, num_pages=9, page=16, width=4, tokens=7, slots=40,
             offsets=48, granted=52):
    f = lib.xattn_cache_reserve
    f.restype, f.argtypes = I, [P] * 5 + [I] * 5 + [P] * 4
    return f(table, ctx, new, free, count, B, num_pages, page, width, tokens, slots, offsets, granted, None)


def _release(lib, table=16, held=20, keep=24, free=28, count=32, B=2, num_pages=9, page=16, width=4):
    f = lib.xattn_cache_release
    f.restype, f.argtypes = I, [P] * 5 + [I] * 4 + [P]
    return f(table, held, keep, free, count, B, num_pages, page, width, None)


def test_table_checks(lib):
    for call, arrays in ((_reserve, ("table", "ctx", "new", "free", "count", "offsets", "granted")),
                         (_release, ("table", "held", "keep", "free", "count"))):
        for name in arrays:
            assert call(lib, **{name: None}) == 1, name
            assert call(lib, **{name: 18}) == 5, name
        for name in ("B", "num_pages", "width"):
            assert call(lib, **{name: 0}) == 2, name
        assert call(lib, page=17) == 14
        assert call(lib, page=128, width=2**23 + 1) == 14
        if not torch.cuda.is_available():
            assert call(lib) == NO_GPU
    assert _reserve(lib, slots=None) == 1
    assert _reserve(lib, slots=44) == 5
    assert _reserve(lib, tokens=-1) == 2
    if not torch.cuda.is_available():
        assert _reserve(lib, tokens=0, slots=None) == NO_GPU


def _write(lib, k=16, v=32, kp=48, vp=64, slots=80, rows=3, nkv=2, hd=64, num_pages=3, page=16):
    f = lib.xattn_cache_write
    f.restype, f.argtypes = I, [P] * 5 + [I] * 5 + [P]
    return f(k, v, kp, vp, slots, rows, nkv, hd, num_pages, page, None)


def _latent_write(lib, k=16, v=32, kp=48, slots=80, rows=3, dc=64, dr=16, num_pages=3, page=16):
    f = lib.xattn_latent_write
    f.restype, f.argtypes = I, [P] * 4 + [I] * 5 + [P]
    return f(k, v, kp, slots, rows, dc, dr, num_pages, page, None)


@pytest.mark.parametrize("call,sizes", [(_write, ("nkv", "hd")), (_latent_write, ("dc", "dr"))])
def test_write_checks(lib, call, sizes):
    for name in ("k", "v", "kp", "slots"):
        assert call(lib, **{name: None}) == 1, name
        assert call(lib, **{name: 20}) == 5, name
    for name in (*sizes, "num_pages", "page"):
        assert call(lib, **{name: 0}) == 2, name
    assert call(lib, rows=-1) == 2
    assert call(lib, **{sizes[1]: 12}) == 4
    assert call(lib, rows=2**31 - 1, **{sizes[0]: 2**20}) == 2
    assert call(lib, rows=0, k=None, v=None, slots=None) == 0            # nothing to write: no device needed
    if not torch.cuda.is_available():
        assert call(lib, page=5) == NO_GPU


def test_binding_checks():
    from bwd_xattn_fwd_gb300 import xattn
    bf = dict(dtype=torch.bfloat16)
    q, kv, rope = torch.zeros(1, 4, 2, 48, **bf), torch.zeros(1, 4, 2, 64, **bf), torch.zeros(1, 4, 16, **bf)
    with pytest.raises(ValueError):
        xattn.attention_latent_fwd(q, kv, rope)                          # not on a GPU
    with pytest.raises(ValueError):
        xattn.attention_latent_fwd(q, kv, rope[0])
    with pytest.raises(ValueError):
        xattn.attention_latent_fwd(rope[:, :, None], kv, rope)           # no dn left
    with pytest.raises(TypeError):
        xattn.attention_latent_fwd(q.float(), kv, rope)
    with pytest.raises(ValueError):
        xattn.attention_latent_bwd(q, kv, rope, q, q, q)
    pages, table, lens = torch.zeros(2, 16, 144, **bf), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        xattn.attention_latent_decode(torch.zeros(1, 1, 2, 144, **bf), pages, table, lens, 128, 0.1)
    with pytest.raises(ValueError):
        xattn.attention_latent_decode(torch.zeros(1, 1, 2, 144, **bf), pages, table, lens, 144, 0.1)
    with pytest.raises(ValueError):
        xattn.cache_reserve(table, lens, lens, lens, lens, 16, 4)
    with pytest.raises(TypeError):
        xattn.cache_release(table.long(), lens, lens, lens, lens, 16)
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        xattn.latent_write(torch.zeros(3, 128, **bf), torch.zeros(3, 16, **bf), pages, slots)
    with pytest.raises(ValueError):
        xattn.cache_write(q, q, q, q, slots)


def test_the_plain_form_against_autograd():
    """Gradients of the reference: those of the definition, k_rope's summed over the heads."""
    x = {n: t.double() for n, t in latent_inputs(2, 9, 3, 16, 16, 32, seed=1, device="cpu").items()}
    leaf = {n: x[n].clone().requires_grad_() for n in ("q", "kv", "k_rope")}
    k = torch.cat([leaf["kv"][..., :16], leaf["k_rope"][:, :, None].expand(-1, -1, 3, -1)], 3)
    s = torch.einsum("bihd,bjhd->bhij", leaf["q"], k) * 0.3
    s = s.masked_fill(torch.ones(9, 9, dtype=torch.bool).triu(1), -math.inf)
    o = torch.einsum("bhij,bjhd->bihd", torch.softmax(s, 3), leaf["kv"][..., 16:])
    (o * x["dO"]).sum().backward()
    ref = latent_reference(x, 0.3)
    assert float((ref["o"][0] - o.detach()).abs().max()) <= 1e-12
    for n in leaf:
        assert float((ref["d" + n][0] - leaf[n].grad).abs().max()) <= 1e-12, n


def test_the_absorbed_form_is_the_expanded_one():
    """A decode step with absorbed queries gives, through the value projection, the last row of the expanded
    attention over the same latents."""
    g = torch.Generator().manual_seed(0)
    T, nh, dc, dn, dr, dv = 21, 3, 128, 16, 16, 32
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    w_k, w_v = rnd(nh, dc, dn) * dc ** -0.5, rnd(nh, dc, dv) * dc ** -0.5
    pages, table = latent_state(1, 1, dc + dr, 16, [T - 1], seed=2, dtype=torch.float64)
    rows = torch.tensor([table[0][p // 16] * 16 + p % 16 for p in range(T)])
    lat = pages.view(-1, dc + dr)[rows]
    q = rnd(1, T, nh, dn + dr)
    kv = torch.cat([torch.einsum("jc,hcd->jhd", lat[:, :dc], w) for w in (w_k, w_v)], 2)[None]
    x = {"q": q, "kv": kv, "k_rope": lat[None, :, dc:], "dO": torch.zeros(1, T, nh, dv)}
    ref = latent_reference(x, 0.2)
    absorbed = torch.cat([torch.einsum("hd,hcd->hc", q[0, -1, :, :dn], w_k), q[0, -1, :, dn:]], 1)[None, None]
    (o, _), (lse, _) = latent_decode_reference(absorbed, pages, table, [T - 1], dc, 0.2)
    out = torch.einsum("hc,hcd->hd", o[0, 0], w_v)
    assert float((out - ref["o"][0][0, -1]).abs().max()) <= 1e-12
    assert float((lse[0, 0] - ref["lse"][0][0, -1]).abs().max()) <= 1e-12


def test_plain_reserve_and_release():
    table = [[7, -1, -1], [3, 4, -1], [-1, -1, -1]]
    free = [0, 1, 2, 5, 6, -1, -1, -1]
    # One more page for sequence 0 (5 + 20 > 16), none for 1 (20 + 3), two for 2.
    t, count, slots, offsets, granted = reserve_reference(table, [5, 20, 0], [20, 3, 17], free, 5, 16, 42, 8)
    assert t == [[7, 6, -1], [3, 4, -1], [5, 2, -1]] and count == 2
    assert offsets == [0, 20, 23, 40] and granted == [20, 3, 17]
    assert slots[:20] == [*range(7 * 16 + 5, 8 * 16), *range(96, 105)]
    assert slots[20:23] == [68, 69, 70] and slots[23:40] == [*range(80, 96), 32] and slots[40:] == [-1, -1]
    back = release_reference(t, [25, 23, 17], [5, 20, 0], free, count, 16, 8)
    assert back == (table, free, 5)
    # Two free pages do not reach sequence 2; sequence 1 needs none.
    t, count, slots, _, granted = reserve_reference(table, [5, 20, 0], [20, 3, 17], free, 2, 16, 42, 8)
    assert count == 1 and granted == [20, 3, 0] and t[2] == [-1, -1, -1] and slots[23:] == [-1] * 19
    # The slot map ends inside sequence 1's tokens.
    assert reserve_reference(table, [5, 20, 0], [20, 3, 17], free, 5, 16, 22, 8)[4] == [20, 0, 0]


def test_more_sequences_than_the_tables_count(lib):
    """Beyond 2^30 sequences sums of their number and a block's width would wrap: the plan would serve nobody, the search in
    the offsets start before them."""
    for B in (2**30 + 1, 2**31 - 1024, 2**31 - 1):
        assert _reserve(lib, B=B, width=1) == 2 and _release(lib, B=B, width=1) == 2
    if not torch.cuda.is_available():
        assert _reserve(lib, B=2**30, width=1) == NO_GPU and _release(lib, B=2**30, width=1) == NO_GPU
