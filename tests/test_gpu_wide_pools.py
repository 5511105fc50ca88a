"""Pools of more than 2^31 numbers: slots, pages and rows beyond what 32 bits address, for the absorbed form, both writes, and the
tables whose slots name them."""
import pytest
import torch

from latent_ref import latent_decode_reference
from paged_ref import check_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _give_back():
    yield
    from bwd_xattn_fwd_gb300 import xattn
    torch.cuda.empty_cache()
    xattn.xattn_trim_scratch(0)


def _need(gigabytes):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    if torch.cuda.mem_get_info()[0] < gigabytes << 30:
        pytest.skip(f"{gigabytes} GB of free device memory needed")


def test_latent_rows_behind_2_to_the_32_numbers():
    """A serving step in the last pages of a pool of 2^32 numbers and more (8.6 GB): reserved, written, attended to, and no row
    written that the same offset modulo 2^31 or 2^32 would name."""
    from bwd_xattn_fwd_gb300 import xattn
    _need(24)
    dc, dr, page, B, S, nh = 512, 64, 64, 2, 130, 16
    width = dc + dr
    num_pages = 2 ** 32 // (page * width) + 40
    pages = torch.zeros(num_pages, page, width, dtype=torch.bfloat16, device="cuda")
    assert pages.numel() > 2 ** 32
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ids = list(range(num_pages - 6, num_pages))                      # the last six, topmost first taken
    table, free = i32([[-1] * 3] * B), torch.zeros(num_pages, dtype=torch.int32, device="cuda")
    free[:6], count = i32(ids), i32([6])
    slots, _, granted = xattn.cache_reserve(table, i32([0] * B), i32([S] * B), free, count, page, B * S)
    assert granted.tolist() == [S] * B and count.item() == 0
    at = [[ids[5 - 3 * b - p // page] * page + p % page for p in range(S)] for b in range(B)]
    assert slots.tolist() == at[0] + at[1] and min(at[1]) * width > 2 ** 32
    g = torch.Generator("cuda").manual_seed(0)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.5).bfloat16()
    c, rope, q = rnd(B * S, dc), rnd(B * S, dr), rnd(B, 1, nh, width)
    xattn.latent_write(c, rope, pages, slots)
    rows = torch.cat([c, rope], 1)
    assert torch.equal(pages.view(-1, width)[slots], rows)
    assert int((pages.view(-1, width)[:, 0] != 0).sum()) == int((rows[:, 0] != 0).sum())        # nothing elsewhere
    o, lse = xattn.attention_latent_decode(q, pages, table, i32([S - 1] * B), dc, 0.07)
    small = torch.zeros(6, page, width, dtype=torch.bfloat16, device="cuda")                      # the same rows in a small pool
    near = [[x - ids[0] * page for x in row] for row in at]
    small.view(-1, width)[torch.tensor(near[0] + near[1], device="cuda")] = rows
    small_table = (table - ids[0]).tolist()
    check_tree(o, lse, latent_decode_reference(q, small, small_table, [S - 1] * B, dc, 0.07), "last pages")
    xattn.cache_release(table, granted, i32([0] * B), free, count, page)
    assert count.item() == 6 and free[:6].tolist() == ids
    assert xattn.xattn_check_device_status() == 0


@pytest.mark.parametrize("rows", [5, 9000])
def test_kv_rows_behind_2_to_the_31_numbers(rows):
    from bwd_xattn_fwd_gb300 import xattn
    _need(24)
    nkv, hd, page = 4, 128, 64
    num_pages = 2 ** 31 // (page * nkv * hd) + 300
    kp, vp = (torch.zeros(num_pages, page, nkv, hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 31
    g = torch.Generator("cuda").manual_seed(rows)
    k, v = (torch.randn(rows, nkv, hd, generator=g, device="cuda").bfloat16() for _ in range(2))
    slots = num_pages * page - 1 - torch.randperm(300 * page, generator=torch.Generator().manual_seed(rows))[:rows].cuda()
    xattn.cache_write(k, v, kp, vp, slots)
    for pool, new in ((kp, k), (vp, v)):
        flat = pool.view(-1, nkv, hd)
        assert torch.equal(flat[slots], new)
        assert int((flat[:, 0, 0] != 0).sum()) == int((new[:, 0, 0] != 0).sum())
    assert xattn.xattn_check_device_status() == 0


def test_expanded_tensors_of_more_than_2_to_the_31_numbers():
    """1024 heads: the last heads of the last sequence, behind 2^31 numbers of every tensor and of the backward's scratch, have the
    bits that they have in a call of their own."""
    from bwd_xattn_fwd_gb300 import xattn
    _need(90)
    B, S, nh, dn, dr, dv = 9, 2050, 1024, 64, 64, 64
    g = torch.Generator("cuda").manual_seed(0)

    def fill(*shape, times=0.5):
        t = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
        for b in range(shape[0]):
            t[b] = (torch.randn(shape[1:], generator=g, device="cuda") * times).bfloat16()
        return t

    q, kv, rope, dO = fill(B, S, nh, dn + dr), fill(B, S, nh, dn + dv), fill(B, S, dr), fill(B, S, nh, dv, times=1.0)
    assert q[:-1].numel() > 2 ** 31 and B * S * nh * dr > 2 ** 30
    o, lse = xattn.attention_latent_fwd(q, kv, rope)
    dq, dkv, _ = xattn.attention_latent_bwd(q, kv, rope, o, dO, lse)
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0
    cut = lambda t: t[-1:, :, -3:].contiguous()
    o1, lse1 = xattn.attention_latent_fwd(cut(q), cut(kv), rope[-1:].contiguous())
    dq1, dkv1, _ = xattn.attention_latent_bwd(cut(q), cut(kv), rope[-1:].contiguous(), o1, cut(dO), lse1)
    for a, b in ((o, o1), (lse, lse1), (dq, dq1), (dkv, dkv1)):
        assert torch.equal(cut(a), b)


def test_absorbed_queries_of_more_than_2_to_the_31_numbers():
    """64 tokens of 65536 heads, 65536 row tiles: the last heads of the last token against the definition."""
    from bwd_xattn_fwd_gb300 import xattn
    _need(40)
    n, nh, dc, dr, page, ctx = 64, 65536, 512, 64, 16, 30
    q = torch.empty(1, n, nh, dc + dr, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(0)
    for i in range(n):
        q[0, i] = (torch.randn(nh, dc + dr, generator=g, device="cuda") * 0.5).bfloat16()
    pages = (torch.randn(6, page, dc + dr, generator=g, device="cuda") * 0.5).bfloat16()
    table = [[3, 1, 5, 0, 2, 4]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    o, lse = xattn.attention_latent_decode(q, pages, i32(table), i32([ctx]), dc, 0.07)
    torch.cuda.synchronize()
    assert o[0, :-1].numel() > 2 ** 31 - 2 ** 26 and q.numel() > 2 ** 31 and xattn.xattn_check_device_status() == 0
    for heads in (slice(0, 2), slice(nh - 3, nh)):
        check_tree(o[:, :, heads], lse[:, :, heads],
                   latent_decode_reference(q[:, :, heads].contiguous(), pages, table, [ctx], dc, 0.07), str(heads))
