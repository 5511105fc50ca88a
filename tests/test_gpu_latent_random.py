"""Random calls over the documented ranges, the same ones in every run: latent attention's two forms against 64 bits, page tables
and writes against plain Python."""
import math
import random

import pytest
import torch

from latent_ref import (check_norms, latent_decode_reference, latent_inputs, latent_norms, latent_reference, latent_state,
                        release_reference, reserve_reference)
from paged_ref import check_tree
from window_ref import check

pytestmark = pytest.mark.gpu
CALLS = 12


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn  # noqa: F401  (fails loudly if not built)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _clear(what):
    from bwd_xattn_fwd_gb300 import xattn
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0, what


@pytest.mark.parametrize("seed", range(8))
def test_expanded(seed):
    from bwd_xattn_fwd_gb300 import xattn
    rng = random.Random(seed)
    for call in range(CALLS):
        dn, dr, dv = (16 * rng.randint(1, top) for top in rng.choice([(8, 4, 8), (4, 4, 4)]))
        S, nh = _log_int(rng, 1, 1300), rng.choice([1, 2, 3, 5, 8])
        shape = (max(1, min(_log_int(rng, 1, 40), 2500 // (S * nh) + 1)), S, nh, dn, dr, dv)
        usual = (dn + dr) ** -0.5
        scale = rng.choice([usual, usual, usual, -usual, 2.5 * usual, 0.0])
        x = latent_inputs(*shape, seed=1000 * seed + call)
        o, lse = xattn.attention_latent_fwd(x["q"], x["kv"], x["k_rope"], scale)
        dq, dkv, drope = xattn.attention_latent_bwd(x["q"], x["kv"], x["k_rope"], o, x["dO"], lse, scale)
        what = f"{shape}, scale {scale}"
        _clear(what)
        got = {"o": o, "lse": lse, "dq": dq, "dkv": dkv, "dk_rope": drope}
        check(got, latent_reference(x, scale), what)
        if S >= 129 and abs(scale) == usual:
            check_norms(got, dn, latent_norms(x, scale), what)


@pytest.mark.parametrize("seed", range(8))
def test_absorbed(seed):
    """Rows that no token sees hold NaN; some pages are missing."""
    from bwd_xattn_fwd_gb300 import xattn
    rng = random.Random(100 + seed)
    for call in range(CALLS):
        dc, dr, page = rng.choice([128, 256, 384, 512]), 16 * rng.randint(1, 4), rng.choice([16, 32, 64, 128, 256, 384])
        n, nh = rng.choice([(1, 1), (1, 16), (1, 7), (2, 16), (3, 11), (1, 100), (5, 30), (64, 2), (17, 3)])
        top = _log_int(rng, 1, 6000)
        B = max(1, min(_log_int(rng, 1, 100), 60000 // (top * n) + 1))
        lens = [rng.choice([0, 1, top, rng.randint(0, top)]) for _ in range(B)]
        pages, table = latent_state(B, n, dc + dr, page, lens, seed=seed, device="cuda",
                                    table_width=(max(lens) + n + page - 1) // page + rng.randint(0, 3))
        for b in range(B):
            if rng.random() < 0.2:
                table[b][rng.randrange(len(table[b]))] = rng.choice([-1, -9, pages.shape[0], 2**31 - 1])
        q = (torch.randn(B, n, nh, dc + dr, generator=torch.Generator().manual_seed(call)) * 0.5).bfloat16().cuda()
        scale = rng.choice([0.07, 0.07, -0.07, 0.3, 0.0])
        o, lse = xattn.attention_latent_decode(q, pages, _i32(table), _i32(lens), dc, scale)
        what = f"B {B} n {n} nh {nh} dc {dc} dr {dr} page {page} longest {top} scale {scale}"
        _clear(what)
        check_tree(o, lse, latent_decode_reference(q, pages, table, lens, dc, scale), what)


@pytest.mark.parametrize("seed", range(8))
def test_tables_and_writes(seed):
    from bwd_xattn_fwd_gb300 import xattn
    rng = random.Random(200 + seed)
    for call in range(CALLS):
        B, page, width = _log_int(rng, 1, 3000), rng.choice([16, 32, 64, 128, 256]), _log_int(rng, 1, 40)
        cap = width * page
        ctx = [rng.choice([0, rng.randint(0, cap), rng.randint(0, cap), cap, -5, 10**9]) for _ in range(B)]
        most = rng.choice([1, 3, 20, cap + 10])
        new = [rng.choice([0, most, rng.randint(0, most), -2]) for _ in range(B)]
        num_pages = B * width + rng.randint(1, 50)
        ids = list(range(num_pages))
        rng.shuffle(ids)
        held = [(min(max(c, 0), cap) + page - 1) // page for c in ctx]
        table = [[ids.pop() for _ in range(h)] + [-1] * (width - h) for h in held]
        spare = rng.choice([0, len(ids), rng.randint(0, len(ids))])
        free = ids + [-1] * (num_pages - len(ids))
        tokens = max(0, rng.choice([0, 3, -7]) + sum(max(x, 0) for x in new))
        t, f, c = _i32(table), _i32(free), _i32([spare])
        slots, offsets, granted = xattn.cache_reserve(t, _i32(ctx), _i32(new), f, c, page, tokens)
        what = f"B {B} page {page} width {width} spare {spare} tokens {tokens}"
        rt, rc, rs, ro, rg = reserve_reference(table, ctx, new, free, spare, page, tokens, num_pages)
        assert slots.tolist() == rs and offsets.tolist() == ro and granted.tolist() == rg, what
        assert t.tolist() == rt and c.tolist() == [rc] and f.tolist() == free, what
        if num_pages * page <= 1 << 20:
            dc, dr = 8 * rng.randint(1, 20), 8 * rng.randint(1, 8)
            pages = torch.zeros(num_pages, page, dc + dr, dtype=torch.bfloat16, device="cuda")
            rows = torch.randn(tokens, dc + dr, generator=torch.Generator().manual_seed(call)).bfloat16().cuda()
            want = pages.clone()
            want.view(-1, dc + dr)[slots[slots >= 0]] = rows[slots >= 0]
            xattn.latent_write(rows[:, :dc].contiguous(), rows[:, dc:].contiguous(), pages, slots)
            assert torch.equal(pages, want), what
        back = [x + g for x, g in zip(ctx, rg)]
        keep = [rng.choice([0, x, rng.randint(-3, cap)]) for x in ctx]
        xattn.cache_release(t, _i32(back), _i32(keep), f, c, page)
        bt, bf, bc = release_reference(rt, back, keep, free, rc, page, num_pages)
        assert t.tolist() == bt and f.tolist() == bf and c.tolist() == [bc], what
        _clear(what)
