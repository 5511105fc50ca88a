"""The serving step that README.md gives, run as it stands there, turn after turn: sequences advance by what they accept, one
that finds no page is denied without harm to the others and goes on when pages come free."""
import os
import re

import pytest
import torch

from latent_ref import latent_decode_reference, rows_of
from paged_ref import check_tree

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _step():
    with open(os.path.join(ROOT, "README.md"), encoding="utf-8") as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(compile(b, "README.md", "exec") for b in blocks if "cache_reserve" in b)


@pytest.mark.parametrize("stale", [float("nan"), 1000.0])
def test_the_serving_step(stale):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from bwd_xattn_fwd_gb300 import xattn
    step = _step()
    B, n, nh, dc, dr, page, num_pages, width = 3, 2, 8, 128, 16, 16, 6, 8
    g = torch.Generator("cuda").manual_seed(0)
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * 0.5).bfloat16()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    keep = [2, 1, 2]
    ns = {"xattn": xattn, "torch": torch, "n": n, "dc": dc, "scale": 0.1, "page_size": page, "tokens": B * n,
          "page_table": i32([[-1] * width] * B), "ctx_lens": i32([0] * B), "new_lens": i32([n] * B),
          "free_pages": torch.randperm(num_pages, generator=torch.Generator().manual_seed(1)).int().cuda(),
          "free_count": i32([num_pages]), "pages": torch.full((num_pages, page, dc + dr), stale, device="cuda").bfloat16(),
          "accept": lambda o: i32(keep)}
    history, denied, ctx = [[] for _ in range(B)], [], [0] * B
    for turn in range(60):
        ns.update(c=rnd(B * n, dc), k_rope=rnd(B * n, dr), q=rnd(B, n, nh, dc + dr))
        exec(step, ns)
        granted = ns["granted"].tolist()
        denied.append([b for b in range(B) if granted[b] < n])
        served = [b for b in range(B) if granted[b] == n]
        # The table after the step has lost pages that only rejected tokens held; what the call saw is what is there with them.
        table, flat = ns["page_table"].tolist(), ns["pages"].view(-1, dc + dr)
        rows = torch.cat([ns["c"], ns["k_rope"]], 1)
        for b in served:
            pool = torch.cat([torch.stack(history[b]), rows[b * n:b * n + n]] if history[b] else [rows[b * n:b * n + n]])
            at = [list(range((len(pool) + page - 1) // page))]
            own = torch.zeros(len(at[0]) * page, dc + dr, dtype=torch.bfloat16, device="cuda")
            own[:len(pool)] = pool
            check_tree(ns["o"][b:b + 1], ns["lse"][b:b + 1],
                       latent_decode_reference(ns["q"][b:b + 1], own.view(-1, page, dc + dr), at, [ctx[b]], dc, 0.1), f"turn {turn}")
            history[b] += list(rows[b * n:b * n + keep[b]])
            ctx[b] += keep[b]
        assert ns["ctx_lens"].tolist() == ctx
        for b in range(B):
            if history[b]:
                assert torch.equal(flat[rows_of(table, b, range(ctx[b]), page, num_pages)], torch.stack(history[b]))
        held = sum((c + page - 1) // page for c in ctx)
        assert ns["free_count"].item() == num_pages - held
        assert sorted([e for r in table for e in r if e >= 0] + ns["free_pages"].tolist()[:num_pages - held]) == list(range(num_pages))
        if turn == 40:                                      # the longest request ends
            last = ctx.index(max(ctx))
            kept = i32([0 if b == last else c for b, c in enumerate(ctx)])
            xattn.cache_release(ns["page_table"], ns["ctx_lens"], kept, ns["free_pages"], ns["free_count"], page)
            ns["ctx_lens"].copy_(kept)
            history[last], ctx[last] = [], 0
    assert any(denied[:41]) and any(not d for d in denied[41:]) and xattn.xattn_check_device_status() == 0
