"""Latent attention's and the page tables' kernels in the debug build (on-device bounds checks that record
XATTN_ERR_DEVICE_BOUNDS), in a child process that loads it in place of the release library: every check passes on edge shapes,
and the results stay within their bounds."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import random, sys
sys.path.insert(0, "tests")
sys.path.insert(0, ".")
import torch
from bwd_xattn_fwd_gb300 import xattn
from latent_ref import (latent_decode_reference, latent_inputs, latent_reference, latent_state, release_reference,
                        reserve_reference)
from paged_ref import check_tree
from window_ref import check

assert xattn.xattn_build_flags() & xattn.BUILD_DEVICE_CHECKS
i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")
def clear(what):
    torch.cuda.synchronize()
    assert xattn.xattn_check_device_status() == 0, what
# Every kernel of the expanded form: dn, dv <= 64 full and not, beyond 64 full and not, a negative scale; many units a CTA
for shape, scale in [((2, 257, 3, 64, 32, 64), 0.1), ((1, 385, 2, 32, 16, 48), 0.1), ((2, 300, 2, 128, 64, 128), 0.07),
                     ((1, 255, 5, 80, 48, 112), 0.08), ((1, 200, 2, 16, 64, 128), -0.1), ((1, 130, 2, 64, 32, 64), -0.1),
                     ((40, 200, 8, 64, 32, 64), 0.1), ((30, 300, 8, 128, 64, 128), 0.07), ((1, 1, 1, 16, 16, 16), 0.2)]:
    x = latent_inputs(*shape, seed=5)
    o, lse = xattn.attention_latent_fwd(x["q"], x["kv"], x["k_rope"], scale)
    dq, dkv, drope = xattn.attention_latent_bwd(x["q"], x["kv"], x["k_rope"], o, x["dO"], lse, scale)
    clear(shape)
    check({"o": o, "lse": lse, "dq": dq, "dkv": dkv, "dk_rope": drope}, latent_reference(x, scale), str(shape))
# The absorbed form: 16, 32 and 64 rows a tile, pages below and above a tile, cut sequences, more row tiles than half the SMs
for B, n, nh, dc, dr, page, lens in [(3, 1, 16, 512, 64, 16, [0, 333, 1200]), (2, 2, 16, 512, 64, 64, [700, 90]),
                                     (2, 4, 32, 512, 64, 256, [2000, 17]), (1, 1, 8, 384, 48, 32, [9000]),
                                     (70, 1, 16, 128, 16, 16, [13 * i for i in range(70)]), (2, 64, 80, 128, 16, 64, [40, 100])]:
    pages, table = latent_state(B, n, dc + dr, page, lens, seed=3, device="cuda")
    if B == 3:
        table[1][2], table[2][0] = -1, pages.shape[0]
    q = (torch.randn(B, n, nh, dc + dr, generator=torch.Generator().manual_seed(1)) * 0.5).to(torch.bfloat16).cuda()
    o, lse = xattn.attention_latent_decode(q, pages, i32(table), i32(lens), dc, 0.07)
    clear((B, n, nh))
    check_tree(o, lse, latent_decode_reference(q, pages, table, lens, dc, 0.07), str((B, n, nh)))
# Tables: one block and several kernels of each, too few pages and slots, lengths and entries out of range
for B, width, page, top, most, spare, over in [(1, 3, 16, 20, 30, 2, 3), (64, 66, 64, 4096, 1, 64, 3), (33, 9, 16, 100, 90, 400, -50),
                                               (1000, 10, 16, 80, 5, 700, 11), (5000, 4, 16, 30, 3, 1500, 9), (5, 70, 128, 3000, 5000, 200, 1)]:
    rng = random.Random(B)
    ctx = [rng.choice([0, top, rng.randint(0, top), -3, 10**9]) for _ in range(B)]
    new = [rng.choice([0, most, rng.randint(0, most)]) for _ in range(B)]
    ids = list(range(B * width + spare))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(width)] for _ in range(B)]
    table[0][0], table[B // 2][width - 1] = -1, 2**31 - 1
    free = ids + [-1] * (B * width)
    tokens = max(sum(new) + over, 0)
    t, f, c = i32(table), i32(free), i32([spare])
    slots, offsets, granted = xattn.cache_reserve(t, i32(ctx), i32(new), f, c, page, tokens)
    rt, rc, rs, ro, rg = reserve_reference(table, ctx, new, free, spare, page, tokens, len(free))
    assert slots.tolist() == rs and granted.tolist() == rg and t.tolist() == rt and c.tolist() == [rc]
    keep = [rng.choice([0, 5, -1, 10**9]) for _ in range(B)]
    held = [rng.choice([x, 10**9]) for x in ctx]
    xattn.cache_release(t, i32(held), i32(keep), f, c, page)
    bt, bf, bc = release_reference(rt, held, keep, free, rc, page, len(free))
    assert t.tolist() == bt and f.tolist() == bf and c.tolist() == [bc]
    rows = min(tokens, 5000)
    pool, new_c, new_r = torch.zeros(len(free), page, 24, device="cuda").bfloat16(), torch.ones(rows, 16, device="cuda").bfloat16(), torch.ones(rows, 8, device="cuda").bfloat16()
    xattn.latent_write(new_c, new_r, pool, slots[:rows])
    kp, vp = (torch.zeros(len(free), page, 1, 16, device="cuda").bfloat16() for _ in range(2))
    xattn.cache_write(new_c[:, None], new_c[:, None], kp, vp, slots[:rows])
    clear((B, width))
    there = [s for s in rs[:rows] if s >= 0]
    assert int((pool.view(-1, 24) == 1).all(1).sum()) == len(there) and int((kp != 0).sum()) == 16 * len(there)
print("debug build ok")
"""


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")


def test_debug_build_checks_pass():
    from bwd_xattn_fwd_gb300 import build
    env = dict(os.environ, XATTN_LIBRARY=build.build(debug=True))
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "debug build ok" in r.stdout
