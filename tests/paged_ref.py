"""A paged cache's operators in plain form: positions looked up one by one, attention in 64
bits with elementwise bounds (u = 2^-8: P and o are rounded to bf16, each off by at most half a
step; t: fp32 scores, exponentials and sums)."""
import math
import random

import torch


def rows_of(table, b, positions, page, num_pages):
    """Pool row of each position, -1 where there is none."""
    out = []
    for p in positions:
        e = table[b][p // page] if 0 <= p < len(table[b]) * page else -1
        out.append(e * page + p % page if 0 <= e < num_pages else -1)
    return out


def tree_reference(q, k_pages, v_pages, table, lens, words, window, sinks, scale):
    """((o, bound), (lse, bound)) in float64; words: [B][n] ints, or None for a run."""
    B, n, nh, hd = q.shape
    num_pages, page, nkv, _ = k_pages.shape
    group, dev, cap = nh // nkv, q.device, len(table[0]) * page
    o = torch.zeros(B, n, nh, hd, dtype=torch.float64, device=dev)
    o_err = torch.full_like(o, 1e-30)
    lse = torch.full((B, n, nh), -math.inf, dtype=torch.float64, device=dev)
    lse_err = torch.zeros_like(lse)
    for b in range(B):
        ctx = min(max(lens[b], 0), cap - n)
        rows = rows_of(table, b, range(ctx + n), page, num_pages)
        sees = torch.zeros(n, ctx + n, dtype=torch.bool)
        for i in range(n):
            w = (words[b][i] if words else (2 << i) - 1) & ((1 << n) - 1)
            pos = ctx + max(bin(w).count("1") - 1, 0)
            near = max(pos - window + 1, 0)
            sees[i, near:ctx] = True
            sees[i, :min(sinks, ctx)] = True
            for j in range(n):
                sees[i, ctx + j] = bool((w >> j) & 1)
        there = torch.tensor([r >= 0 for r in rows])
        sees &= there
        used = torch.nonzero(sees.any(0))[:, 0]
        if len(used) == 0:
            continue
        at = torch.tensor(rows)[used].to(dev)
        sees = sees[:, used].to(dev)
        k = k_pages.view(-1, nkv, hd)[at].double().repeat_interleave(group, 1)
        v = v_pages.view(-1, nkv, hd)[at].double().repeat_interleave(group, 1)
        qb = q[b].double()
        s = torch.einsum("ihd,phd->ihp", qb, k) * scale
        s_err = 2.0 ** -23 * hd * abs(scale) * float(torch.einsum("ihd,phd->ihp", qb.abs(), k.abs()).max())
        s = s.masked_fill(~sees[:, None], -math.inf)
        some = sees.any(1)
        lse[b] = torch.logsumexp(s, 2)
        p = torch.where(some[:, None, None], torch.exp(s - lse[b][..., None]), torch.zeros_like(s))
        o[b] = torch.einsum("ihp,phd->ihd", p, v)
        u, t = 2.0 ** -8, 2.0 ** -14 + 2 * s_err
        o_err[b] += (u * o[b].abs() + (u + t) * torch.einsum("ihp,phd->ihd", p, v.abs())) * (1 + 2.0 ** -6)
        lse_err[b] = 2.0 ** -16 + 2 * s_err + 2.0 ** -20 * torch.where(some[:, None], lse[b], 0.0).abs()
    return (o, o_err), (lse, lse_err)


def check_tree(o, lse, ref, label):
    (ro, eo), (rl, el) = ref
    assert bool(torch.isfinite(o).all()), f"{label}: o not finite"
    over = float(((o.double() - ro).abs() / eo).max())
    assert over <= 1.0, f"{label}: o {over:.3f} of its bound"
    none = torch.isinf(rl)
    assert torch.equal(torch.isinf(lse) & (lse < 0), none), f"{label}: rows that see nothing"
    off = torch.where(none, torch.zeros_like(rl), (lse.double() - rl).abs() - el)
    assert float(off.max()) <= 0.0, f"{label}: lse over its bound by {float(off.max()):.3e}"


def random_words(B, n, seed):
    """Words of random trees: a token's ancestors and itself."""
    rng = random.Random(seed)
    words = []
    for _ in range(B):
        row = [1]
        for i in range(1, n):
            row.append(row[rng.randrange(i)] | (1 << i))
        words.append(row)
    return words


def signed(words):
    return [[w - (1 << 64) if w >> 63 else w for w in row] for row in words]


def paged_state(B, n, nkv, hd, page, lens, seed=0, spare=3, dtype=torch.bfloat16, device="cpu", width=None):
    """Pools whose rows all hold NaN but those of positions 0 .. len + n - 1, in shuffled pages;
    table entries past a sequence's last page are -1."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    width = width or (max(lens) + n + page - 1) // page
    need = [(c + n + page - 1) // page for c in lens]
    num_pages = sum(need) + spare
    ids = list(range(num_pages))
    rng.shuffle(ids)
    table = [[ids.pop() if e < need[b] else -1 for e in range(width)] for b in range(B)]
    k = torch.full((num_pages, page, nkv, hd), math.nan)
    v = torch.full((num_pages, page, nkv, hd), math.nan)
    for b in range(B):
        at = torch.tensor(rows_of(table, b, range(lens[b] + n), page, num_pages))
        for pool in (k, v):
            pool.view(-1, nkv, hd)[at] = torch.randn(len(at), nkv, hd, generator=g) * 0.5
    return k.to(dtype).to(device), v.to(dtype).to(device), table


def append_reference(k_new, v_new, k_pages, v_pages, table, lens):
    B, n, nkv, hd = k_new.shape
    num_pages, page = k_pages.shape[:2]
    k, v = k_pages.clone(), v_pages.clone()
    for b in range(B):
        for i, r in enumerate(rows_of(table, b, range(lens[b], lens[b] + n), page, num_pages)):
            if r >= 0:
                k.view(-1, nkv, hd)[r] = k_new[b, i]
                v.view(-1, nkv, hd)[r] = v_new[b, i]
    return k, v


def compact_reference(k_pages, v_pages, table, lens, path, accepted):
    num_pages, page, nkv, hd = k_pages.shape
    k, v = k_pages.clone(), v_pages.clone()
    for b, row in enumerate(path):
        n = len(row)
        for i in range(min(max(accepted[b], 0), n)):
            if not i < row[i] < n:
                continue
            src, dst = rows_of(table, b, [lens[b] + row[i], lens[b] + i], page, num_pages)
            if src >= 0 and dst >= 0:
                k.view(-1, nkv, hd)[dst] = k_pages.view(-1, nkv, hd)[src]
                v.view(-1, nkv, hd)[dst] = v_pages.view(-1, nkv, hd)[src]
    return k, v
