"""Latent attention in 64 bits, straight from its definition, with elementwise error bounds for a
computation that rounds where the library does; and the paged cache's tables and slot maps in
plain Python.

Bounds as in window_ref.py (u = 2^-8: P, dS and the outputs are rounded to bf16, each off by at most
half a step; t = 2^-11 and the scores' slack for exponentials and sums in fp32), with a head's key the
dn numbers of kv and the dr of k_rope. dk_rope is summed over the heads before it is rounded: its
bound is the sum of theirs. Decode rounds P and o once each: u |o| + (u + t) sum P |c|.
"""
import math
import random

import torch


def latent_inputs(B, S, nh, dn, dr, dv, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, times=0.5):
        return (torch.randn(*shape, generator=g) * times).to(torch.bfloat16).to(device)

    return {"q": rnd(B, S, nh, dn + dr), "kv": rnd(B, S, nh, dn + dv), "k_rope": rnd(B, S, dr),
            "dO": rnd(B, S, nh, dv, times=1.0)}


def latent_reference(x, scale):
    """dict name -> (value, bound) in float64."""
    q, kv, rope, dO = (x[n].double() for n in ("q", "kv", "k_rope", "dO"))
    B, S, nh, dqk = q.shape
    dr = rope.shape[2]
    dn = dqk - dr
    qh, doh, kvh = q.transpose(1, 2), dO.transpose(1, 2), kv.transpose(1, 2)
    kh = torch.cat([kvh[..., :dn], rope[:, None].expand(B, nh, S, dr)], 3)
    vh = kvh[..., dn:]
    hidden = torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1)
    s = (qh @ kh.transpose(2, 3)) * scale
    lse = torch.logsumexp(s.masked_fill(hidden, -math.inf), dim=3)
    p = torch.exp(s - lse[..., None]).masked_fill(hidden, 0.0)
    o = p @ vh
    ds = p * (doh @ vh.transpose(2, 3) - (doh * o).sum(3, keepdim=True))
    s_err = 2.0 ** -23 * dqk * float((qh.abs() @ kh.abs().transpose(2, 3)).max()) * abs(scale)
    u, t = 2.0 ** -8, 2.0 ** -11 + 2 * s_err
    lse_tol = 8e-5 + 2 * s_err + 2.0 ** -20 * float(lse.abs().max())
    pv = p @ vh.abs()
    e = (2 * u + t) * (doh.abs() * pv).sum(3, keepdim=True)
    ds_err = (2 * u + t) * ds.abs() + t * p * ((doh.abs() @ vh.abs().transpose(2, 3)) + e) + p * e
    a = abs(scale)
    dk, dk_err = (ds.transpose(2, 3) @ qh) * scale, a * (ds_err.transpose(2, 3) @ qh.abs())
    dv, dv_err = p.transpose(2, 3) @ doh, (u + t) * (p.transpose(2, 3) @ doh.abs())
    dq, dkv = (ds @ kh) * scale, torch.cat([dk[..., :dn], dv], 3)
    out = {
        "o": (o, u * o.abs() + (u + t) * pv),
        "dq": (dq, u * dq.abs() + a * (ds_err @ kh.abs())),
        "dkv": (dkv, u * dkv.abs() + torch.cat([dk_err[..., :dn], dv_err], 3)),
    }
    out = {n: (val.transpose(1, 2), err.transpose(1, 2) * (1 + 2.0 ** -6) + 1e-30) for n, (val, err) in out.items()}
    rope_grad = dk[..., dn:].sum(1)
    out["dk_rope"] = (rope_grad, (u * rope_grad.abs() + dk_err[..., dn:].sum(1)) * (1 + 2.0 ** -6) + 1e-30)
    out["lse"] = (lse.transpose(1, 2), torch.full_like(lse.transpose(1, 2), lse_tol))
    return out


def rows_of(table, b, positions, page, num_pages):
    """Pool row of each position, -1 where there is none."""
    out = []
    for p in positions:
        e = table[b][p // page] if 0 <= p < len(table[b]) * page else -1
        out.append(e * page + p % page if 0 <= e < num_pages else -1)
    return out


def latent_state(B, n, width, page, lens, seed=0, spare=3, device="cpu", dtype=torch.bfloat16, table_width=None):
    """A pool of rows that hold NaN but those of positions 0 .. len + n - 1, in shuffled pages, and its table."""
    rng = random.Random(seed)
    g = torch.Generator().manual_seed(seed)
    table_width = table_width or (max(lens) + n + page - 1) // page
    need = [(c + n + page - 1) // page for c in lens]
    num_pages = sum(need) + spare
    ids = list(range(num_pages))
    rng.shuffle(ids)
    table = [[ids.pop() if e < need[b] else -1 for e in range(table_width)] for b in range(B)]
    pages = torch.full((num_pages, page, width), math.nan)
    for b in range(B):
        at = torch.tensor(rows_of(table, b, range(lens[b] + n), page, num_pages))
        pages.view(-1, width)[at] = torch.randn(len(at), width, generator=g) * 0.5
    return pages.to(dtype).to(device), table


def latent_decode_reference(q, pages, table, lens, dc, scale):
    """((o, bound), (lse, bound)) in float64."""
    B, n, nh, width = q.shape
    num_pages, page, _ = pages.shape
    dev, cap = q.device, len(table[0]) * page
    o = torch.zeros(B, n, nh, dc, dtype=torch.float64, device=dev)
    o_err = torch.full_like(o, 1e-30)
    lse = torch.full((B, n, nh), -math.inf, dtype=torch.float64, device=dev)
    lse_err = torch.zeros_like(lse)
    u = 2.0 ** -8
    for b in range(B):
        ctx = min(max(lens[b], 0), cap - n)
        rows = rows_of(table, b, range(ctx + n), page, num_pages)
        for i in range(n):
            at = [r for r in rows[:ctx + i + 1] if r >= 0]
            if not at:
                continue
            row = pages.view(-1, width)[torch.tensor(at, device=dev)].double()
            qi = q[b, i].double()
            s = qi @ row.T * scale
            s_err = 2.0 ** -23 * width * abs(scale) * float((qi.abs() @ row.abs().T).max())
            t = 2.0 ** -14 + 2 * s_err
            lse[b, i] = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[b, i][:, None])
            o[b, i] = p @ row[:, :dc]
            o_err[b, i] += (u * o[b, i].abs() + (u + t) * (p @ row[:, :dc].abs())) * (1 + 2.0 ** -6)
            lse_err[b, i] = 2.0 ** -16 + 2 * s_err + 2.0 ** -20 * lse[b, i].abs()
    return (o, o_err), (lse, lse_err)


def pages_for(positions, page):
    return (positions + page - 1) // page


def reserve_reference(table, ctx, new, free, count, page, tokens, num_pages):
    """(table, count, slots, offsets, granted) after the pages of `new` positions are taken."""
    table, cap = [list(r) for r in table], len(table[0]) * page
    count = min(max(count, 0), num_pages)
    slots, offsets, granted, upto, taken = [-1] * tokens, [0], [], 0, 0
    for b in range(len(table)):
        c = min(max(ctx[b], 0), cap)
        fresh = max(new[b], 0)
        room = min(fresh, cap - c)
        held, full = pages_for(c, page), pages_for(c + room, page)
        first, upto = upto, upto + full - held
        end = offsets[b] + fresh
        ok = (full == held or upto <= count) and end <= tokens
        if ok:
            for k in range(full - held):
                table[b][held + k] = free[count - 1 - (first + k)]
                taken = upto
            for i in range(room):
                e = table[b][(c + i) // page]
                slots[offsets[b] + i] = e * page + (c + i) % page if 0 <= e < num_pages else -1
        granted.append(room if ok else 0)
        offsets.append(end)
    return table, count - taken, slots, offsets, granted


def release_reference(table, held, keep, free, count, page, num_pages):
    """(table, free, count) after the pages behind `keep` are given back."""
    table, free, cap = [list(r) for r in table], list(free), len(table[0]) * page
    count = min(max(count, 0), num_pages)
    back = []
    for b, row in enumerate(table):
        lo, hi = (pages_for(min(max(x[b], 0), cap), page) for x in (keep, held))
        for j in range(lo, hi):
            if 0 <= row[j] < num_pages:
                back.append(row[j])
            row[j] = -1
    for r, e in enumerate(back):
        at = count + len(back) - 1 - r
        if at < num_pages:
            free[at] = e
    return table, free, min(count + len(back), num_pages)
