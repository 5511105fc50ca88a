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


# ---- how far off the norms may be -----------------------------------------------------------
#
# The bounds above add every rounding with one sign, so that behind a few hundred positions a fault may hide in them. The
# norms below do not. A rounding of v to bf16 is off by an amount spread evenly over half a step to either side, h(v) =
# 2^(floor(log2 |v|) - 8) (0 where bf16 holds v), of variance h(v)^2 / 3, and the roundings are independent. With u^2 for those
# variances, the squared error of an output row is expected to be
#   o_i:  u^2(o_i) + sum_j u^2(P_ij) v_j^2
#   dv_j: u^2(dv_j) + sum_i u^2(P_ij) dO_i^2
#   dq_i: u^2(dq_i) + a^2 (sum_j u^2(dS_ij) k_j^2 + H_i (sum_j P_ij k_j)^2)
#   dk_j: u^2(dk_j) + a^2 sum_i (u^2(dS_ij) + H_i P_ij^2) q_i^2
# (a: scale), with H_i = sum_d dO_id^2 u^2(o_id), the variance of D = dO . o from o's rounding. Roundings in fp32 are 2^-16 of
# these and drop out.
# The sum over a block spreads about its expectation E. A row's roundings of P or dS add the square of several independent numbers
# of expectation e, whose standard deviation is at most that of one number's square, 2^(1/2) e; different rows' are independent:
# (2 sum e^2)^(1/2). D_i's error reaches dq_i alone (the same with e = a^2 H_i |sum_j P_ij k_j|^2), but every dk_j: there the sum is a
# quadratic form of the D_i's errors with M_ik = a^2 (H_i H_k)^(1/2) (q_i . q_k) sum_j P_ij P_kj, of standard deviation 2^(1/2) |M|
# (Frobenius), for the sum over the heads at most the sum of theirs. With d the sum of these, a squared error may be E + 8 d: 12
# times E for a sum that one number rules (the first rows' gradients are by far the largest), which it passes once in 2000.
SPREADS = 8.0


def _variance(v):
    half_step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -120))) - 8)
    return torch.where(v.to(torch.bfloat16).double() == v, 0.0, half_step ** 2 / 3)


def _blocks(S):
    """Blocks of 128 rows, the last of them the last 128, and the whole."""
    return [slice(r, r + 128) for r in sorted({min(r, max(S - 128, 0)) for r in range(0, S, 128)})] + [slice(0, S)]


def latent_norms(x, scale):
    """dict part -> (exact [B, nh, S, columns], allowed squared errors [blocks, B, nh]) in float64 (dk_rope: one head). Parts: o, dv,
    dk, dk_rope, and dq's two."""
    q, kv, rope, dO = (x[n].double() for n in ("q", "kv", "k_rope", "dO"))
    B, S, nh, dqk = q.shape
    dr = rope.shape[2]
    dn = dqk - dr
    qh, doh, kvh = q.transpose(1, 2), dO.transpose(1, 2), kv.transpose(1, 2)
    kh = torch.cat([kvh[..., :dn], rope[:, None].expand(B, nh, S, dr)], 3)
    vh = kvh[..., dn:]
    hidden = torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1)
    s = ((qh @ kh.transpose(2, 3)) * scale).masked_fill(hidden, -math.inf)
    p = torch.softmax(s, dim=3)
    del s
    o = p @ vh
    ds = p * (doh @ vh.transpose(2, 3) - (doh * o).sum(3, keepdim=True))
    dq, dk, dv = (ds @ kh) * scale, (ds.transpose(2, 3) @ qh) * scale, p.transpose(2, 3) @ doh
    up, ud = _variance(p), _variance(ds)
    H = (doh ** 2 * _variance(o)).sum(3, keepdim=True)
    by_query = scale ** 2 * (ud @ kh ** 2 + H * (p @ kh) ** 2)             # of dq, [B, nh, S, dn + dr]
    v2 = (vh ** 2).sum(3)

    def rows(val, e):                                                      # e: [B, nh, S]
        own = _variance(val).sum(3)
        return val, torch.stack([(own[..., r] + e[..., r]).sum(2) + SPREADS * (2 * (e[..., r] ** 2).sum(2)) ** 0.5
                                 for r in _blocks(S)])

    def keys(val, u, x, of_D, heads=lambda t: t):
        """What sum_i r_ij x_i adds to the keys' rows, r of the variances u [B, nh, query, key]. heads: the sum over the heads."""
        own, x2 = _variance(val).sum(3), (x ** 2).sum(3)
        e = heads((u.transpose(2, 3) @ x2[..., None])[..., 0])
        gram = (x @ x.transpose(2, 3)) * (H * H.transpose(2, 3)).sqrt() if of_D else None
        out = []
        for r in _blocks(S):
            room = (own[..., r] + e[..., r]).sum(2) + SPREADS * (2 * (e[..., r] ** 2).sum(2)) ** 0.5
            if of_D:
                m = gram * (p[..., r] @ p[..., r].transpose(2, 3))
                room = room + scale ** 2 * heads(m.diagonal(dim1=2, dim2=3).sum(2) + SPREADS * (2 * (m ** 2).sum((2, 3))) ** 0.5)
            out.append(room)
        return val, torch.stack(out)

    return {
        "o": rows(o, (up @ v2[..., None])[..., 0]), "dq": rows(dq[..., :dn], by_query[..., :dn].sum(3)),
        "dq rope": rows(dq[..., dn:], by_query[..., dn:].sum(3)), "dv": keys(dv, up, doh, False),
        "dk": keys(dk[..., :dn], scale ** 2 * ud, qh[..., :dn], True),
        "dk_rope": keys(dk[..., dn:].sum(1, keepdim=True), scale ** 2 * ud, qh[..., dn:], True, lambda t: t.sum(1, keepdim=True)),
    }


def norm_parts(got, dn):
    """The parts of latent_norms in what the calls give."""
    t = {n: got[n].double().transpose(1, 2) for n in ("o", "dq", "dkv")}
    return {"o": t["o"], "dv": t["dkv"][..., dn:], "dq": t["dq"][..., :dn], "dq rope": t["dq"][..., dn:],
            "dk": t["dkv"][..., :dn], "dk_rope": got["dk_rope"].double()[:, None]}


def norm_ratios(got, dn, norms):
    """dict part -> (the largest error's norm over the allowed one, of the blocks and of the whole of a head)."""
    out = {}
    for name, val in norm_parts(got, dn).items():
        exact, room = norms[name]
        err = ((val - exact) ** 2).sum(3)
        err = torch.stack([err[..., r].sum(2) for r in _blocks(exact.shape[2])])
        ratio = (err / room.clamp(min=1e-60)).sqrt().nan_to_num(math.inf)
        out[name] = float(ratio[:-1].max()), float(ratio[-1].max())
    return out


def check_norms(got, dn, norms, what):
    ratios = norm_ratios(got, dn, norms)
    assert all(max(r) <= 1.0 for r in ratios.values()), f"{what}: error norms over the allowed (blocks, whole): {ratios}"


def rounded_latent(x, scale, fault=None):
    """The calls' outputs with the library's roundings (P, dS, o, D from the rounded o, the outputs; all else in 64 bits). fault: a
    mistake to plant, see test_latent_norms_cpu.py."""
    bf = lambda t: t.to(torch.bfloat16).double()
    q, kv, rope, dO = (x[n].double() for n in ("q", "kv", "k_rope", "dO"))
    B, S, nh, dqk = q.shape
    dr = rope.shape[2]
    dn = dqk - dr
    qh, doh, kvh = q.transpose(1, 2), dO.transpose(1, 2), kv.transpose(1, 2)
    kh = torch.cat([kvh[..., :dn], rope[:, None].expand(B, nh, S, dr)], 3)
    vh = kvh[..., dn:]
    s = ((qh @ kh.transpose(2, 3)) * scale).masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), -math.inf)
    lse = torch.logsumexp(s, 3)
    p = torch.exp(s - lse[..., None])
    e = torch.exp(s - s.amax(3, keepdim=True))
    o = bf((bf(e) @ vh) / e.sum(3, keepdim=True))
    D = (doh * o).sum(3, keepdim=True)
    if fault == "no D behind the middle":
        D[:, :, S // 2:] = 0.0
    ds = p * (doh @ vh.transpose(2, 3) - D)
    if fault == "dS of bf16 P":
        ds = bf(p) * (doh @ vh.transpose(2, 3) - D)
    if fault == "16 keys dropped":
        ds[:, :, -128:, 64:80] = 0.0
    if fault == "dS off by 1 %":
        ds = ds * 1.01
    ds = bf(ds)
    dq, dk, dv = bf((ds @ kh) * scale), (ds.transpose(2, 3) @ qh) * scale, bf(bf(p).transpose(2, 3) @ doh)
    rope_grad = dk[..., dn:].sum(1)
    if fault == "one head's k_rope":
        rope_grad = dk[:, 0, :, dn:]
    out = {"o": o, "dq": dq, "dkv": torch.cat([bf(dk[..., :dn]), dv], 3)}
    out = {n: t.transpose(1, 2).contiguous() for n, t in out.items()}
    out.update(dk_rope=bf(rope_grad), lse=lse.transpose(1, 2).contiguous())
    if fault == "no gradient":
        out.update({n: torch.zeros_like(out[n]) for n in ("dq", "dkv", "dk_rope")})
    if fault == "negated":
        out.update({n: -out[n] for n in ("dq", "dkv", "dk_rope")})
    return out
