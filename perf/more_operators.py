"""Cases, plain forms and exact forms of latent attention and of the paged cache's bookkeeping.

Kinds of case:
  fwd     latent attention in its expanded form, forward: (o, lse)
  step    its forward and backward, as a training step calls them: (o, lse, dq, dkv, dk_rope)
  decode  its absorbed form: n new tokens a sequence over a paged cache of latent rows: (o, lse)
  pages   pages reserved for the new positions of a batch, with the slot map of its tokens, and given
          back: (slots, offsets, granted, page_table, free_pages, free_count)
  write   rows of a ragged batch into the pages by its slot map: (pages), or (k_pages, v_pages)

Expanded form: head h of token j has the key (kv[j, h, :dn], k_rope[j]) and the value kv[j, h, dn:]; k_rope is
shared by the heads. Query i sees keys j <= i. Absorbed form: every head's key of a position is its
cached row (c, k_rope) of dc + dr numbers, and its value is c; new token i of a sequence with ctx
committed positions sees the positions up to ctx + i.
"""
import math
import random

import torch

own = False


def listed():
    return [
        # Smallest forward: a short odd batch of the 12-head decoder layer at head dim 64.
        dict(name="fwd_short", kind="fwd", B=2, S=257, nh=12, dn=64, dr=32, dv=64),
        # A prompt pass of 16 heads at head dim 128, its length odd.
        dict(name="fwd_long", kind="fwd", B=4, S=4093, nh=16, dn=128, dr=64, dv=128),
        # Training step of the 12-head layer on the sequence length that its trainer uses.
        dict(name="step_dim768", kind="step", B=8, S=1024, nh=12, dn=64, dr=32, dv=64),
        # Training step of 16 heads at head dim 128 on long sequences, their length odd.
        dict(name="step_long", kind="step", B=2, S=4001, nh=16, dn=128, dr=64, dv=128),
        # Smallest serving call: the next token of one sequence with a short cache.
        dict(name="decode_single", kind="decode", B=1, n=1, nh=16, dc=512, dr=64, page=64, ctx=1000, lens=1),
        # The decode step of a serving batch: 64 ragged sequences of up to 4096 positions, 16 heads.
        dict(name="decode_batch", kind="decode", B=64, n=1, nh=16, dc=512, dr=64, page=64, ctx=4096, lens=2),
        # Drafted decoding with many heads: 4 tokens of 32 heads each (128 rows a sequence), small pages.
        dict(name="decode_draft", kind="decode", B=48, n=4, nh=32, dc=512, dr=64, page=16, ctx=4096, lens=3),
        # A decode step's bookkeeping: one new position for each of 64 sequences.
        dict(name="pages_step", kind="pages", B=64, new=1, page=64, ctx=4096, spare=1.5, lens=4),
        # Ragged prompts of 512 requests, more than the free pages hold (the last ones get none).
        dict(name="pages_prompts", kind="pages", B=512, new=4096, page=16, ctx=0, spare=0.9, lens=5),
        # New latent rows of a decode step of 64 sequences.
        dict(name="write_step", kind="write", pool="latent", B=64, new=1, dc=512, dr=64, page=64, ctx=4096, lens=6),
        # Ragged prompts' latent rows.
        dict(name="write_prompts", kind="write", pool="latent", B=32, new=4096, dc=512, dr=64, page=64, ctx=0, lens=7),
        # Ragged prompts' K and V rows of 4 heads at head dim 128.
        dict(name="write_prompts_kv", kind="write", pool="kv", B=16, new=4096, nkv=4, hd=128, page=16, ctx=0, lens=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "step", "step", "decode", "decode", "decode", "pages", "pages", "write", "write"])
    lens = rng.randrange(1 << 30)
    if kind in ("fwd", "step"):
        dn, dr, dv = rng.choice([(128, 64, 128), (128, 64, 128), (64, 32, 64), (64, 32, 64), (96, 32, 64), (32, 16, 48)])
        S, nh = _log_int(rng, 30, 4090), rng.choice([1, 3, 4, 8, 12, 16])
        most = 4 * 16 * 4093 * 4093 if kind == "fwd" else 2 * 16 * 4001 * 4001
        return dict(kind=kind, B=max(1, min(_log_int(rng, 1, 16), most // (S * S * nh))), S=S, nh=nh, dn=dn, dr=dr, dv=dv)
    page = rng.choice([16, 32, 64, 128])
    if kind == "decode":
        dc, dr = rng.choice([(512, 64), (512, 64), (512, 64), (256, 32), (256, 64), (128, 16)])
        n, nh = rng.choice([(1, 16), (1, 16), (1, 8), (1, 64), (1, 128), (2, 16), (4, 12), (3, 40), (7, 5), (16, 4), (1, 1)])
        ctx = _log_int(rng, 20, 16384)
        return dict(kind=kind, B=max(1, min(_log_int(rng, 1, 64), 64 * 4096 // ctx, 48 * 4 * 32 * 4096 // (ctx * n * nh))),
                    n=n, nh=nh, dc=dc, dr=dr, page=page, ctx=ctx, lens=lens)
    B = _log_int(rng, 1, 512)
    new = rng.choice([1, 1, 5]) if rng.random() < 0.4 else _log_int(rng, 2, 4096)
    if kind == "pages":
        return dict(kind=kind, B=B, new=new, page=page, ctx=rng.choice([0, _log_int(rng, 1, 4096)]),
                    spare=rng.choice([0.5, 0.95, 1.2, 2.0]), lens=lens)
    B = max(1, min(B, 32 * 4096 // new))
    wide = dict(pool="latent", dc=512, dr=64) if rng.random() < 0.5 else rng.choice(
        [dict(pool="latent", dc=128, dr=16), dict(pool="kv", nkv=2, hd=64), dict(pool="kv", nkv=4, hd=128),
         dict(pool="kv", nkv=1, hd=32)])
    if wide.get("nkv") == 4:
        B = max(1, min(B, 16 * 4096 // new))
    return dict(kind=kind, B=B, new=new, page=page, ctx=rng.choice([0, _log_int(rng, 1, 600)]), lens=lens, **wide)


# ---- what a program has in hand before the call -----------------------------------------

def _ctx_lens(case):
    """Committed positions of each sequence: ragged, the longest of them case["ctx"], one in ten new."""
    rng = random.Random(case["lens"])
    full = case["ctx"]
    lens = [0 if rng.random() < 0.1 else rng.randint(full // 4, full) for _ in range(case["B"])]
    lens[rng.randrange(case["B"])] = full
    return lens


def _new_lens(case):
    """New positions of each sequence: case["new"] of them, or ragged up to it when it is a prompt's length."""
    if case["new"] <= 5:
        return [case["new"]] * case["B"]
    rng = random.Random(case["lens"] + 1)
    return [rng.randint(0, case["new"]) for _ in range(case["B"])]


def _pages_of(positions, page):
    return (positions + page - 1) // page


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)

    def randn(*shape, times=0.5):
        return (torch.randn(shape, generator=gen, device="cuda") * times).to(torch.bfloat16)

    st = dict(case)
    if case["kind"] in ("fwd", "step"):
        B, S, nh, dn, dr, dv = (case[x] for x in ("B", "S", "nh", "dn", "dr", "dv"))
        st.update(q=randn(B, S, nh, dn + dr), kv=randn(B, S, nh, dn + dv), k_rope=randn(B, S, dr),
                  scale=(dn + dr) ** -0.5)
        if case["kind"] == "step":
            st["dO"] = randn(B, S, nh, dv, times=1.0)
        return st
    B, page = case["B"], case["page"]
    ctx = _ctx_lens(case)
    new = [case["n"]] * B if case["kind"] == "decode" else _new_lens(case)
    held = [_pages_of(c, page) if case["kind"] == "pages" else _pages_of(c + x, page) for c, x in zip(ctx, new)]
    width = max(_pages_of(c + x, page) for c, x in zip(ctx, new)) + 1
    need = sum(_pages_of(c + x, page) for c, x in zip(ctx, new)) - sum(held)
    spare = int(case["spare"] * need) + 1 if case["kind"] == "pages" else 3
    pool = sum(held) + spare + 64              # 64 pages of other requests
    ids = list(range(pool))
    rng.shuffle(ids)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-1] * (width - h))
        at += h
    st.update(table=_int32(table), ctx_t=_int32(ctx))
    if case["kind"] == "decode":
        dc, dr = case["dc"], case["dr"]
        st.update(pages=randn(pool, page, dc + dr), q=randn(B, case["n"], case["nh"], dc + dr), scale=192 ** -0.5)
        return st
    total = sum(new)
    if case["kind"] == "pages":
        st.update(new_t=_int32(new), free=_int32(ids[at:at + spare] + [-1] * (pool - spare)), count=_int32([spare]), tokens=total + 3)
        return st
    slots = []
    for b in range(B):
        row = table[b]
        slots += [row[p // page] * page + p % page for p in range(ctx[b], ctx[b] + new[b])]
    slots += [-1] * 3                          # a padded batch: rows without a place
    st["slots"] = torch.tensor(slots, dtype=torch.int64, device="cuda")
    if case["pool"] == "latent":
        st.update(pages=randn(pool, page, case["dc"] + case["dr"]), c=randn(total + 3, case["dc"]),
                  k_rope=randn(total + 3, case["dr"]))
    else:
        nkv, hd = case["nkv"], case["hd"]
        st.update(k_pages=randn(pool, page, nkv, hd), v_pages=randn(pool, page, nkv, hd), k_new=randn(total + 3, nkv, hd),
                  v_new=randn(total + 3, nkv, hd))
    return st


# ---- plain forms: elementary torch operations in 32 bits --------------------------------

def _plain_expanded(st):
    S, nh, dn, dv, scale = st["S"], st["nh"], st["dn"], st["dv"], st["scale"]
    qf = st["q"].float().transpose(1, 2)                                   # [B, nh, S, dn + dr]
    kvf = st["kv"].float().transpose(1, 2)
    rope = st["k_rope"].float()[:, None].expand(-1, nh, -1, -1)
    kf, vf = torch.cat([kvf[..., :dn], rope], dim=3), kvf[..., dn:]
    pos = torch.arange(S, device=qf.device)
    s = (qf @ kf.transpose(2, 3)) * scale
    s = s.masked_fill(pos[None, :] > pos[:, None], -math.inf)
    m = s.amax(dim=3, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(dim=3, keepdim=True)
    p = e / total
    o = p @ vf
    out = o.transpose(1, 2).to(torch.bfloat16)
    lse = (m + torch.log(total))[..., 0].transpose(1, 2).contiguous()
    if st["kind"] == "fwd":
        return out, lse
    do = st["dO"].float().transpose(1, 2)
    dv_ = p.transpose(2, 3) @ do
    ds = p * (do @ vf.transpose(2, 3) - (do * o).sum(dim=3, keepdim=True))
    dq = (ds @ kf) * scale
    dk = (ds.transpose(2, 3) @ qf) * scale
    dkv = torch.cat([dk[..., :dn], dv_], dim=3)
    return (out, lse, dq.transpose(1, 2).to(torch.bfloat16), dkv.transpose(1, 2).to(torch.bfloat16),
            dk[..., dn:].sum(dim=1).to(torch.bfloat16))


def _plain_decode(st):
    q, table, ctx = st["q"], st["table"], st["ctx_t"].long()
    B, n, nh, dc, page = (st[x] for x in ("B", "n", "nh", "dc", "page"))
    T = table.shape[1] * page
    rows = st["pages"][table.clamp(min=0).long()].view(B, T, -1).float()
    there = (table >= 0).repeat_interleave(page, dim=1)
    p = torch.arange(T, device=q.device)
    last = ctx[:, None] + torch.arange(n, device=q.device)                  # [B, n]
    seen = (p <= last[:, :, None]) & there[:, None, :]
    s = (q.float().view(B, n * nh, -1) @ rows.transpose(1, 2)) * st["scale"]
    s = s.view(B, n, nh, T).masked_fill(~seen[:, :, None], -math.inf)
    m = s.amax(dim=3, keepdim=True).clamp(min=-1e30)
    e = torch.exp(s - m)
    total = e.sum(dim=3, keepdim=True)
    o = (e.view(B, n * nh, T) @ rows[..., :dc]).view(B, n, nh, dc) / total.clamp(min=1e-30)
    return o.to(torch.bfloat16), (m + torch.log(total))[..., 0]


def _plain_reserve(table, ctx, new, free, count, page, tokens):
    B, width = table.shape
    c = ctx.long().clamp(0, width * page)
    room = torch.minimum(new.long().clamp(min=0), width * page - c)
    held, full = (c + page - 1) // page, (c + room + page - 1) // page
    need = full - held
    upto = torch.cumsum(need, 0)
    ok = (need == 0) | (upto <= count)
    granted = torch.where(ok, room, 0)
    j = torch.arange(width, device=table.device)
    fresh = (j >= held[:, None]) & (j < full[:, None]) & ok[:, None]
    k = (upto - need)[:, None] + j - held[:, None]
    ids = free[(count.long() - 1 - k).clamp(0, free.numel() - 1)]
    table.copy_(torch.where(fresh, ids, table))
    count.sub_(torch.where(ok & (need > 0), upto, 0).amax().to(torch.int32))
    ends = torch.cumsum(new.long().clamp(min=0), 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(tokens, device=table.device)
    b = torch.searchsorted(ends, t, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    at = t - offsets[b]
    inside &= at < granted[b]
    pos = torch.where(inside, c[b] + at, 0)
    ids = table[b, pos // page].long()
    slots = torch.where(inside & (ids >= 0), ids * page + pos % page, -1)
    return slots, offsets.to(torch.int32), granted.to(torch.int32)


def _plain_release(table, held, keep, free, count, page):
    width = table.shape[1]
    hp = (held.long().clamp(0, width * page) + page - 1) // page
    kp = (keep.long().clamp(0, width * page) + page - 1) // page
    j = torch.arange(width, device=table.device)
    gone = (j >= kp[:, None]) & (j < hp[:, None])
    real = gone & (table >= 0) & (table < free.numel())
    rank = torch.cumsum(real.view(-1).long(), 0) - 1
    total = rank[-1] + 1
    to = count.long() + total - 1 - rank
    to = torch.where(real.view(-1) & (to < free.numel()), to, free.numel())
    longer = torch.cat([free, free[:1]])
    longer[to] = table.view(-1)
    free.copy_(longer[:-1])
    count.copy_((count + total).clamp(max=free.numel()).to(torch.int32))
    table.masked_fill_(gone, -1)


def _plain_write(st):
    inside = (st["slots"] >= 0).nonzero()[:, 0]
    at = st["slots"][inside]
    if st["pool"] == "latent":
        pool = st["pages"].view(-1, st["dc"] + st["dr"])
        pool[at] = torch.cat([st["c"], st["k_rope"]], dim=1)[inside]
        return st["pages"]
    nkv, hd = st["nkv"], st["hd"]
    st["k_pages"].view(-1, nkv, hd)[at] = st["k_new"][inside]
    st["v_pages"].view(-1, nkv, hd)[at] = st["v_new"][inside]
    return st["k_pages"], st["v_pages"]


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    st = state
    kind = st["kind"]
    if not own:
        if kind in ("fwd", "step"):
            return _plain_expanded(st)
        if kind == "decode":
            return _plain_decode(st)
        if kind == "write":
            return _plain_write(st)
        out = _plain_reserve(st["table"], st["ctx_t"], st["new_t"], st["free"], st["count"], st["page"], st["tokens"])
        _plain_release(st["table"], st["ctx_t"] + out[2], st["ctx_t"], st["free"], st["count"], st["page"])
        return (*out, st["table"], st["free"], st["count"])
    from bwd_xattn_fwd_gb300 import xattn
    if kind in ("fwd", "step"):
        o, lse = xattn.attention_latent_fwd(st["q"], st["kv"], st["k_rope"])
        if kind == "fwd":
            return o, lse
        return (o, lse, *xattn.attention_latent_bwd(st["q"], st["kv"], st["k_rope"], o, st["dO"], lse))
    if kind == "decode":
        return xattn.attention_latent_decode(st["q"], st["pages"], st["table"], st["ctx_t"], st["dc"], st["scale"])
    if kind == "write":
        if st["pool"] == "latent":
            xattn.latent_write(st["c"], st["k_rope"], st["pages"], st["slots"])
            return st["pages"]
        xattn.cache_write(st["k_new"], st["v_new"], st["k_pages"], st["v_pages"], st["slots"])
        return st["k_pages"], st["v_pages"]
    # The turn of a batch whose drafted positions are all rejected: reserved, and given back.
    out = xattn.cache_reserve(st["table"], st["ctx_t"], st["new_t"], st["free"], st["count"], st["page"], st["tokens"])
    xattn.cache_release(st["table"], st["ctx_t"] + out[2], st["ctx_t"], st["free"], st["count"], st["page"])
    return (*out, st["table"], st["free"], st["count"])


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    B = case["B"]
    if case["kind"] in ("fwd", "step"):
        S, nh, dn, dr, dv = (case[x] for x in ("S", "nh", "dn", "dr", "dv"))
        pairs = B * nh * (S * (S + 1) // 2)
        inputs = 2 * B * S * (nh * (2 * dn + dr + dv) + dr)
        o, lse = 2 * B * S * nh * dv, 4 * B * S * nh
        if case["kind"] == "fwd":
            return {"bytes": inputs + o + lse, "flops": 2 * (dn + dr + dv) * pairs}
        return {"bytes": 2 * inputs + 2 * o + lse, "flops": 2 * (4 * (dn + dr) + 3 * dv) * pairs}
    ctx = _ctx_lens(case)
    if case["kind"] == "decode":
        n, nh, dc, dr = (case[x] for x in ("n", "nh", "dc", "dr"))
        seen = sum(c + n for c in ctx)
        pairs = nh * sum(c + i + 1 for c in ctx for i in range(n))
        return {"bytes": 2 * seen * (dc + dr) + 2 * B * n * nh * (2 * dc + dr) + 4 * B * n * nh,
                "flops": 2 * (2 * dc + dr) * pairs}
    new, page = _new_lens(case), case["page"]
    if case["kind"] == "pages":
        # Reserve: lengths, the pages taken (from the stack, into the table), the slots; release: the pages back.
        need = [_pages_of(c + x, page) - _pages_of(c, page) for c, x in zip(ctx, new)]
        taken = sum(need) if case["spare"] >= 1 else int(case["spare"] * sum(need))
        return {"bytes": 8 * (sum(new) + 3) + 16 * B + 24 * taken, "flops": 0}
    row = 2 * (case["dc"] + case["dr"]) if case["pool"] == "latent" else 4 * case["nkv"] * case["hd"]
    return {"bytes": sum(new) * (2 * row + 8), "flops": 0}


# ---- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    if case["kind"] in ("pages", "write"):
        return None                            # whole numbers and copies: nothing is rounded
    st = prepare(case, seed)
    if case["kind"] == "decode":
        return _exact_decode(case, st)
    B, S, nh, dn = (case[x] for x in ("B", "S", "nh", "dn"))
    scale = 1.0 / math.sqrt(dn + case["dr"])
    leaf = {x: st[x].double().requires_grad_(case["kind"] == "step") for x in ("q", "kv", "k_rope")}
    hidden = torch.ones(S, S, dtype=torch.bool, device="cuda").triu(1)
    o = torch.empty(B, S, nh, case["dv"], dtype=torch.float64, device="cuda")
    lse = torch.empty(B, S, nh, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(nh):
            q, kv = leaf["q"][b, :, h], leaf["kv"][b, :, h]
            s = q[:, :dn] @ kv[:, :dn].T + q[:, dn:] @ leaf["k_rope"][b].T
            s = s.mul(scale).masked_fill(hidden, -math.inf)
            out = torch.softmax(s, dim=1) @ kv[:, dn:]
            if case["kind"] == "step":
                (out * st["dO"][b, :, h].double()).sum().backward()
            o[b, :, h] = out.detach()
            lse[b, :, h] = torch.logsumexp(s.detach(), dim=1)
    if case["kind"] == "fwd":
        return o, lse
    return (o, lse, *(leaf[x].grad for x in ("q", "kv", "k_rope")))


def _exact_decode(case, st):
    B, n, nh, dc, page = (case[x] for x in ("B", "n", "nh", "dc", "page"))
    o = torch.zeros(B, n, nh, dc, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, n, nh, dtype=torch.float64, device="cuda")
    table = st["table"].tolist()
    for b, c in enumerate(_ctx_lens(case)):
        rows = torch.tensor([table[b][p // page] * page + p % page for p in range(c + n)], device="cuda")
        row = st["pages"].view(-1, dc + case["dr"])[rows].double()
        for i in range(n):
            s = st["q"][b, i].double() @ row[:c + i + 1].T * st["scale"]
            lse[b, i] = torch.logsumexp(s, dim=1)
            o[b, i] = torch.softmax(s, dim=1) @ row[:c + i + 1, :dc]
    return o, lse
