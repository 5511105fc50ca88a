"""Cases, plain forms and exact forms of the windowed, tree and paged-cache operators.

Kinds of case:
  fwd     window attention with sinks, forward: (o, lse)
  step    its forward and backward, as a training step calls them: (o, lse, dq, dk, dv)
  tree    attention of n drafted tokens a sequence over a paged cache: (o, lse); n = 1 is the decode step
  append  new K/V rows into the pages of a cache: (k_pages, v_pages)
  turn    append of n drafted rows, then compaction to the accepted path: (k_pages, v_pages)

Query i sees key j when j <= i and (i - j < window or j < sinks). In a tree, drafted token i of
a sequence with c committed positions sees the drafted tokens of its word's bits, and the committed
position p when c + depth_i - p < window or p < sinks, depth_i being its number of ancestors.
"""
import math
import random

import torch

own = False

NO_WINDOW = 2**31 - 1


def listed():
    return [
        # Smallest forward: the 12-head decoder layer at hd 32 on short sequences, a short window.
        dict(name="fwd_dim384", kind="fwd", dtype="bf16", B=16, S=256, nh=12, nkv=12, hd=32, window=64, sinks=4),
        # A prompt pass of the long grouped-head shape, its length odd, a quarter of it in the window.
        dict(name="fwd_long", kind="fwd", dtype="bf16", B=4, S=4093, nh=16, nkv=4, hd=64, window=1024, sinks=4),
        # Training step of the grouped-head shape with a window of a quarter of the sequence.
        dict(name="step_gqa", kind="step", dtype="bf16", B=8, S=2048, nh=8, nkv=2, hd=64, window=512, sinks=4),
        # Training step at hd 128: odd length, a window that ends inside tiles, sinks over a tile's end.
        dict(name="step_long_hd128", kind="step", dtype="bf16", B=2, S=4001, nh=16, nkv=4, hd=128, window=1000,
             sinks=130),
        # Training step in fp32 on a short odd sequence, as gradient checks run it.
        dict(name="step_f32", kind="step", dtype="f32", B=2, S=499, nh=4, nkv=2, hd=64, window=100, sinks=3),
        # Smallest serving call: one sequence, a short cache, a tree of 8 drafted tokens.
        dict(name="tree_single", kind="tree", B=1, n=8, nh=16, nkv=4, hd=64, page=16, ctx=300, window=NO_WINDOW, sinks=0,
             lens=1),
        # A serving batch: 64 sequences of up to 4096 cached positions, trees of 16 drafted tokens.
        dict(name="tree_batch", kind="tree", B=64, n=16, nh=16, nkv=4, hd=64, page=64, ctx=4096, window=NO_WINDOW,
             sinks=0, lens=2),
        # The single-token step of a windowed model at hd 128: long caches whose pages behind the window are freed.
        dict(name="token_window", kind="tree", B=64, n=1, nh=16, nkv=4, hd=128, page=16, ctx=16384, window=2048, sinks=4,
             lens=3),
        # New rows of a decode step of 48 sequences.
        dict(name="append_step", kind="append", B=48, n=1, nkv=4, hd=64, page=16, ctx=1000, lens=4),
        # Prompts written to the pages: 16 sequences of 4096 rows at hd 128.
        dict(name="append_prompt", kind="append", B=16, n=4096, nkv=4, hd=128, page=64, ctx=0, lens=5),
        # A turn of drafted decoding on a serving batch: trees of 16 rows appended, the accepted path kept.
        dict(name="turn_batch", kind="turn", B=64, n=16, nkv=4, hd=64, page=64, ctx=2048, lens=6),
        # The same with the largest trees, wide heads and small pages.
        dict(name="turn_wide", kind="turn", B=256, n=61, nkv=8, hd=128, page=16, ctx=300, lens=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "step", "step", "tree", "tree", "tree", "append", "turn"])
    hd = rng.choice([32, 64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    lens = rng.randrange(1 << 30)
    if kind in ("fwd", "step"):
        S = _log_int(rng, 40, 4090)
        nh = nkv * rng.choice([1, 2, 4])
        if kind == "step" and rng.random() < 0.2:
            B = max(1, min(8, 2 * 499 * 499 * 4 // (S * S * nh)))
            S = min(S, 700)
            return dict(kind=kind, dtype="f32", B=B, S=S, nh=nh, nkv=nkv, hd=min(hd, 64), window=_log_int(rng, 8, S),
                        sinks=rng.choice([0, 1, 4, 9]))
        most = 4 * 16 * 4093 * 4093 if kind == "fwd" else 2 * 16 * 4001 * 4001
        B = max(1, min(_log_int(rng, 1, 16), int(most * (64 / max(hd, 64)) / (S * S * nh))))
        return dict(kind=kind, dtype="bf16", B=B, S=S, nh=nh, nkv=nkv, hd=hd, window=_log_int(rng, 16, 2 * S),
                    sinks=rng.choice([0, 1, 4, 4, 16, 64, 130, 200]))
    page = rng.choice([16, 32, 64, 128])
    if kind == "tree":
        n = rng.choice([1, 1, 2, 5, 8, 16, 27, 64])
        ctx = _log_int(rng, 20, 16384)
        B = max(1, min(_log_int(rng, 1, 64), 64 * 16384 // (ctx * nkv)))
        windowed = rng.random() < 0.5
        return dict(kind=kind, B=B, n=n, nh=nkv * rng.choice([1, 2, 4, 7]), nkv=nkv, hd=hd, page=page, ctx=ctx,
                    window=max(n, _log_int(rng, 64, 4096)) if windowed else NO_WINDOW,
                    sinks=rng.choice([0, 4, 100]) if windowed else 0, lens=lens)
    if kind == "append":
        n = _log_int(rng, 1, 4096)
        B = max(1, min(_log_int(rng, 1, 64), 16 * 4096 * 4 * 128 // (n * nkv * hd)))
        return dict(kind=kind, B=B, n=n, nkv=nkv, hd=hd, page=page, ctx=_log_int(rng, 1, 600), lens=lens)
    n = rng.choice([2, 7, 16, 33, 61, 64])
    return dict(kind=kind, B=_log_int(rng, 1, 256), n=n, nkv=nkv, hd=hd, page=page, ctx=_log_int(rng, 1, 600), lens=lens)


# ---- what a program has in hand before the call -----------------------------------------

def _ctx_lens(case):
    """Committed positions of each sequence: ragged, the longest of them case["ctx"]."""
    rng = random.Random(case["lens"])
    full = case["ctx"]
    lens = [rng.randint(full // 4, full) for _ in range(case["B"])]
    lens[rng.randrange(case["B"])] = full
    return lens


def _trees(case, rng):
    """One word a drafted token: its ancestors' bits and its own (token 0 is the root)."""
    words = []
    for _ in range(case["B"]):
        row = [1]
        for i in range(1, case["n"]):
            row.append(row[max(0, i - 1 - int(rng.random() * rng.random() * 6))] | (1 << i))
        words.append([w - (1 << 64) if w >> 63 else w for w in row])
    return words


def _paths(case, rng):
    """Accepted drafted rows of each sequence, ascending, and how many they are."""
    paths, counts = [], []
    for _ in range(case["B"]):
        a = min(case["n"], 1 + int(rng.random() * rng.random() * 10))
        rows = [0] + sorted(rng.sample(range(1, case["n"]), a - 1))
        paths.append(rows + [0] * (case["n"] - a))
        counts.append(a)
    return paths, counts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    dt = torch.float32 if case.get("dtype") == "f32" else torch.bfloat16

    def randn(*shape, times=0.5):
        return (torch.randn(shape, generator=gen, device="cuda") * times).to(dt)

    st = dict(case)
    if case["kind"] in ("fwd", "step"):
        B, S, nh, nkv, hd = (case[x] for x in ("B", "S", "nh", "nkv", "hd"))
        st.update(q=randn(B, S, nh, hd), k=randn(B, S, nkv, hd), v=randn(B, S, nkv, hd))
        if case["kind"] == "step":
            st["dO"] = randn(B, S, nh, hd, times=1.0)
        return st
    B, n, nkv, hd, page = (case[x] for x in ("B", "n", "nkv", "hd", "page"))
    lens = _ctx_lens(case)
    width = (case["ctx"] + n + page - 1) // page
    window, sinks = case.get("window", NO_WINDOW), case.get("sinks", 0)
    rows, used = [], 0
    for c in lens:
        live = [p * page < c + n and (p * page < sinks or (p + 1) * page > c - window) for p in range(width)]
        rows.append(live)
        used += sum(live)
    ids = list(range(used))
    rng.shuffle(ids)
    table = [[ids.pop() if x else -1 for x in row] for row in rows]
    st.update(k_pages=randn(used, page, nkv, hd), v_pages=randn(used, page, nkv, hd),
              table=torch.tensor(table, dtype=torch.int32, device="cuda"),
              lens_t=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if case["kind"] == "tree":
        st["q"] = randn(B, n, case["nh"], hd)
        st["words"] = torch.tensor(_trees(case, rng), dtype=torch.int64, device="cuda")
        return st
    st.update(k_new=randn(B, n, nkv, hd), v_new=randn(B, n, nkv, hd))
    if case["kind"] == "turn":
        paths, counts = _paths(case, rng)
        st.update(path=torch.tensor(paths, dtype=torch.int32, device="cuda"),
                  accepted=torch.tensor(counts, dtype=torch.int32, device="cuda"))
    return st


# ---- plain forms: elementary torch operations in 32 bits --------------------------------

def _seen(S, window, sinks, device):
    i = torch.arange(S, device=device)[:, None]
    j = torch.arange(S, device=device)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def _heads(x, group):
    """[B, S, heads, hd] -> fp32 [B, heads * group, S, hd]."""
    return x.float().transpose(1, 2).repeat_interleave(group, dim=1)


def _plain_window(st):
    q, k, v, hd = st["q"], st["k"], st["v"], st["hd"]
    group, scale = st["nh"] // st["nkv"], st["hd"] ** -0.5
    seen = _seen(st["S"], st["window"], st["sinks"], q.device)
    qf, kf, vf = _heads(q, 1), _heads(k, group), _heads(v, group)
    s = (qf @ kf.transpose(2, 3)) * scale
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(dim=3, keepdim=True)
    e = torch.exp(s - m)
    total = e.sum(dim=3, keepdim=True)
    p = e / total
    o = p @ vf
    lse = (m + torch.log(total))[..., 0].transpose(1, 2).contiguous()
    out = o.transpose(1, 2).to(q.dtype)
    if st["kind"] == "fwd":
        return out, lse
    do = _heads(st["dO"], 1)
    dv = p.transpose(2, 3) @ do
    ds = p * (do @ vf.transpose(2, 3) - (do * o).sum(dim=3, keepdim=True))
    dq = (ds @ kf) * scale
    dk = (ds.transpose(2, 3) @ qf) * scale
    B, S, nkv = st["B"], st["S"], st["nkv"]
    dk = dk.view(B, nkv, group, S, hd).sum(dim=2)
    dv = dv.view(B, nkv, group, S, hd).sum(dim=2)
    return (out, lse, dq.transpose(1, 2).to(q.dtype), dk.transpose(1, 2).to(q.dtype), dv.transpose(1, 2).to(q.dtype))


def _plain_tree(st):
    q, table, lens = st["q"], st["table"], st["lens_t"].long()
    B, n, nkv, hd, page = (st[x] for x in ("B", "n", "nkv", "hd", "page"))
    group, T = st["nh"] // nkv, table.shape[1] * page
    there = (table >= 0).repeat_interleave(page, dim=1)
    k = st["k_pages"][table.clamp(min=0).long()].view(B, T, nkv, hd).float()
    v = st["v_pages"][table.clamp(min=0).long()].view(B, T, nkv, hd).float()
    bits = (st["words"][:, :, None] >> torch.arange(n, device=q.device)) & 1
    pos = lens[:, None] + (bits.sum(dim=2) - 1).clamp(min=0)
    p = torch.arange(T, device=q.device)
    at = (p[None, :] - lens[:, None]).clamp(0, n - 1)
    drafted = bits.gather(2, at[:, None, :].expand(B, n, T)).bool()
    drafted &= ((p[None, :] >= lens[:, None]) & (p[None, :] < lens[:, None] + n))[:, None, :]
    near = (pos[:, :, None] - p < st["window"]) | (p < st["sinks"])
    seen = (drafted | ((p[None, :] < lens[:, None])[:, None, :] & near)) & there[:, None, :]
    qf = q.float().view(B, n, nkv, group, hd).permute(0, 2, 3, 1, 4).reshape(B, nkv, group * n, hd)
    s = (qf @ k.permute(0, 2, 3, 1)) * hd ** -0.5
    s = s.view(B, nkv, group, n, T).masked_fill(~seen[:, None, None], -math.inf)
    m = s.amax(dim=4, keepdim=True).clamp(min=-1e30)
    e = torch.exp(s - m)
    total = e.sum(dim=4, keepdim=True)
    o = (e.view(B, nkv, group * n, T) @ v.transpose(1, 2)).view(B, nkv, group, n, hd) / total.clamp(min=1e-30)
    lse = m + torch.log(total)
    return (o.permute(0, 3, 1, 2, 4).reshape(B, n, st["nh"], hd).to(q.dtype),
            lse.permute(0, 3, 1, 2, 4).reshape(B, n, st["nh"]).contiguous())


def _rows(st, positions):
    """Rows of the flattened pools that hold the given positions [B, x]."""
    page = st["page"]
    return st["table"].long().gather(1, positions // page) * page + positions % page


def _plain_append(st):
    n, nkv, hd = st["n"], st["nkv"], st["hd"]
    at = st["lens_t"].long()[:, None] + torch.arange(n, device="cuda")
    rows = _rows(st, at).view(-1)
    st["k_pages"].view(-1, nkv, hd)[rows] = st["k_new"].view(-1, nkv, hd)
    st["v_pages"].view(-1, nkv, hd)[rows] = st["v_new"].view(-1, nkv, hd)
    return st["k_pages"], st["v_pages"]


def _plain_compact(st):
    n, nkv, hd = st["n"], st["nkv"], st["hd"]
    base, step = st["lens_t"].long()[:, None], torch.arange(n, device="cuda")
    kept = step[None, :] < st["accepted"][:, None]
    src = _rows(st, base + torch.where(kept, st["path"].long(), step)).view(-1)
    dst = _rows(st, base + step).view(-1)
    k, v = st["k_pages"].view(-1, nkv, hd), st["v_pages"].view(-1, nkv, hd)
    k[dst] = k[src]
    v[dst] = v[src]
    return st["k_pages"], st["v_pages"]


# ---- one pass ----------------------------------------------------------------------------

def run(state):
    st = state
    if not own:
        if st["kind"] in ("fwd", "step"):
            return _plain_window(st)
        if st["kind"] == "tree":
            return _plain_tree(st)
        out = _plain_append(st)
        return out if st["kind"] == "append" else _plain_compact(st)
    from bwd_xattn_fwd_gb300 import xattn
    if st["kind"] in ("fwd", "step"):
        o, lse = xattn.attention_window_fwd(st["q"], st["k"], st["v"], st["window"], st["sinks"])
        if st["kind"] == "fwd":
            return o, lse
        return (o, lse, *xattn.attention_window_bwd(st["q"], st["k"], st["v"], o, st["dO"], lse, st["window"],
                                                    st["sinks"]))
    if st["kind"] == "tree":
        return xattn.attention_tree_decode(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens_t"],
                                           tree=st["words"], window=st["window"], sinks=st["sinks"])
    xattn.cache_append(st["k_new"], st["v_new"], st["k_pages"], st["v_pages"], st["table"], st["lens_t"])
    if st["kind"] == "turn":
        xattn.cache_compact(st["k_pages"], st["v_pages"], st["table"], st["lens_t"], st["path"], st["accepted"])
    return st["k_pages"], st["v_pages"]


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    hd, nkv = case["hd"], case["nkv"]
    if case["kind"] in ("fwd", "step"):
        B, S, nh, W = case["B"], case["S"], case["nh"], case["window"]
        size = 4 if case["dtype"] == "f32" else 2
        pairs = sum(min(i + 1, W) + min(case["sinks"], max(0, i + 1 - W)) for i in range(S))
        qo, kv = B * S * nh * hd * size, B * S * nkv * hd * size
        if case["kind"] == "fwd":
            return {"bytes": 2 * qo + 2 * kv + 4 * B * S * nh, "flops": 4 * hd * pairs * B * nh}
        return {"bytes": 4 * qo + 4 * kv + 4 * B * S * nh, "flops": 14 * hd * pairs * B * nh}
    B, n = case["B"], case["n"]
    if case["kind"] == "tree":
        W = case["window"]
        seen = sum(min(c, W) + min(case["sinks"], max(0, c - W)) + n for c in _ctx_lens(case))
        return {"bytes": 4 * seen * nkv * hd + 4 * B * n * case["nh"] * hd + 4 * B * n * case["nh"],
                "flops": 4 * hd * seen * n * case["nh"]}
    rows = 2 * 2 * B * n * nkv * hd * 2      # K and V, read and written
    return {"bytes": rows if case["kind"] == "append" else int(1.25 * rows), "flops": 0}


# ---- the definitions in 64 bits ----------------------------------------------------------

def exact(case, seed):
    if case["kind"] in ("append", "turn"):
        return None                            # copies: nothing is computed
    st = prepare(case, seed)
    scale = 1.0 / math.sqrt(case["hd"])
    group = case["nh"] // case["nkv"]
    if case["kind"] == "tree":
        return _exact_tree(case, st, scale, group)
    names = ("q", "k", "v")
    leaf = {x: st[x].double().requires_grad_(case["kind"] == "step") for x in names}
    S = case["S"]
    hidden = torch.ones(S, S, dtype=torch.bool, device="cuda").triu(1)
    far = torch.ones(S, S, dtype=torch.bool, device="cuda").tril(-case["window"])
    far[:, :case["sinks"]] = False
    hidden |= far
    outs, lses = [], []
    for b in range(case["B"]):
        k = torch.stack([leaf["k"][b, :, h // group] for h in range(case["nh"])])
        v = torch.stack([leaf["v"][b, :, h // group] for h in range(case["nh"])])
        s = torch.einsum("ihd,hjd->hij", leaf["q"][b], k).mul(scale).masked_fill(hidden, -math.inf)
        lse = torch.logsumexp(s, dim=2)
        outs.append(torch.einsum("hij,hjd->ihd", torch.softmax(s, dim=2), v))
        lses.append(lse.detach().transpose(0, 1))
        if case["kind"] == "step":
            (outs[-1] * st["dO"][b].double()).sum().backward()
            outs[-1] = outs[-1].detach()
    o, lse = torch.stack(outs), torch.stack(lses)
    if case["kind"] == "fwd":
        return o, lse
    return (o, lse, *(leaf[x].grad for x in names))


def _exact_tree(case, st, scale, group):
    B, n, nh, nkv, hd, page = (case[x] for x in ("B", "n", "nh", "nkv", "hd", "page"))
    o = torch.zeros(B, n, nh, hd, dtype=torch.float64, device="cuda")
    lse = torch.full((B, n, nh), -math.inf, dtype=torch.float64, device="cuda")
    table, words = st["table"].tolist(), st["words"].tolist()
    for b, c in enumerate(_ctx_lens(case)):
        places = [p for p in range(c + n) if table[b][p // page] >= 0]
        rows = torch.tensor([table[b][p // page] * page + p % page for p in places], device="cuda")
        p = torch.tensor(places, device="cuda")
        depth = [bin(w & (2**64 - 1)).count("1") - 1 for w in words[b]]
        seen = torch.stack([torch.where(p < c, (c + depth[i] - p < case["window"]) | (p < case["sinks"]),
                                        ((words[b][i] >> (p - c).clamp(0, 63)) & 1).bool()) for i in range(n)])
        k = st["k_pages"].view(-1, nkv, hd)[rows].double()
        v = st["v_pages"].view(-1, nkv, hd)[rows].double()
        q = st["q"][b].double().view(n, nkv, group, hd)
        s = torch.einsum("ikgd,pkd->kgip", q, k).mul(scale).masked_fill(~seen, -math.inf)
        lse[b] = torch.logsumexp(s, dim=3).permute(2, 0, 1).reshape(n, nh)
        o[b] = torch.einsum("kgip,pkd->ikgd", torch.softmax(s, dim=3), v).reshape(n, nh, hd)
    return o, lse
