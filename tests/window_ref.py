"""Window attention with sinks in 64 bits, straight from its definition, with elementwise
error bounds for a computation that rounds where the library does.

Query i sees key j when j <= i and (i - j < window or j < sinks). Bounds (u = half a step of
the output type, relative: 2^-8 for bf16, and P and dS are rounded to bf16 too; t = slack for
the fp32 arithmetic: exponentials within 8e-5, and scores accumulated in fp32):
  o   : u |o| + (u + t) sum_j P |v|
  dv  : u |dv| + (u + t) sum_i P |dO|
  dS  : (2 u + t) |dS| + P E, where E_i = (2 u + t) sum_d |dO| (P |v|) bounds the error of
        D_i = dO_i . o_i (o is rounded, and carries P's rounding)
  dq  : u |dq| + scale sum_j err(dS) |k|;   dk : the same over i with |q|
In fp32 mode u is 0 and t covers sums of `n` terms, each off by at most n 2^-24 relative.
"""
import torch


def seen(S, window, sinks, device):
    i = torch.arange(S, device=device)[:, None]
    j = torch.arange(S, device=device)[None, :]
    return (j <= i) & ((i - j < window) | (j < sinks))


def reference(x, window, sinks, scale, bf16):
    """dict name -> (value, bound) in float64 for q, k, v, dO of x ([B,S,heads,hd])."""
    q, k, v, dO = (x[n].double() for n in ("q", "k", "v", "dO"))
    B, S, nh, hd = q.shape
    nkv = k.shape[2]
    group = nh // nkv
    qh, doh = q.transpose(1, 2), dO.transpose(1, 2)
    kh, vh = (t.transpose(1, 2).repeat_interleave(group, 1) for t in (k, v))
    vis = seen(S, window, sinks, q.device)
    s = (qh @ kh.transpose(2, 3)) * scale
    lse = torch.logsumexp(s.masked_fill(~vis, float("-inf")), dim=3)
    p = torch.exp(s - lse[..., None]).masked_fill(~vis, 0.0)
    o = p @ vh
    ds = p * (doh @ vh.transpose(2, 3) - (doh * o).sum(3, keepdim=True))
    # fp32 slack: the scores' sums (hd terms, each step 2^-23 allowed for) and the exponentials
    s_err = 2.0 ** -23 * hd * float((qh.abs() @ kh.abs().transpose(2, 3)).max()) * abs(scale)
    if bf16:
        u, t = 2.0 ** -8, 2.0 ** -11 + 2 * s_err
        lse_tol = 8e-5 + 2 * s_err + 2.0 ** -20 * float(lse.abs().max())
    else:
        u, t = 0.0, 2.0 ** -24 * (2 * hd + 4 * S * group + 64) + 2 * s_err
        lse_tol = t + 2.0 ** -20 * float(lse.abs().max())
    pv = p @ vh.abs()
    e = (2 * u + t) * (doh.abs() * pv).sum(3, keepdim=True)
    ds_err = (2 * u + t) * ds.abs() + t * p * ((doh.abs() @ vh.abs().transpose(2, 3)) + e) + p * e

    def kv(z):
        return z.view(B, nkv, group, S, hd).sum(2)

    dq, dk, dv = (ds @ kh) * scale, kv(ds.transpose(2, 3) @ qh) * scale, kv(p.transpose(2, 3) @ doh)
    a = abs(scale)
    out = {
        "o": (o, u * o.abs() + (u + t) * pv),
        "dq": (dq, u * dq.abs() + a * (ds_err @ kh.abs())),
        "dk": (dk, u * dk.abs() + a * kv(ds_err.transpose(2, 3) @ qh.abs())),
        "dv": (dv, u * dv.abs() + (u + t) * kv(p.transpose(2, 3) @ doh.abs())),
    }
    out = {n: (val.transpose(1, 2), err.transpose(1, 2) * (1 + 2.0 ** -6) + 1e-30) for n, (val, err) in out.items()}
    out["lse"] = (lse.transpose(1, 2), torch.full_like(lse.transpose(1, 2), lse_tol))
    return out


def check(got, ref, label):
    """Every element of every output of `got` within its bound."""
    for name, t in got.items():
        val, err = ref[name]
        t = t.double()
        assert bool(torch.isfinite(t).all()), f"{label} {name}: not finite"
        over = ((t - val).abs() / err).max()
        assert float(over) <= 1.0, f"{label} {name}: {float(over):.3f} of its bound"
