"""fp64 reference of sliding-window attention with sinks, and element-wise
bounds of what the kernels may be off by.

u is half a step of the tensors' type (2^-8 in bf16, 2^-24 in fp32), e = 2^-24.

bf16 kernels: scores, sums and statistics are fp32 (the tensor cores' sums round
toward zero, 2 e a term); P and dS are rounded to bf16 for the second products,
outputs once.  A score is off by at most ds = 2 d e scale sum|q k|, so a
probability, formed with ex2.approx (2^-22) against an fp32 sum of at most N
terms, by the factor f = 2 ds + 2^-19.
   O:   u |O| + (u + f) sum P|v|
   lse: ds + 2^-18 (1 + |lse|)
   dV:  u |dV| + (u + f) sum P|dO|
   dS:  the rounding of P and its own, 2 u + f of |dS|, and P times what dP - D is
        off by: 2 d e sum|dO v|, and D = <dO, O> as O is off: sum |dO| err(O)
   dQ, dK: u of the value, plus scale sum err(dS) |k| or |q|, plus the fp32 sums.
fp32 kernels: the same with P and dS unrounded and d e for the products.
"""
import torch

E = 2.0 ** -24


def allowed(N, window, sinks, cu, device="cuda"):
    i = torch.arange(N, device=device)
    ends = torch.tensor((cu or [0, N])[1:], device=device)
    starts = torch.tensor((cu or [0, N])[:-1], device=device)
    start = starts[torch.searchsorted(ends, i, right=True)]
    i, j, s = i[:, None], i[None], start[:, None]
    return (j >= s) & (j <= i) & ((i - j < window) | (j - s < sinks))


def grouped(t, Hkv):  # [S][B][N][H][d] -> [S][B][Hkv][G][N][d], fp64
    S, B, N, H, d = t.shape
    return t.cuda().double().view(S, B, N, Hkv, H // Hkv, d).permute(0, 1, 3, 4, 2, 5)


def ungrouped(t):
    S, B, Hkv, G, N, d = t.shape
    return t.permute(0, 1, 4, 2, 3, 5).reshape(S, B, N, Hkv * G, d)


def reference(q, k, v, dout, mask, scale, rounded):
    """Values {o, lse, dq, dk, dv} and the bounds of their errors."""
    Hkv, d, N = k.shape[3], q.shape[4], k.shape[2]
    q, dout = grouped(q, Hkv), grouped(dout, Hkv)
    k, v = (grouped(t, Hkv) for t in (k, v))
    unit = 2.0 ** -8 if rounded else E
    step = 2 if rounded else 1
    kT, vT = k.transpose(-1, -2), v.transpose(-1, -2)
    s = (q @ kT * scale).masked_fill(~mask, -torch.inf)
    lse = s.logsumexp(-1, keepdim=True)
    p = (s - lse).exp()
    o = p @ v
    ds_err = (step * d * E * scale * (q.abs() @ kT.abs())).masked_fill(~mask, 0).amax(-1, keepdim=True)
    f = 2 * ds_err + (2.0 ** -19 if rounded else (N + 64) * E)
    second = unit if rounded else (N + 64) * E  # P's rounding, or the second product's sum
    err = {"o": unit * o.abs() + (second + f) * (p @ v.abs()), "lse": ds_err + 2.0 ** -18 * (1 + lse.abs())
           if rounded else ds_err + (N + 64) * E * (1 + lse.abs())}
    dp = dout @ vT
    D = (dout * o).sum(-1, keepdim=True)
    ds = p * (dp - D)
    D_err = (dout.abs() * (err["o"] + d * E * o.abs())).sum(-1, keepdim=True)
    wrong = (2 * unit if rounded else (N + 64) * E) + f
    dS_err = wrong * ds.abs() + p * (step * d * E * (dout.abs() @ vT.abs()) + D_err)
    pT, sT = p.transpose(-1, -2), ds.transpose(-1, -2)
    sums = (N + 64) * step * E  # the products' fp32 sums over rows and heads
    group = lambda t: t.sum(3, keepdim=True)
    val = {"o": o, "lse": lse, "dq": ds @ k * scale, "dk": group(sT @ q) * scale, "dv": group(pT @ dout)}
    err["dq"] = unit * val["dq"].abs() + scale * ((dS_err + sums * ds.abs()) @ k.abs())
    eT = (dS_err + sums * ds.abs()).transpose(-1, -2)
    err["dk"] = unit * val["dk"].abs() + scale * group(eT @ q.abs())
    err["dv"] = unit * val["dv"].abs() + group(((second + f + sums) * p).transpose(-1, -2) @ dout.abs())
    for t in (val, err):
        for n in t:
            t[n] = t[n][..., 0].flatten(2, 3) if n == "lse" else ungrouped(t[n])
    return val, err


def check(name, got, val, err):
    got = got.double()
    assert got.shape == val.shape, name
    off = (got - val).abs() - err
    assert not torch.isnan(off).any(), f"{name}: not a number"
    assert off.max() <= 0, f"{name}: {off.max().item()} beyond its bound ({(off > 0).sum().item()} values)"
    size = val.norm()
    return float((got - val).norm() / size) if size > 0 else 0.0
