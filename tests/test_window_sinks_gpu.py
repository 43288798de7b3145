"""The sinks' gradients under a sliding window in bf16: many sinks, documents that
share tiles with theirs, and their accuracy over walks of tens of thousands of rows."""
import math

import pytest
import torch

from test_window_attn_gpu import inputs, run
from window_ref import allowed, check, reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

CASES = [
    # S, B, N, Hq, Hkv, window, sinks, documents
    (1, 1, 900, 2, 1, 40, 16, None),
    (1, 1, 900, 2, 1, 40, 17, None),
    (2, 1, 1025, 4, 2, 1, 64, None),
    (1, 1, 1100, 2, 1, 130, 65, None),
    (1, 1, 8400, 2, 1, 100, 65, None),                  # many sinks apart
    (1, 1, 9100, 1, 1, 20, 70, [0, 127, 4000, 4100, 9100]),
    (1, 1, 25700, 1, 1, 1, 200, None),
    (1, 1, 2600, 2, 1, 100, 300, None),
    (2, 1, 1400, 4, 2, 1, 512, None),
    (1, 1, 1400, 2, 1, 1, 513, None),
    (1, 1, 2500, 3, 1, 20, 130, [0, 127, 900, 1000, 2500]),  # sinks across three tiles
    (1, 2, 1800, 2, 2, 3, 400, [0, 60, 500, 1300, 1310, 1800]),
    (1, 2, 1500, 3, 1, 20, 33, [0, 120, 700, 760, 1500]),   # sinks across two tiles
    (1, 1, 1000, 1, 1, 1, 3, [0, 300, 301, 303, 640, 1000]),
    (1, 1, 700, 2, 2, 10, 64, [0, 100, 300, 400, 700]),     # a second tile of sinks that another document ends
    (1, 1, 513, 2, 1, 1, 64, [0, 127, 256, 380, 513]),
    (1, 1, 400, 2, 1, 5, 40, [0, 30, 390, 400]),        # fewer keys than sinks
    (1, 1, 900, 3, 1, 33, 160, None),                   # 32 behind a whole tile
    (1, 1, 900, 2, 1, 300, 161, None),
    (1, 2, 1300, 3, 1, 7, 140, [0, 90, 700, 1300]),     # sinks that end at key 230 and 840
    (1, 1, 1000, 2, 1, 128, 40, [0, 100, 1000]),
    # enough tiles for the forward to take single heads' rows two tiles at a time
    (4, 1, 1300, 8, 8, 200, 3, None),
    (4, 1, 1153, 8, 8, 1, 0, None),
    (2, 2, 1400, 6, 2, 130, 140, None),
    (4, 1, 1200, 6, 2, 90, 30, [0, 1, 130, 300, 310, 700, 1100, 1200]),
    (2, 2, 1290, 5, 5, 2000, 0, [0, 128, 640, 650, 1290]),
    (5, 1, 1030, 3, 1, 17, 300, [0, 500, 1030]),
]


@pytest.mark.parametrize("S,B,N,Hq,Hkv,window,sinks,cu", CASES)
def test_against_reference(uly, S, B, N, Hq, Hkv, window, sinks, cu):
    q, k, v, dout = inputs(S, B, N, Hq, Hkv, 128, BF16, seed=5)
    val, err = reference(q, k, v, dout, allowed(N, window, sinks, cu), 1 / math.sqrt(128), True)
    got = run(uly, q, k, v, dout, window, sinks, cu)
    for n in val:
        check(n, got[n], val[n], err[n])


def sink_sums(q, k, v, dout, window, start, end, sinks):
    """fp64 dK and dV of a document's first keys, what the kernel may be off by, and dV with
    P rounded to bf16.

    P and dS enter in two bf16 parts (2^-16 of a term), their scores and statistics
    are a few steps of fp32 off; together less than e = 2^-13 of a term, rows apart.  An
    fp32 sum of at most 400 additions, each of which rounds the partial sum of terms of
    both signs, adds less than 400 * 2^-23 < e.  Six standard deviations of a sum of
    independent errors of at most e |x_i| are at most 6 e sqrt(sum x_i^2).  D = <dO, O>
    takes O as stored: half a step u = 2^-8 of each of its elements, independent, so
    that dS_i is off by P_i times u sqrt(sum_c (dO_c O_c)^2).  u of the value at the end.
    """
    e, u, scale = 2.0 ** -13, 2.0 ** -8, 1 / math.sqrt(128)
    G = q.shape[3] // k.shape[3]
    rep = lambda t: t.repeat_interleave(G, 2)[0].double()  # [rows][Hq][d]
    out = {n: 0.0 for n in ("dk", "dv", "dk2", "dv2", "D2", "one")}
    fold = lambda t: t.unflatten(0, (-1, G)).sum(1)
    for r0 in range(start, end, 1024):
        r1 = min(r0 + 1024, end)
        lo = max(start, r0 - window + 1)
        head = min(start + sinks, lo)
        keys = torch.cat([torch.arange(start, head, device="cuda"), torch.arange(lo, r1, device="cuda")])
        i, j = torch.arange(r0, r1, device="cuda")[:, None], keys[None]
        mask = (j <= i) & ((i - j < window) | (j - start < sinks))
        qq, dd = q[0, 0, r0:r1].double().transpose(0, 1), dout[0, 0, r0:r1].double().transpose(0, 1)  # [Hq][rows][d]
        kk, vv = (rep(t[0, :, keys]).transpose(0, 1) for t in (k, v))
        p = (qq @ kk.transpose(1, 2) * scale).masked_fill(~mask, -math.inf).softmax(-1)
        o, dp = p @ vv, dd @ vv.transpose(1, 2)
        ds = p * (dp - (dd * o).sum(-1, keepdim=True))
        n = int((keys < start + sinks).sum())
        p, ds = p[..., :n].transpose(1, 2), ds[..., :n].transpose(1, 2)  # [Hq][sinks][rows]
        D = (dd * o).square().sum(-1)[:, None] * u * u
        for name, x in (("dk", ds @ qq), ("dv", p @ dd), ("dk2", ds.square() @ qq.square()),
                        ("dv2", p.square() @ dd.square()), ("D2", (p.square() * D) @ qq.square()),
                        ("one", p.to(BF16).double() @ dd)):
            x = fold(x)
            if n < sinks:  # the block of the document's first rows has them all, if it has that many
                x = torch.nn.functional.pad(x, (0, 0, 0, sinks - n))
            out[name] = out[name] + x
    dk, dv = out["dk"] * scale, out["dv"]
    dk_err = u * dk.abs() + 6 * scale * (2 * e * out["dk2"].sqrt() + out["D2"].sqrt())
    return dk, dv, dk_err, u * dv.abs() + 12 * e * out["dv2"].sqrt(), out["one"]


@pytest.mark.parametrize("window,sinks,cu", [(256, 4, None), (30, 1, None), (2000, 40, [0, 17, 9000, 9050, 24000]),
                                             (300, 130, None)])
def test_long_walks_keep_their_precision(uly, window, sinks, cu):
    """Queries share a direction that the sinks answer to, as trained ones do."""
    N, Hq, Hkv = 24000, 4, 2
    q, k, v, dout = inputs(1, 1, N, Hq, Hkv, 128, BF16, seed=11)
    shared = torch.randn(Hkv, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) / 2
    q = (q.float() + shared.repeat_interleave(Hq // Hkv, 0)).to(BF16)
    k = k.float()
    for a in (cu or [0, N])[:-1]:
        k[:, :, a:a + sinks] += shared
    k = k.to(BF16)
    got = run(uly, q, k, v, dout, window, sinks, cu)
    for a, b in zip((cu or [0, N])[:-1], (cu or [0, N])[1:]):
        if b - a > window:
            dk, dv, dk_err, dv_err, one = sink_sums(q, k, v, dout, window, a, b, sinks)
            assert ((one - dv).abs() > dv_err).any()  # one part would not do
            for name, want, err in (("dk", dk, dk_err), ("dv", dv, dv_err)):
                off = (got[name][0, 0, a:a + sinks].double().transpose(0, 1) - want).abs()
                print(name, a, float((off / err).max()))
                assert (off <= err).all(), (name, a, float((off / err).max()))
