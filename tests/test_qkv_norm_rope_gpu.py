"""Norm, rotation and move of Q, K and V on the GPU against the fp64 oracle.

Tolerances count roundings.  u = 2^-24.  The rounding of a result to its type
is off by at most eps/2 of its value.  Before it, in fp32: the mean of squares
(at most d/16 + 8 sequential additions and products), its root and quotient,
two products, the sine and cosine (the angle is held to 2^-25 half turns, so
they are off by pi 2^-25 < 1.6 u, plus 2 units of their last place) and two
products and a sum: below 32 u of the pair's length.  The backward adds the
mean of w * g * xhat (again d/16 + 8 additions) on both sides: 64 u of the
terms' sizes.  dw is a sum over R rows: at most (R + 64) u of the sum of the
absolute terms.
"""
import numpy as np
import pytest
import torch

import oracle.norm_rope as nr
from parity_utils import Guards, bytes_equal, log_errors

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6
BF16, FP32 = torch.bfloat16, torch.float32


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def make(P, B, N, Hq, Hkv, d, dtype, rot, axes=1, packed=False, to_head=True, positions="none", norm=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    Np = N // P
    rand = lambda *s: torch.randn(*s, generator=g)
    x = (rand(P, B, Np, Hq + 2 * Hkv, d) * (0.1 + 3 * torch.rand(Hq + 2 * Hkv, 1, generator=g))).to(dtype)
    w = [(1 + 0.3 * rand(d)).to(dtype) for _ in range(2)] if norm else [None, None]
    far = lambda H: (P, B, N, H // P, d) if to_head else (P, B, Np, H, d)
    dy = [rand(*far(H)).to(dtype) for H in (Hq, Hkv, Hkv)]
    pos = None
    if positions == "far":
        pos = torch.randint(-2_000_000, 2_000_000, (axes, P, B, Np), generator=g)
    elif positions == "docs":
        pos = torch.randint(0, 50, (axes, P, B, Np), generator=g)
    half = rot // 2
    inv = 1e4 ** (-np.arange(half) / max(half, 1))
    axis = np.arange(half) % axes if axes > 1 else None
    return dict(x=x, w=w, dy=dy, pos=pos, inv=inv, axis=axis, heads=(Hq, Hkv), packed=packed, to_head=to_head, P=P)


def split(c, x):
    Hq, Hkv = c["heads"]
    parts = x.split([Hq, Hkv, Hkv], dim=3)
    return list(parts) if c["packed"] else [p.contiguous() for p in parts]


def to_seq(y, P):
    """Head layout -> sequence layout, numpy."""
    _, B, N, Hp, d = y.shape
    return y.reshape(P, B, P, N // P, Hp, d).transpose(2, 1, 3, 0, 4, 5).reshape(P, B, N // P, P * Hp, d)


def oracle_angles(c):
    P, B, Np = c["x"].shape[:3]
    pos = c["pos"]
    if pos is None:
        pos = torch.arange(P * Np).view(1, P, 1, Np).expand(1, P, B, Np)
        if c["axis"] is not None:
            pos = pos.expand(int(c["axis"].max()) + 1, P, B, Np)
    return nr.angles(pos.numpy(), c["inv"], c["axis"])


def kwargs(c, inter):
    cu = lambda t: None if t is None else t.cuda()
    pos = c["pos"]
    if pos is not None and pos.shape[0] == 1:
        pos = pos[0]
    return dict(inv_freq=c["inv"], q_weight=cu(c["w"][0]), k_weight=cu(c["w"][1]), positions=cu(pos),
                axis_of_freq=c["axis"], interleaved=inter, eps=EPS, to_head=c["to_head"])


def pair_size(x, t, inter):
    """The length of the pair each value belongs to (its own size if it does not turn)."""
    rot = 2 * t.shape[-1]
    a, b = nr._pairs(rot, inter)
    s = np.abs(x).copy()
    s[..., a] = s[..., b] = np.hypot(x[..., a], x[..., b])
    return s


def check(got, ref, tol, what):
    got = got.detach().cpu().double().numpy()
    assert np.isfinite(got).all(), what
    over = np.abs(got - ref) - tol
    assert (over <= 0).all(), (what, float(over.max()), np.unravel_index(over.argmax(), over.shape))
    log_errors(what, worst=float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()))


def run_fwd(uly, c, inter, g=None, **more):
    g = g or Guards()
    x = split(c, c["x"].cuda())
    y = [g.empty(t.shape, t.dtype, float("nan")) for t in c["dy"]]
    uly.ulysses_qkv_norm_rope_fwd(*x, *y, c["P"], **{**kwargs(c, inter), **more})
    return x, y, g


CASES = [
    # P, B, N, Hq, Hkv, d, dtype, rot, axes, inter, packed, to_head, positions, norm
    (1, 1, 1, 1, 1, 128, BF16, 128, 1, False, False, True, "none", True),       # one token, one head
    (1, 3, 1, 32, 8, 128, BF16, 128, 1, False, True, False, "far", True),       # a new token of three sequences
    (4, 1, 64, 8, 4, 128, BF16, 128, 1, False, True, True, "none", True),
    (2, 2, 34, 6, 2, 128, BF16, 64, 3, False, False, True, "docs", True),       # half a head turns, three axes
    (3, 1, 33, 9, 3, 64, BF16, 64, 1, True, True, True, "far", True),           # interleaved pairs
    (2, 1, 10, 4, 4, 64, BF16, 16, 2, True, False, False, "far", True),
    (4, 2, 64, 8, 4, 128, FP32, 128, 1, False, True, True, "far", True),
    (1, 1, 257, 5, 1, 64, FP32, 32, 3, False, False, False, "far", True),       # odd heads, odd tokens
    (2, 3, 14, 4, 2, 128, FP32, 48, 1, True, True, True, "docs", True),
    (2, 1, 50, 4, 2, 128, BF16, 128, 1, False, False, True, "far", False),      # rotation alone
    (2, 1, 50, 4, 2, 64, FP32, 64, 8, True, True, False, "far", False),
    (1, 1, 9, 3, 3, 128, BF16, 0, 1, False, False, True, "none", True),         # norm alone
    (8, 1, 4096, 8, 8, 64, BF16, 64, 1, False, True, True, "docs", True),       # many tokens a warp
    (3, 1, 3999, 3, 3, 128, FP32, 128, 3, False, True, True, "docs", True),
]


def _unpack(case):
    P, B, N, Hq, Hkv, d, dtype, rot, axes, inter, packed, to_head, positions, norm = case
    return make(P, B, N, Hq, Hkv, d, dtype, rot, axes, packed, to_head, positions, norm, seed=N + rot), inter


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(uly, case):
    c, inter = _unpack(case)
    x, y, g = run_fwd(uly, c, inter)
    g.check()
    t = oracle_angles(c)
    for i, name in enumerate("qk"):
        x64 = x[i].cpu().double().numpy()
        w = None if c["w"][i] is None else c["w"][i].double().numpy()
        ref = nr.norm_rope(x64, w, t, inter, EPS)
        before = nr.rotate(ref, t, inter, back=True)
        tol = _half(c["x"].dtype) * np.abs(ref) + 32 * U * pair_size(before, t, inter)
        got = y[i].cpu()
        if c["to_head"]:
            got = torch.from_numpy(to_seq(got.double().numpy(), c["P"]))
        check(got, ref, tol, f"norm_rope fwd {name} {case}")
    v = split(c, c["x"])[2].contiguous()
    if c["to_head"]:
        vh = torch.empty_like(y[2])
        if v.shape[2] * c["P"] > 0:
            uly.ulysses_seq_to_head(v.cuda(), vh, c["P"])
        assert bytes_equal(y[2], vh)
    else:
        assert bytes_equal(y[2], v)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(uly, case):
    c, inter = _unpack(case)
    dtype, P = c["x"].dtype, c["P"]
    g = Guards()
    x = split(c, c["x"].cuda())
    dx = split(c, g.empty(c["x"].shape, dtype, float("nan")))
    if not c["packed"]:
        dx = [g.empty(t.shape, dtype, float("nan")) for t in dx]
    norm = c["w"][0] is not None
    dw = [g.empty(w.shape, dtype, float("nan")) for w in c["w"]] if norm else [None, None]
    ws = g.workspace(uly.ulysses_qkv_norm_rope_workspace_size(c["x"].shape[-1]))
    ws.fill_(0xFF)  # NaN where nothing is written
    uly.ulysses_qkv_norm_rope_bwd(*x[:2], *[t.cuda() for t in c["dy"]], *dx, P, **kwargs(c, inter),
                                  dq_weight=dw[0], dk_weight=dw[1], workspace=ws)
    g.check()
    t = oracle_angles(c)
    for i, name in enumerate("qk"):
        x64 = x[i].cpu().double().numpy()
        dy = c["dy"][i].double().numpy()
        dy = to_seq(dy, P) if c["to_head"] else dy
        w = c["w"][i].double().numpy() if norm else None
        ref, refw = nr.norm_rope_bwd(x64, w, t, dy, inter, EPS)
        turned = pair_size(dy, t, inter)
        size = turned
        if norm:
            r = 1 / np.sqrt((x64 * x64).mean(-1, keepdims=True) + EPS)
            xhat = np.abs(x64) * r
            size = r * (np.abs(w) * turned + xhat * (np.abs(w) * turned * xhat).mean(-1, keepdims=True))
            terms = (turned * xhat).reshape(-1, x64.shape[-1])
            tolw = _half(dtype) * np.abs(refw) + (terms.shape[0] + 64) * U * terms.sum(0)
            check(dw[i], refw, tolw, f"norm_rope bwd dw{name} {case}")
        check(dx[i], ref, _half(dtype) * np.abs(ref) + 64 * U * size, f"norm_rope bwd {name} {case}")
    dv = c["dy"][2]
    if c["to_head"]:
        dv = torch.from_numpy(to_seq(dv.float().numpy(), P)).to(dtype)
    assert bytes_equal(dx[2], dv)


def test_head_layout_is_the_sequence_layout_swapped(uly):
    """to_head only moves: bit for bit the sequence-layout result through ulysses_seq_to_head."""
    c = make(4, 2, 48, 8, 4, 128, BF16, 128, packed=True, positions="far")
    _, yh, _ = run_fwd(uly, c, False)
    x = split(c, c["x"].cuda())
    ys = [torch.empty(t.shape, dtype=BF16, device="cuda") for t in x]
    uly.ulysses_qkv_norm_rope_fwd(*x, *ys, 4, **{**kwargs(c, False), "to_head": False})
    for s, h in zip(ys, yh):
        want = torch.empty_like(h)
        uly.ulysses_seq_to_head(s, want, 4)
        assert bytes_equal(h, want)


def test_without_v_q_and_k_are_unchanged(uly):
    c = make(2, 1, 20, 4, 2, 64, BF16, 64, positions="docs")
    x, y, _ = run_fwd(uly, c, False)
    y2 = [torch.empty_like(t) for t in y[:2]]
    uly.ulysses_qkv_norm_rope_fwd(*x[:2], None, *y2, None, 2, **kwargs(c, False))
    assert bytes_equal(y[0], y2[0]) and bytes_equal(y[1], y2[1])
    dy = [t.cuda() for t in c["dy"]]
    one, two = [[torch.empty_like(t) for t in x] for _ in range(2)]
    uly.ulysses_qkv_norm_rope_bwd(*x[:2], *dy, *one, 2, **kwargs(c, False))
    uly.ulysses_qkv_norm_rope_bwd(*x[:2], *dy[:2], None, *two[:2], None, 2, **kwargs(c, False))
    assert bytes_equal(one[0], two[0]) and bytes_equal(one[1], two[1])


def test_zero_nan_and_infinite_rows_stay_in_their_rows(uly):
    c = make(1, 1, 6, 4, 2, 128, BF16, 128)
    clean = run_fwd(uly, c, False)[1]
    c["x"][0, 0, 1, 0] = 0.0
    c["x"][0, 0, 2, 1, 5] = float("nan")
    c["x"][0, 0, 3, 5] = float("inf")  # a K head
    _, y, _ = run_fwd(uly, c, False)
    torch.cuda.synchronize()
    assert float(y[0][0, 0, 1, 0].float().abs().max()) == 0.0
    assert torch.isnan(y[0][0, 0, 2, 1].float()).all()
    assert torch.isnan(y[1][0, 0, 3, 1].float()).any()
    for i, bad in ((0, [(1, 0), (2, 1)]), (1, [(3, 1)])):
        a, b = clean[i].clone(), y[i].clone()
        for n, h in bad:
            a[0, 0, n, h] = b[0, 0, n, h] = 0
        assert bytes_equal(a, b)


@pytest.mark.parametrize("inter", [False, True])
def test_values_that_do_not_turn_are_copied(uly, inter):
    """Without a norm, values from rot_dim on are untouched, whatever stands
    beside them (compared as values: a conversion to bf16 has one NaN, so a
    NaN's payload bits do not come back)."""
    same = lambda a, b: torch.equal(torch.isnan(a.cpu()), torch.isnan(b)) and bytes_equal(
        a.cpu().masked_fill(torch.isnan(a.cpu()), 0), b.masked_fill(torch.isnan(b), 0))
    c = make(1, 1, 4, 2, 2, 128, BF16, 32, norm=False, positions="far")
    c["x"][..., 40] = float("inf")
    c["x"][..., 100] = float("nan")
    _, y, _ = run_fwd(uly, c, inter)
    x = split(c, c["x"])
    for i in range(2):
        assert same(y[i].reshape(x[i].shape)[..., 32:], x[i][..., 32:])
        assert torch.isfinite(y[i][..., :32].float()).all()
    dx = [torch.empty_like(t, device="cuda") for t in x]
    dy = [t.cuda().reshape(d.shape) for t, d in zip(x, c["dy"])]
    uly.ulysses_qkv_norm_rope_bwd(None, None, *dy, *dx, 1, **kwargs(c, inter))
    for i in range(2):
        assert same(dx[i][..., 32:], x[i][..., 32:])
        assert torch.isfinite(dx[i][..., :32].float()).all()


def test_weight_gradients_are_the_same_on_every_run(uly):
    c = make(2, 1, 3000, 8, 2, 128, BF16, 128)
    x = split(c, c["x"].cuda())
    dy = [t.cuda() for t in c["dy"]]
    got = []
    for _ in range(3):
        dx = [torch.empty_like(t) for t in x]
        dw = [torch.empty(128, dtype=BF16, device="cuda") for _ in range(2)]
        uly.ulysses_qkv_norm_rope_bwd(*x[:2], *dy, *dx, 2, **kwargs(c, False), dq_weight=dw[0], dk_weight=dw[1])
        got.append(dx + dw)
    for other in got[1:]:
        assert all(bytes_equal(a, b) for a, b in zip(got[0], other))
    # one of the two weight gradients alone
    dk = torch.empty(128, dtype=BF16, device="cuda")
    uly.ulysses_qkv_norm_rope_bwd(*x[:2], *dy, *[torch.empty_like(t) for t in x], 2, **kwargs(c, False), dk_weight=dk)
    assert bytes_equal(dk, got[0][4])


def test_captured_and_on_another_stream(uly):
    """Forward and backward on a side stream, then captured into a graph and replayed on new inputs."""
    c = make(2, 1, 40, 4, 2, 128, BF16, 128, positions="docs")
    x, y, _ = run_fwd(uly, c, False)
    dy = [t.cuda() for t in c["dy"]]
    kw = kwargs(c, False)
    want = [torch.empty_like(t) for t in x]
    wantw = [torch.empty(128, dtype=BF16, device="cuda") for _ in range(2)]
    uly.ulysses_qkv_norm_rope_bwd(*x[:2], *dy, *want, 2, **kw, dq_weight=wantw[0], dk_weight=wantw[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, dx2 = [torch.empty_like(t) for t in y], [torch.empty_like(t) for t in x]
    dw2 = [torch.empty_like(t) for t in wantw]
    uly.ulysses_qkv_norm_rope_fwd(*x, *y2, 2, **kw, stream=side)
    uly.ulysses_qkv_norm_rope_bwd(*x[:2], *dy, *dx2, 2, **kw, dq_weight=dw2[0], dk_weight=dw2[1], stream=side)
    side.synchronize()
    assert all(bytes_equal(a, b) for a, b in zip(y + want + wantw, y2 + dx2 + dw2))
    ws = torch.empty(uly.ulysses_qkv_norm_rope_workspace_size(128), dtype=torch.uint8, device="cuda")
    held = [torch.zeros_like(t) for t in x]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uly.ulysses_qkv_norm_rope_fwd(*held, *y2, 2, **kw)
        uly.ulysses_qkv_norm_rope_bwd(*held[:2], *dy, *dx2, 2, **kw, dq_weight=dw2[0], dk_weight=dw2[1], workspace=ws)
    for t, s in zip(held, x):
        t.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert all(bytes_equal(a, b) for a, b in zip(y + want + wantw, y2 + dx2 + dw2))


def test_offsets_past_32_bits(uly):
    """2^20 tokens of 24 heads, 3.2e9 values: the last tokens as a call of their own on them gives."""
    n, inv = 1 << 20, 1e6 ** (-np.arange(64) / 64)
    x = torch.empty(1, 1, n, 24, 128, device="cuda", dtype=BF16).normal_()
    parts = x.split([16, 4, 4], dim=3)
    y = [torch.empty(1, 1, n, h, 128, device="cuda", dtype=BF16) for h in (16, 4, 4)]
    uly.ulysses_qkv_norm_rope_fwd(*parts, *y, 1, inv_freq=inv)
    tail = [t[:, :, -5:].contiguous() for t in parts]
    want = [torch.empty_like(t) for t in tail]
    at = torch.arange(n - 5, n, device="cuda").view(1, 1, 5)
    uly.ulysses_qkv_norm_rope_fwd(*tail, *want, 1, inv_freq=inv, positions=at)
    assert all(bytes_equal(a[:, :, -5:], b) for a, b in zip(y, want))
    dx = torch.empty_like(x)
    uly.ulysses_qkv_norm_rope_bwd(None, None, *y, *dx.split([16, 4, 4], dim=3), 1, inv_freq=inv)
    back = [torch.empty_like(t) for t in tail]
    uly.ulysses_qkv_norm_rope_bwd(None, None, *want, *back, 1, inv_freq=inv, positions=at)
    assert all(bytes_equal(a[:, :, -5:], b) for a, b in zip(dx.split([16, 4, 4], dim=3), back))
