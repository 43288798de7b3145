"""ulysses_residual_norm_fwd / _bwd against fp64.

Tolerances, element by element: an output is off by its own rounding, u times its
value (u = eps/2 of its type, 2^-8 in bf16, 2^-24 in fp32), and by the fp32
arithmetic before it.  With e = 2^-24: a row's sum of D products goes through at
most 16 additions in a thread, 5 over lanes and 16 over warps, so statistics and
means are within 48 e of their terms' magnitudes; the chains of products behind
them have fewer than 16 roundings.  64 e (forward, dx) and 160 e (dy, which goes
through two such sums and dx) of the summed magnitudes of a value's terms cover
them.  A weight's gradient is a sum over T tokens, off by at most (T + 64) e of
its terms' magnitudes whatever the order, terms included.
"""
import numpy as np
import pytest
import torch

from parity_utils import Guards

pytestmark = pytest.mark.gpu
EPS = 1e-6
E = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def make(B, N, P, D, gate, post, first, dtype, seed=0, scale=0.75):
    g = torch.Generator().manual_seed(seed + N * 1000 + D)
    rand = lambda *s: torch.randn(*s, generator=g)
    rows = (P, B, N // P, D)
    c = {"x": rand(*rows) * (1 + 20 * (torch.rand(D, generator=g) < 0.02)), "weight": 1 + 0.3 * rand(D),
         "dz": rand(*rows), "dh": rand(*rows), "y": None, "post": None, "gate": None}
    if not first:
        c["y"] = 3 * rand(*rows)
        if post:
            c["post"] = 1 + 0.3 * rand(D)
        if gate:
            c["gate"] = rand(*((D,) if gate == "shared" else (B, D)))
    c = {k: None if v is None else v.to(dtype) for k, v in c.items()}
    return c, scale


def reference(c, scale):
    """Values and gradients in fp64 by autograd, and the magnitudes that bound the fp32 arithmetic."""
    c = _gpu(c)
    x, y, w, post, gate = (None if c[n] is None else c[n].double().requires_grad_(True)
                           for n in ("x", "y", "weight", "post", "gate"))
    D = x.shape[-1]
    rms = lambda t: 1 / (t.square().mean(-1, keepdim=True) + EPS).sqrt()
    r2 = torch.ones_like(x[..., :1])
    h, mag_h = x, x.abs()
    g = 1.0 if gate is None else gate[:, None] if gate.dim() == 2 else gate
    if y is not None:
        yh = y
        if post is not None:
            r2 = rms(y)
            yh = y * r2
        u = yh if post is None else yh * post
        h = x + scale * g * u
        mag_h = x.abs() + (scale * g * u).abs()
    r1 = rms(h)
    z = h * r1 * w
    leaves = [t for t in (x, y, w, post, gate) if t is not None]
    grads = iter(torch.autograd.grad([z, h], leaves, [c["dz"].double(), c["dh"].double()]))
    grad = {n: None if t is None else next(grads) for n, t in zip(("x", "y", "weight", "post", "gate"),
                                                                  (x, y, w, post, gate))}
    with torch.no_grad():
        dz, dh = c["dz"].double(), c["dh"].double()
        mh, gz = mag_h * r1, (w * dz).abs()
        t = dh.abs() + r1 * (gz + mh * (gz * mh).mean(-1, keepdim=True))
        mag = {"h": mag_h, "z": mh * w.abs(), "x": t, "weight": (dz.abs() * mh).sum((0, 1, 2))}
        if y is not None:
            f = scale * (g.abs() if gate is not None else 1.0) * (1.0 if post is None else post.abs())
            mag["y"] = r2 * f * t
            if post is not None:
                mag["y"] = r2 * (f * t + yh.abs() * (f * t * yh.abs()).mean(-1, keepdim=True))
                mag["post"] = (f / post.abs() * t * yh.abs()).sum((0, 1, 2))
            if gate is not None:
                mag["gate"] = (scale * t * u.abs()).sum((0, 2) if gate.dim() == 2 else (0, 1, 2))
    return h.detach(), z.detach(), r1[..., 0].detach(), r2[..., 0].detach(), grad, mag


def close(name, got, want, unit, extra):
    got = got.detach().double()
    assert got.shape == want.shape, name
    off = (got - want).abs() - (unit * want.abs() + extra)
    worst = off.max().item()
    assert worst <= 0, f"{name}: {worst} beyond the tolerance at {np.unravel_index(int(off.argmax()), off.shape)}"


CASES = [
    # B, N, P, D, gate, post, first
    (1, 1, 1, 64, None, True, False),
    (8, 1, 1, 2560, None, True, False),
    (8, 1, 1, 2560, "sequence", False, False),
    (2, 303, 3, 776, "sequence", True, False),
    (5, 24, 4, 72, "sequence", True, False),
    (3, 10, 2, 264, "shared", True, False),
    (3, 1000, 1, 64, "shared", False, False),
    (1, 700, 2, 1024, "shared", True, False),
    (1, 257, 1, 4096, None, False, False),
    (2, 6, 3, 4104, "sequence", True, False),
    (2, 6, 3, 8192, "shared", True, False),
    (1, 900, 1, 2560, "shared", True, False),
    (2, 55, 5, 128, None, False, True),
    (1, 321, 1, 2560, None, False, True),
    (40, 2, 2, 16, "sequence", True, False),
    # many slots a block: every ring goes round several times
    (1, 9600, 4, 2560, "shared", True, False),
    (2, 9063, 3, 776, "sequence", True, False),
    (1, 60000, 2, 64, "shared", True, False),
    (1, 3100, 1, 8192, None, False, False),
    (1, 3100, 1, 2048, None, False, True),
    (1, 20000, 1, 512, "shared", True, False),
    # many gates
    (16, 130, 1, 264, "sequence", True, False),
    (130, 6, 2, 776, "sequence", True, False),
    (300, 1, 1, 72, "sequence", False, False),
]


def _gpu(c):
    return {k: None if v is None else v.cuda() for k, v in c.items()}


def forward(uly, c, scale, P, g, **kw):
    d = _gpu(c)
    like = lambda: g.full_like(d["x"], float("nan"))
    h, z = (None if d["y"] is None else like()), like()
    rstd = g.empty((2,) + tuple(d["x"].shape[:3]), FP32, float("nan"))
    uly.ulysses_residual_norm_fwd(d["x"], d["y"], h, z, P, d["weight"], d["post"], d["gate"], scale, rstd, EPS, **kw)
    return d, h, z, rstd


def backward(uly, d, rstd, scale, P, g, dh=True, want=("weight", "post", "gate"), **kw):
    like = lambda n: None if d[n] is None else g.full_like(d[n], float("nan"))
    out = {n: like(n) for n in ("x", "y", "weight", "post", "gate")}
    for n in ("weight", "post", "gate"):
        if n not in want:
            out[n] = None
    B, Np, D = d["x"].shape[1:]
    ws = g.workspace(uly.ulysses_residual_norm_workspace_size(B, Np * P, D, P))
    uly.ulysses_residual_norm_bwd(d["x"], d["y"], d["dh"] if dh else None, d["dz"], out["x"], out["y"], P, d["weight"],
                                  rstd, d["post"], d["gate"], scale, out["weight"], out["post"], out["gate"],
                                  workspace=ws, **kw)
    return out


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,N,P,D,gate,post,first", CASES)
def test_values_and_gradients(uly, B, N, P, D, gate, post, first, dtype):
    c, scale = make(B, N, P, D, gate, post, first, dtype)
    h, z, r1, r2, grad, mag = reference(c, scale)
    unit = torch.finfo(dtype).eps / 2
    g = Guards()
    d, gh, gz, rstd = forward(uly, c, scale, P, g)
    close("rstd of h", rstd[0], r1, E, 64 * E * r1)
    close("rstd of y", rstd[1], r2, E, 64 * E * r2)
    close("z", gz, z, unit, 64 * E * mag["z"])
    if not first:
        close("h", gh, h, unit, 64 * E * mag["h"])
    out = backward(uly, d, rstd, scale, P, g)
    g.check()
    assert uly.ulysses_get_device_status()[0] == 0
    close("dx", out["x"], grad["x"], unit, 64 * E * mag["x"])
    if not first:
        close("dy", out["y"], grad["y"], unit, 160 * E * mag["y"])
    tokens = B * N
    for n in ("weight", "post", "gate"):
        if out[n] is not None:
            close("d" + n, out[n], grad[n], unit, (tokens + 64) * E * mag[n])


@pytest.mark.parametrize("dtype,D", [(BF16, 16384), (FP32, 8192), (BF16, 8200), (FP32, 4100)])
def test_long_rows(uly, dtype, D):
    """Rows of up to 32 KB: two and four chunks a thread, one row in a slot."""
    test_values_and_gradients(uly, 2, 9, 3, D, "sequence", True, False, dtype)


def test_against_differences(uly):
    """The gradients against central differences of the forward itself, fp32."""
    B, N, P, D = 1, 2, 1, 64
    c, scale = make(B, N, P, D, "shared", True, False, FP32)
    g = Guards()
    d, _, _, rstd = forward(uly, c, scale, P, g)
    out = backward(uly, d, rstd, scale, P, g)

    def value(c):
        _, h, z, _ = forward(uly, c, scale, P, g)
        return float((h.double().cpu() * c["dh"].double()).sum() + (z.double().cpu() * c["dz"].double()).sum())

    rng = np.random.default_rng(1)
    for n in ("x", "y", "weight", "post", "gate"):
        way = torch.from_numpy(rng.standard_normal(c[n].shape)).float()
        step = 2.0 ** -6
        at = lambda s: value({**c, n: c[n] + s * way})
        slope = (8 * (at(step) - at(-step)) - (at(2 * step) - at(-2 * step))) / (12 * step)
        want = float((out[n].double().cpu() * way.double()).sum())
        # fourth-order differences: the step's fourth power (2^-24) times the fifth derivative's share, and
        # the values' 2^-24 over the step; 2^-24 * 256 of the values' magnitudes is beyond both
        assert abs(slope - want) <= 2e-3 * (1 + abs(want)), n


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_what_is_left_out(uly, dtype):
    """No h, no rstd, no dh, some of the weights' gradients: the rest keeps its bits."""
    c, scale = make(2, 66, 2, 520, "sequence", True, False, dtype)
    g = Guards()
    d, h, z, rstd = forward(uly, c, scale, 2, g)
    z2 = g.full_like(z, float("nan"))
    uly.ulysses_residual_norm_fwd(d["x"], d["y"], None, z2, 2, d["weight"], d["post"], d["gate"], scale, None, EPS)
    assert torch.equal(z, z2)
    whole = backward(uly, d, rstd, scale, 2, g)
    for want in ((), ("weight",), ("post",), ("gate",), ("post", "gate")):
        part = backward(uly, d, rstd, scale, 2, g, want=want)
        for n in ("x", "y") + want:
            assert torch.equal(part[n], whole[n]), (want, n)
    without = backward(uly, d, rstd, scale, 2, g, dh=False)
    d["dh"].zero_()
    zero = backward(uly, d, rstd, scale, 2, g)
    for n in without:
        assert torch.equal(without[n], zero[n]), n
    g.check()


def test_streams_graphs_and_repeats(uly):
    """Another stream, a captured and replayed call, and repeats give the same bits."""
    c, scale = make(3, 210, 3, 776, "sequence", True, False, BF16)
    g = Guards()
    d, h, z, rstd = forward(uly, c, scale, 3, g)
    out = backward(uly, d, rstd, scale, 3, g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _, h2, z2, rstd2 = forward(uly, c, scale, 3, g, stream=side)
    side.synchronize()
    out2 = backward(uly, d, rstd2, scale, 3, g, stream=side)
    side.synchronize()
    assert torch.equal(z, z2) and torch.equal(h, h2) and torch.equal(rstd, rstd2)
    assert all(torch.equal(out[n], out2[n]) for n in out)
    hg, zg = torch.empty_like(h), torch.empty_like(z)
    grads = {n: torch.empty_like(t) for n, t in out.items()}
    ws = torch.empty(uly.ulysses_residual_norm_workspace_size(3, 210, 776, 3), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uly.ulysses_residual_norm_fwd(d["x"], d["y"], hg, zg, 3, d["weight"], d["post"], d["gate"], scale, rstd2, EPS)
        uly.ulysses_residual_norm_bwd(d["x"], d["y"], d["dh"], d["dz"], grads["x"], grads["y"], 3, d["weight"], rstd2,
                                      d["post"], d["gate"], scale, grads["weight"], grads["post"], grads["gate"],
                                      workspace=ws)
    for _ in range(2):
        for t in [hg, zg] + list(grads.values()):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, zg) and torch.equal(h, hg)
        assert all(torch.equal(out[n], grads[n]) for n in out)


def test_infinities_and_nan_stay_in_their_rows(uly):
    """A row with an infinity or a NaN spoils itself and the sums, no other row."""
    c, scale = make(1, 40, 1, 96, "shared", True, False, FP32)
    g = Guards()
    d, h, z, rstd = forward(uly, c, scale, 1, g)
    clean = backward(uly, d, rstd, scale, 1, g)
    c["x"][0, 0, 7, 3] = float("inf")
    c["y"][0, 0, 21, 5] = float("nan")
    d, h2, z2, rstd2 = forward(uly, c, scale, 1, g)
    spoilt = backward(uly, d, rstd2, scale, 1, g)
    rows = [i for i in range(40) if i not in (7, 21)]
    assert torch.equal(z[0, 0, rows], z2[0, 0, rows]) and torch.equal(h[0, 0, rows], h2[0, 0, rows])
    assert torch.equal(clean["x"][0, 0, rows], spoilt["x"][0, 0, rows])
    assert torch.equal(clean["y"][0, 0, rows], spoilt["y"][0, 0, rows])
    assert torch.isnan(z2[0, 0, 21]).all() and torch.isnan(z2[0, 0, 7, 3])
