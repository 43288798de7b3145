"""ulysses_window_attn_fwd / _bwd against the fp64 reference of window_ref.py,
element by element within its bounds; and over whole tensors within the
attention path's own tolerances (relative Frobenius 5e-3 in bf16, 1e-5 in fp32)."""
import math

import pytest
import torch

from parity_utils import Guards, REL_TOL, log_errors
from window_ref import allowed, check, reference

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def inputs(S, B, N, Hq, Hkv, d, dtype, seed=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * N)
    rand = lambda H: torch.randn(S, B, N, H, d, device="cuda", generator=g)
    return (rand(Hq) * spread).to(dtype), rand(Hkv).to(dtype), rand(Hkv).to(dtype), rand(Hq).to(dtype)


def run(uly, q, k, v, dout, window, sinks, cu, **kw):
    g = Guards()
    nan = float("nan")
    S, B, N, Hq, d = q.shape
    Hkv, nd = k.shape[3], len(cu) - 1 if cu else 0
    o, lse = g.full_like(q, nan), g.empty((S, B, Hq, N), FP32, nan)
    ws = lambda bwd: g.workspace(uly.ulysses_window_attn_workspace_size(B, N, Hq, Hkv, d, S, window, sinks, nd, bwd,
                                                                        q.dtype))
    uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks, cu_seqlens=cu, workspace=ws(False), **kw)
    dq, dk, dv = g.full_like(q, nan), g.full_like(k, nan), g.full_like(v, nan)
    uly.ulysses_window_attn_bwd(q, k, v, o, lse, dout, dq, dk, dv, window, sinks, cu_seqlens=cu, workspace=ws(True),
                                **kw)
    g.check()
    assert uly.ulysses_get_device_status()[0] == 0
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


CASES = [
    # S, B, N, Hq, Hkv, window, sinks, documents
    (1, 1, 1, 1, 1, 1, 0, None),
    (1, 1, 2, 2, 1, 1, 1, None),
    (2, 1, 65, 2, 2, 1, 0, None),             # every row sees itself alone
    (1, 2, 128, 2, 1, 128, 0, None),
    (1, 1, 129, 3, 1, 64, 1, None),
    (1, 1, 200, 2, 1, 1000, 7, None),         # wider than the sequence: causal
    (1, 1, 200, 2, 1, 50, 1000, None),        # every token a sink: causal
    (2, 2, 333, 6, 2, 77, 3, None),
    (1, 1, 300, 8, 1, 7, 4, None),
    (1, 1, 517, 2, 1, 128, 128, None),
    (1, 1, 700, 2, 1, 200, 130, None),        # sinks that end inside the second tile
    (1, 1, 640, 1, 1, 129, 64, None),
    (1, 1, 2500, 2, 1, 100, 4, None),         # the sinks' walk is cut
    (2, 1, 1985, 2, 2, 1, 1, None),
    (1, 1, 2311, 3, 1, 120, 200, None),       # two tiles of sinks, both cut
    (1, 1, 640, 2, 1, 50, 5, [0, 1, 2, 130, 131, 400, 640]),
    (1, 2, 300, 4, 2, 33, 2, [0, 0, 100, 100, 100, 300, 300]),   # empty documents
    (1, 1, 2600, 2, 1, 64, 5, [0, 126, 1900, 2600]),  # sinks across two tiles, walks cut
    (1, 1, 1500, 2, 1, 300, 130, [0, 250, 1500]),
    (1, 1, 1024, 2, 2, 128, 0, [0, 128, 1024]),
]


@pytest.mark.parametrize("S,B,N,Hq,Hkv,window,sinks,cu", CASES)
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP32, 128), (FP32, 64)], ids=["bf16", "fp32-128", "fp32-64"])
def test_against_reference(uly, S, B, N, Hq, Hkv, window, sinks, cu, dtype, d):
    q, k, v, dout = inputs(S, B, N, Hq, Hkv, d, dtype)
    val, err = reference(q, k, v, dout, allowed(N, window, sinks, cu), 1 / math.sqrt(d), dtype == BF16)
    got = run(uly, q, k, v, dout, window, sinks, cu)
    rel = {n: check(n, got[n], val[n], err[n]) for n in val}
    name = "bf16" if dtype == BF16 else "fp32"
    log_errors(f"window {name} N{N} w{window} s{sinks}", **rel)
    if N > 16:  # a one-key row's dQ and dK are remainders of a cancellation
        if window >= 64:  # rows of few keys have a dQ of the same kind
            assert all(rel[n] <= REL_TOL[name] for n in ("o", "dv", "dq", "dk")), rel
        else:
            assert rel["o"] <= REL_TOL[name] and rel["dv"] <= REL_TOL[name], rel


def test_scores_that_rise_along_the_window(uly):
    """Scores far apart: the running maximum rises again and again, and the sinks
    either hold nearly all of a row or nearly nothing."""
    N, d, window, sinks = 900, 128, 300, 4
    for sign in (1, -1):
        q, k, v, dout = inputs(1, 1, N, 2, 1, d, BF16, seed=3)
        way = torch.randn(d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
        way = way / way.norm()
        q = (q.float() + 20 * way).to(BF16)
        ramp = sign * 20 * torch.linspace(0, 1, N, device="cuda")
        k = (k.float() + ramp[:, None, None] * way).to(BF16)
        val, err = reference(q, k, v, dout, allowed(N, window, sinks, None), 1 / math.sqrt(d), True)
        got = run(uly, q, k, v, dout, window, sinks, None)
        for n in val:
            check(n, got[n], val[n], err[n])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_scale_and_allocated_workspace(uly, dtype):
    """A softmax scale of the caller's, and workspaces that the call allocates."""
    q, k, v, dout = inputs(1, 1, 300, 4, 2, 128, dtype)
    val, err = reference(q, k, v, dout, allowed(300, 90, 3, None), 0.05, dtype == BF16)
    o, lse = torch.empty_like(q), torch.empty(1, 1, 4, 300, device="cuda")
    uly.ulysses_window_attn_fwd(q, k, v, o, lse, 90, 3, softmax_scale=0.05)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    uly.ulysses_window_attn_bwd(q, k, v, o, lse, dout, *grads, 90, 3, softmax_scale=0.05)
    for n, t in zip(("o", "lse", "dq", "dk", "dv"), [o, lse] + grads):
        check(n, t, val[n], err[n])


@pytest.mark.parametrize("cu", [None, [0, 126, 1900, 2600]], ids=["whole", "documents"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_streams_graphs_and_repeats(uly, dtype, cu):
    """Another stream and a captured, replayed call give the same bits (bf16 dQ,
    summed with atomics, stays within two roundings); the documents a captured
    call was given are the ones it replays with."""
    N, window, sinks = 2600, 100, 4
    q, k, v, dout = inputs(1, 1, N, 2, 1, 128, dtype)
    want = run(uly, q, k, v, dout, window, sinks, cu)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = run(uly, q, k, v, dout, window, sinks, cu, stream=side)
    got = {n: torch.empty_like(t) for n, t in want.items()}
    nd = len(cu) - 1 if cu else 0
    ws = [torch.empty(uly.ulysses_window_attn_workspace_size(1, N, 2, 1, 128, 1, window, sinks, nd, b, dtype),
                      dtype=torch.uint8, device="cuda") for b in (False, True)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        docs = list(cu) if cu else None
        uly.ulysses_window_attn_fwd(q, k, v, got["o"], got["lse"], window, sinks, cu_seqlens=docs, workspace=ws[0])
        uly.ulysses_window_attn_bwd(q, k, v, got["o"], got["lse"], dout, got["dq"], got["dk"], got["dv"], window, sinks,
                                    cu_seqlens=docs, workspace=ws[1])
    del docs
    for _ in range(2):
        for t in list(got.values()) + ws:
            t.fill_(float("nan") if t.is_floating_point() else 0x7f)
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            for t in (got[n], again[n]):
                if n == "dq" and dtype == BF16:
                    assert (t.float() - want[n].float()).abs().max() <= 2.0 ** -7 * want[n].float().abs().max()
                else:
                    assert torch.equal(t, want[n]), n
    assert uly.ulysses_get_device_status()[0] == 0


def test_two_calls_at_once(uly):
    """Two calls on two streams, each with its own workspace."""
    a, b = (inputs(1, 1, 1500, 2, 1, 128, BF16, seed=s) for s in (1, 2))
    want = [run(uly, *t, 200, 4, None) for t in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for t, s in zip((a, b), streams):
        q, k, v, dout = t
        o, lse = torch.empty_like(q), torch.empty(1, 1, 2, 1500, device="cuda")
        grads = [torch.empty_like(x) for x in (q, k, v)]
        torch.cuda.synchronize()
        got.append((o, lse, grads))
    for t, s, (o, lse, grads) in zip((a, b), streams, got):
        q, k, v, dout = t
        uly.ulysses_window_attn_fwd(q, k, v, o, lse, 200, 4, stream=s)
        uly.ulysses_window_attn_bwd(q, k, v, o, lse, dout, *grads, 200, 4, stream=s)
    torch.cuda.synchronize()
    for w, (o, lse, grads) in zip(want, got):
        assert torch.equal(w["o"], o) and torch.equal(w["lse"], lse)
        assert torch.equal(w["dk"], grads[1]) and torch.equal(w["dv"], grads[2])


def test_against_full_attention(uly):
    """A window as wide as the sequence is ulysses_attn_fwd / _bwd, whatever the sinks."""
    q, k, v, dout = inputs(2, 1, 777, 4, 2, 128, BF16)
    o, lse = torch.empty_like(q), torch.empty(2, 1, 4, 777, device="cuda")
    uly.ulysses_attn_fwd(q, k, v, o, lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    uly.ulysses_attn_bwd(q, k, v, o, lse, dout, *grads)
    got = run(uly, q, k, v, dout, 777, 5, None)
    val, err = reference(q, k, v, dout, allowed(777, 777, 0, None), 1 / math.sqrt(128), True)
    for n, t in zip(("o", "lse", "dq", "dk", "dv"), [o, lse] + grads):
        check(n, t, val[n], err[n])
        check(n, got[n], val[n], err[n])


def test_gradients_against_differences(uly):
    """fp32 gradients against central differences of the forward, cut walk and all."""
    N, window, sinks, cu = 1300, 20, 2, [0, 40, 1300]
    q, k, v, dout = inputs(1, 1, N, 2, 1, 64, FP32, seed=5)
    got = run(uly, q, k, v, dout, window, sinks, cu)
    g = torch.Generator(device="cuda").manual_seed(9)

    def value(q, k, v):
        o, lse = torch.empty_like(q), torch.empty(1, 1, 2, N, device="cuda")
        uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks, cu_seqlens=cu)
        return float((o.double() * dout.double()).sum())

    for i, n in enumerate(("dq", "dk", "dv")):
        way = torch.randn(got[n].shape, device="cuda", generator=g)
        step = 2.0 ** -6

        def at(s):
            t = [q, k, v]
            t[i] = t[i] + s * way
            return value(*t)

        slope = (8 * (at(step) - at(-step)) - (at(2 * step) - at(-2 * step))) / (12 * step)
        want = float((got[n].double() * way.double()).sum())
        # a value is off by about 2^-24 of its terms' magnitudes (sum |o dO| below 2^18), over a step of 2^-6 with
        # weights 18/12: 2^-24 2^18 2^6 1.5 < 2^1 at the very worst, and errors of that many terms cancel to its root
        assert abs(slope - want) <= 0.05 * (1 + 2.0 ** -4 * abs(want)), (n, slope, want)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("N,window,sinks,cu", [(1, 5, 3, None), (65, 1, 0, None), (300, 1, 0, [0, 130, 300]),
                                               (4, 9, 2, [0, 1, 2, 3, 4])])
def test_rows_that_see_only_themselves(uly, dtype, N, window, sinks, cu):
    """dS = P (dP - <dO, O>) is 0 exactly, and so are dQ and dK; O is V, dV the group's dO."""
    q, k, v, dout = inputs(1, 2, N, 4, 2, 128, dtype)
    got = run(uly, q, k, v, dout, window, sinks, cu)
    assert (got["dq"] == 0).all() and (got["dk"] == 0).all()
    assert torch.equal(got["o"], v.repeat_interleave(2, dim=3))
    want = dout.double().view(1, 2, N, 2, 2, 128).sum(4)
    assert (got["dv"].double() - want).abs().max() <= torch.finfo(dtype).eps / 2 * want.abs().max()


def test_rows_of_few_keys(uly):
    """Rows of two to eight keys, one of which holds most of the row: dS of that key is the small rest of a
    cancellation, which D = <dO, O> from the rounded O would lose.  Each of dS's factors is then off by a rounding
    (P, dS: 2^-9 on average 2^-10 each) and the gradient by its own, together below 4e-3 of its norm."""
    for N, window, sinks, cu in ((2, 9, 0, None), (4, 50, 1, None), (900, 3, 1, None), (300, 2, 1, None),
                                 (22, 90, 1, [0, 3, 5, 9, 11, 16, 22])):
        q, k, v, dout = inputs(2, 2, N, 8, 2, 128, BF16, seed=7)
        first = torch.zeros(N, dtype=torch.bool, device="cuda")
        first[torch.tensor((cu or [0, N])[:-1], device="cuda")] = True
        common = torch.randn(128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        q = (q.float() + 0.5 * common).to(BF16)
        k = torch.where(first[:, None, None], k.float() + 0.5 * common, k.float()).to(BF16)
        val, _ = reference(q, k, v, dout, allowed(N, window, sinks, cu), 1 / math.sqrt(128), True)
        got = run(uly, q, k, v, dout, window, sinks, cu)
        for n in ("dq", "dk"):
            off = float((got[n].double() - val[n]).norm() / val[n].norm())
            assert off <= 4.5e-3, (N, n, off)
