"""Calls that ulysses_window_attn_* and ulysses_residual_norm_* refuse on the
host, before anything is launched (CPU only; the pointers are made up and never
dereferenced)."""
import ctypes

import pytest
import torch

import long_context_sequence_head_gb300 as uly_py

OK, INVALID, UNSUPPORTED, MISALIGNED, OVERLAP, CUDA, WORKSPACE = 0, 1, 2, 3, 4, 5, 7
BF16, FP32 = 0, 1
A = [(i + 1) << 44 for i in range(16)]  # addresses far from each other


def _cu(cu):
    if cu is None:
        return None, 0
    arr = (ctypes.c_int32 * len(cu))(*cu)
    return ctypes.cast(arr, ctypes.c_void_p), len(cu) - 1


def _attn(uly, bwd, B=1, N=256, Hq=8, Hkv=2, d=128, S=1, window=64, sinks=4, cu=None, nd=None, dt=BF16, wsb=1 << 40,
          **at):
    names = ("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "ws") if bwd else ("q", "k", "v", "o", "lse", "ws")
    p = dict(zip(names, A))
    p.update(at)
    cu_p, n = _cu(cu)
    fn = uly.load().ulysses_window_attn_bwd if bwd else uly.load().ulysses_window_attn_fwd
    return fn(*[p[n] for n in names[:-1]], B, N, Hq, Hkv, d, S, window, sinks, cu_p, n if nd is None else nd, 0.0, dt,
              p["ws"], wsb, None)


@pytest.mark.parametrize("bwd", [False, True], ids=["fwd", "bwd"])
def test_attention_refusals(uly, bwd):
    f = lambda **k: _attn(uly, bwd, **k)
    names = ("q", "k", "v", "o", "lse", "ws") + (("dout", "dq", "dk", "dv") if bwd else ())
    for name in names:
        assert f(**{name: None}) == INVALID, name
        base = dict(zip(("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "ws") if bwd else
                        ("q", "k", "v", "o", "lse", "ws"), A))[name]
        assert f(**{name: base + 8}) == MISALIGNED, name
    assert f(B=0) == f(N=0) == f(Hq=0) == f(Hkv=0) == f(S=0) == f(Hkv=3) == f(dt=5) == INVALID
    assert f(window=0) == f(window=-1) == f(sinks=-1) == INVALID
    assert f(d=64) == f(d=96) == f(N=1 << 31) == f(S=1 << 11, B=1 << 10) == UNSUPPORTED
    assert f(N=1 << 30, Hq=1024) == f(S=1 << 10, B=1 << 10, N=1 << 20) == UNSUPPORTED  # blocks of one launch
    assert f(cu=[0, 100]) == f(cu=[1, 256]) == f(cu=[0, 200, 100, 256]) == f(nd=2) == f(cu=[0, 256], nd=0) == INVALID
    assert f(wsb=0) == WORKSPACE
    outs = ("dq", "dk", "dv", "ws") if bwd else ("o", "lse", "ws")
    ins = ("q", "k", "v") + (("o", "lse", "dout") if bwd else ())
    at = dict(zip(("q", "k", "v", "o", "lse", "dout", "dq", "dk", "dv", "ws") if bwd else
                  ("q", "k", "v", "o", "lse", "ws"), A))
    for out in outs:
        for other in ins + tuple(n for n in outs if n != out):
            assert f(**{out: at[other]}) == OVERLAP, (out, other)
        assert f(**{out: at["q"] + 256 * 8 * 128 * 2 - 16}) == OVERLAP, out


def test_attention_workspace(uly):
    ws = uly.ulysses_window_attn_workspace_size
    args = dict(B=1, N=4096, Hq_local=8, Hkv_local=2, d=128, num_shards=1, window=256, sinks=4, num_docs=0,
                for_bwd=True, dtype=torch.bfloat16)
    need = ws(**args)
    assert need >= 8 * 4096 * (128 + 2) * 4
    assert _attn(uly, True, N=4096, window=256, wsb=need - 1) == WORKSPACE
    assert ws(**{**args, "window": 0}) == ws(**{**args, "sinks": -1}) == ws(**{**args, "num_docs": -1}) == 0
    assert ws(**{**args, "d": 64}) == ws(**{**args, "Hkv_local": 3}) == ws(**{**args, "N": 0}) == 0
    assert ws(**{**args, "for_bwd": False}) <= 256
    # documents that the size does not know: never less than what a call with them takes
    assert ws(**{**args, "num_docs": 5}) >= need
    assert _attn(uly, True, N=4096, window=256, cu=[0, 9, 900, 4096], wsb=ws(**{**args, "num_docs": 3}) - 1) == WORKSPACE


def _decode(uly, B=2, C=64, Hq=8, Hkv=2, d=128, S=1, window=32, sinks=4, dt=BF16, wsb=1 << 40, **at):
    names = ("q", "k", "v", "lens", "o", "lse", "ws")
    p = dict(zip(names, A))
    p.update(at)
    return uly.load().ulysses_window_attn_decode(*[p[n] for n in names[:-1]], B, C, Hq, Hkv, d, S, window, sinks, 0.0, dt,
                                                 p["ws"], wsb, None)


def test_decode_refusals(uly):
    f = lambda **k: _decode(uly, **k)
    for i, name in enumerate(("q", "k", "v", "lens", "o", "lse", "ws")):
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: A[i] + 4}) == MISALIGNED, name
    assert f(lens=A[3] + 8, wsb=0) == WORKSPACE  # lengths need 8 bytes of alignment, no more
    assert f(B=0) == f(C=0) == f(Hq=0) == f(Hkv=3) == f(S=0) == f(window=0) == f(sinks=-1) == f(dt=2) == INVALID
    assert f(d=64) == f(d=32, dt=FP32) == f(C=(1 << 30) + 1) == f(S=1 << 11, B=1 << 10) == UNSUPPORTED
    assert f(B=1 << 20, Hq=64, Hkv=64) == UNSUPPORTED
    assert f(wsb=0) == WORKSPACE
    for out in ("o", "lse", "ws"):
        for i, other in enumerate(("q", "k", "v", "lens", "o", "lse", "ws")):
            if other != out:
                assert f(**{out: A[i]}) == OVERLAP, (out, other)
        assert f(**{out: A[1] + 2 * 64 * 2 * 128 * 2 - 16}) == OVERLAP
    ws = uly.ulysses_window_attn_decode_workspace_size
    assert ws(2, 64, 8, 2, 128, 1, 32, 4, torch.bfloat16) > 0
    assert ws(2, 64, 8, 3, 128, 1, 32, 4, torch.bfloat16) == ws(2, 64, 8, 2, 128, 1, 0, 4, torch.bfloat16) == 0


def _norm_fwd(uly, B=2, N=8, D=64, P=2, rows=1, scale=1.0, eps=1e-6, dt=BF16, **at):
    names = ("x", "y", "w1", "w2", "gate", "h", "z", "rstd")
    p = dict(zip(names, A))
    p.update(at)
    return uly.load().ulysses_residual_norm_fwd(p["x"], p["y"], p["w1"], p["w2"], p["gate"], rows, scale, eps, p["h"],
                                                p["z"], p["rstd"], B, N, D, P, dt, None)


def _norm_bwd(uly, B=2, N=8, D=64, P=2, rows=1, scale=1.0, dt=BF16, wsb=1 << 40, **at):
    names = ("x", "y", "w1", "w2", "gate", "rstd", "dh", "dz", "dx", "dy", "dw1", "dw2", "dgate", "ws")
    p = dict(zip(names, A))
    p.update(at)
    return uly.load().ulysses_residual_norm_bwd(
        p["x"], p["y"], p["w1"], p["w2"], p["gate"], rows, scale, p["rstd"], p["dh"], p["dz"], p["dx"], p["dy"],
        p["dw1"], p["dw2"], p["dgate"], B, N, D, P, dt, p["ws"], wsb, None)


def test_norm_sizes(uly):
    for f in (lambda **k: _norm_fwd(uly, **k), lambda **k: _norm_bwd(uly, **k)):
        assert f(B=0) == f(N=0) == f(D=0) == f(P=0) == f(N=9) == f(dt=7) == INVALID
        assert f(scale=float("nan")) == f(scale=float("inf")) == INVALID
        assert f(rows=0) == f(rows=3) == f(rows=-1) == f(gate=None) == INVALID
        assert f(gate=None, rows=0, x=None) == f(w1=None) == INVALID
        assert f(D=60) == f(D=16392) == f(D=8196, dt=FP32) == f(B=1 << 20, N=1 << 12) == UNSUPPORTED
        assert f(x=A[0] + 8) == f(gate=A[4] + 8) == MISALIGNED


def test_norm_forward_refusals(uly):
    f = lambda **k: _norm_fwd(uly, **k)
    assert f(eps=-1.0) == f(eps=float("nan")) == f(eps=float("inf")) == f(z=None) == INVALID
    assert f(y=None) == f(y=None, gate=None, rows=0) == f(y=None, w2=None, gate=None, rows=0) == INVALID  # h without y
    for i, name in enumerate(("x", "y", "w1", "w2", "gate", "h", "z", "rstd")):
        assert f(**{name: A[i] + 8}) == MISALIGNED, name
    for out in ("h", "z", "rstd"):
        for i, other in enumerate(("x", "y", "w1", "w2", "gate", "h", "z", "rstd")):
            if other != out:
                assert f(**{out: A[i]}) == OVERLAP, (out, other)
    assert f(h=A[0] + 2 * 8 * 64 * 2 - 16) == OVERLAP  # no update in place either
    assert f(rows=2, z=A[4] + 64 * 2) == OVERLAP       # the second sequence's gate


def test_norm_backward_refusals(uly):
    f = lambda **k: _norm_bwd(uly, **k)
    assert f(rstd=None) == f(dz=None) == f(dx=None) == f(dy=None) == f(ws=None) == INVALID
    assert f(y=None, w2=None, gate=None, rows=0, dw2=None, dgate=None) == INVALID  # dy without y
    assert f(w2=None) == f(gate=None, rows=0) == INVALID                           # gradients of what is not there
    names = ("x", "y", "w1", "w2", "gate", "rstd", "dh", "dz", "dx", "dy", "dw1", "dw2", "dgate", "ws")
    for i, name in enumerate(names):
        assert f(**{name: A[i] + 8}) == MISALIGNED, name
    for out in names[8:]:
        for i, other in enumerate(names):
            if other != out:
                assert f(**{out: A[i]}) == OVERLAP, (out, other)
    need = uly.ulysses_residual_norm_workspace_size(2, 8, 64, 2)
    assert need > 0 and f(wsb=need - 1) == WORKSPACE
    assert uly.ulysses_residual_norm_workspace_size(2, 9, 64, 2) == 0
    assert uly.ulysses_residual_norm_workspace_size(2, 8, 20000, 2) == 0


# ------------------------------------------------------------ the binding

def test_binding_checks_before_the_library():
    """Shapes, types and devices are told apart before any pointer is passed on."""
    bf, fp = torch.bfloat16, torch.float32
    x = torch.zeros(2, 1, 4, 64, dtype=bf)
    w = torch.zeros(64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        uly_py.ulysses_residual_norm_fwd(x, x, x, x, 2, w)
    with pytest.raises(ValueError, match="P=3"):
        uly_py.ulysses_residual_norm_fwd(x, x, x, x, 3, w)
    with pytest.raises(ValueError, match="without y"):
        uly_py.ulysses_residual_norm_fwd(x, None, x, x, 2, w)
    with pytest.raises(ValueError, match="go together"):
        uly_py.ulysses_residual_norm_bwd(x, x, x, x, x, None, 2, w, torch.zeros(2, 2, 1, 4))
    with pytest.raises(ValueError, match="dpost_weight"):
        uly_py.ulysses_residual_norm_bwd(x, x, x, x, x, x, 2, w, torch.zeros(2, 2, 1, 4), dpost_weight=w)
    q, k = torch.zeros(1, 1, 8, 4, 128, dtype=bf), torch.zeros(1, 1, 8, 2, 128, dtype=bf)
    lse = torch.zeros(1, 1, 4, 8)
    with pytest.raises(ValueError, match="lse"):
        uly_py.ulysses_window_attn_fwd(q, k, k, q, lse[..., :7], 4)
    with pytest.raises(ValueError, match="dtype"):
        uly_py.ulysses_window_attn_fwd(q, k.to(fp), k, q, lse, 4)
    with pytest.raises(ValueError, match="CUDA"):
        uly_py.ulysses_window_attn_fwd(q, k, k, q, lse, 4)
    one, n = q[:, :, :1].contiguous(), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="q must be"):
        uly_py.ulysses_window_attn_decode(q, k, k, n, q, lse, 4)
    with pytest.raises(ValueError, match="lens"):
        uly_py.ulysses_window_attn_decode(one, k, k, n.int(), one, lse[..., :1], 4)
    with pytest.raises(ValueError, match="k_cache"):
        uly_py.ulysses_window_attn_decode(one, k, k[..., :64], n, one, lse[..., :1], 4)
    with pytest.raises(ValueError, match="CUDA"):
        uly_py.ulysses_window_attn_decode(one, k, k, n, one, lse[..., :1].contiguous(), 4)
