"""Calls that ulysses_qkv_norm_rope_* and ulysses_sharded_linear_ce_loss refuse
on the host, before anything is launched (CPU only; the pointers are made up
and never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import long_context_sequence_head_gb300 as uly_py

OK, INVALID, UNSUPPORTED, MISALIGNED, OVERLAP, WORKSPACE = 0, 1, 2, 3, 4, 7
BF16, FP32 = 0, 1
A = [(i + 1) << 36 for i in range(16)]  # addresses far from each other


def _desc(uly, rot=64, inv=None, axis=None, axes=1, inter=0, pos=None):
    inv = np.ones(max(rot // 2, 1)) if inv is None else np.asarray(inv, dtype=np.float64)
    axis = None if axis is None else np.asarray(axis, dtype=np.int32)
    d = uly._RopeDesc(pos, inv.ctypes.data, None if axis is None else axis.ctypes.data, rot, axes, inter)
    d.keep = (inv, axis)
    return d


def _fwd(uly, ptrs=None, B=1, N=8, Hq=4, Hkv=2, d=128, P=2, strides=(0, 0, 0), desc=None, eps=1e-6, to_head=1,
         dt=BF16, **at):
    p = dict(q=A[0], k=A[1], v=A[2], wq=A[3], wk=A[4], qo=A[5], ko=A[6], vo=A[7])
    p.update(at)
    desc = _desc(uly) if desc is None else desc
    return uly.load().ulysses_qkv_norm_rope_fwd(
        p["q"], p["k"], p["v"], p["wq"], p["wk"], p["qo"], p["ko"], p["vo"], B, N, Hq, Hkv, d, P, *strides,
        ctypes.addressof(desc) if desc != 0 else None, eps, to_head, dt, None)


def test_forward_refusals(uly):
    f = lambda **k: _fwd(uly, **k)
    assert f(q=None) == f(ko=None) == INVALID
    assert f(v=None) == f(vo=None) == INVALID                     # one of V and its output
    assert f(wk=None) == INVALID                                  # one of the two weights
    assert f(desc=0) == INVALID
    assert f(B=0) == f(N=0) == f(P=0) == f(Hq=0) == f(Hkv=0) == INVALID
    assert f(N=9) == INVALID                                      # N % P
    assert f(Hq=5) == INVALID                                     # Hq % Hkv
    assert f(Hq=4, Hkv=1) == INVALID                              # Hkv % P in the head layout
    assert f(Hq=4, Hkv=1, to_head=0, q=A[0] + 8) == MISALIGNED    # not in the sequence layout
    assert f(to_head=2) == f(dt=5) == f(eps=-1.0) == f(eps=float("nan")) == f(eps=float("inf")) == INVALID
    assert f(d=96) == UNSUPPORTED
    assert f(B=1 << 20, N=1 << 12) == UNSUPPORTED                 # tokens
    for name in ("q", "k", "v", "wq", "wk", "qo", "ko", "vo"):
        base = dict(q=A[0], k=A[1], v=A[2], wq=A[3], wk=A[4], qo=A[5], ko=A[6], vo=A[7])[name]
        assert f(**{name: base + 8}) == MISALIGNED, name
    assert f(desc=_desc(uly, pos=A[9] + 4)) == MISALIGNED


def test_rotation_refusals(uly):
    f = lambda **k: _fwd(uly, desc=_desc(uly, **k))
    assert f(rot=-16) == f(rot=144) == INVALID
    assert f(rot=24) == UNSUPPORTED                               # not a multiple of 16
    assert f(axes=0) == f(axes=9) == f(inter=2) == INVALID
    assert f(axis=[0] * 31 + [1]) == INVALID                      # an axis that is not there
    assert f(axes=2, axis=[0] * 31 + [-1]) == INVALID
    assert f(inv=[float("nan")] * 32) == f(inv=[float("inf")] * 32) == INVALID
    none = uly._RopeDesc(None, None, None, 64, 1, 0)
    assert _fwd(uly, desc=none) == INVALID                        # no frequencies


def test_strides_and_overlaps(uly):
    f = lambda **k: _fwd(uly, **k)
    assert f(strides=(511, 0, 0)) == INVALID                      # less than a token's heads
    assert f(strides=(0, 0, 255)) == INVALID
    assert f(strides=(516, 0, 0)) == INVALID                      # not a multiple of 16 bytes
    row = 8 * 128  # a packed projection's token: 4 + 2 + 2 heads
    packed = dict(q=A[0], k=A[0] + 2 * 4 * 128, v=A[0] + 2 * 6 * 128, strides=(row, row, row))
    assert f(**packed, qo=A[5] + 8) == MISALIGNED                 # accepted up to there
    assert f(qo=A[0]) == f(ko=A[2] + 256) == f(vo=A[7], ko=A[7]) == f(qo=A[3]) == OVERLAP
    assert f(qo=A[5], ko=A[5] + 8 * 512 * 2 - 16) == OVERLAP
    assert f(**packed, vo=A[0] + 7 * row * 2) == OVERLAP          # the last packed token


def _bwd(uly, B=1, N=8, Hq=4, Hkv=2, d=128, P=2, strides=(0,) * 5, desc=None, to_head=1, dt=BF16, wsb=1 << 24, **at):
    names = ("q", "k", "wq", "wk", "gq", "gk", "gv", "dq", "dk", "dv", "dwq", "dwk", "ws")
    p = dict(zip(names, A))
    p.update(at)
    desc = _desc(uly) if desc is None else desc
    return uly.load().ulysses_qkv_norm_rope_bwd(
        *(p[n] for n in names[:12]), B, N, Hq, Hkv, d, P, *strides, ctypes.addressof(desc), 1e-6, to_head, dt,
        p["ws"], wsb, None)


def test_backward_refusals(uly):
    f = lambda **k: _bwd(uly, **k)
    assert f(gq=None) == f(dk=None) == f(gv=None) == f(dv=None) == INVALID
    assert f(q=None) == f(k=None) == f(ws=None) == INVALID        # the norm needs them
    assert f(wq=None) == INVALID
    assert f(wq=None, wk=None) == INVALID                         # weight gradients without weights
    assert f(wq=None, wk=None, dwq=None, dwk=None, q=None, k=None, ws=None, dq=A[7] + 8) == MISALIGNED
    assert f(wsb=uly.ulysses_qkv_norm_rope_workspace_size(128) - 1) == WORKSPACE
    for name, base in (("dwq", A[10]), ("ws", A[12]), ("gq", A[4])):
        assert f(**{name: base + 8}) == MISALIGNED
    assert f(dq=A[0]) == f(dq=A[4]) == f(dwq=A[2]) == f(dwk=A[10]) == f(ws=A[7]) == OVERLAP
    row = 8 * 128
    packed = dict(dq=A[7], dk=A[7] + 2 * 4 * 128, dv=A[7] + 2 * 6 * 128, strides=(0, 0, row, row, row))
    assert f(**packed, wsb=0) == WORKSPACE                        # views of one buffer: accepted up to there
    packed["dv"] -= 16
    assert f(**packed) == OVERLAP                                 # columns that meet
    packed["dv"] += 32
    assert f(**packed) == OVERLAP                                 # past the row: the next token's q
    assert f(strides=(0, 0, 0, 0, 100)) == INVALID
    assert uly.ulysses_qkv_norm_rope_workspace_size(96) == 0


def _ce(uly, B=1, N=64, D=64, V=100, P=4, dt=BF16, wsb=1 << 34, **at):
    names = ("h", "w", "y", "dh", "dw", "sl", "sg", "tot", "ws")
    p = dict(zip(names, A))
    p.update(at)
    return uly.load().ulysses_sharded_linear_ce_loss(*(p[n] for n in names[:8]), B, N, D, V, P, dt, p["ws"], wsb, None)


def test_linear_ce_refusals(uly):
    f = lambda **k: _ce(uly, **k)
    for name in ("h", "w", "y", "sl", "sg", "tot", "ws"):
        assert f(**{name: None}) == INVALID, name
    assert f(N=65) == f(B=0) == f(V=0) == f(D=0) == f(P=0) == f(dt=3) == INVALID
    assert f(D=60) == f(D=62, dt=FP32) == UNSUPPORTED             # rows of 16 bytes
    assert f(D=65544) == f(V=(1 << 21) + 1) == f(B=1 << 20, N=1 << 12) == UNSUPPORTED
    for i, name in enumerate(("h", "w", "y", "dh", "dw", "sl", "sg", "tot", "ws")):
        assert f(**{name: A[i] + 8}) == MISALIGNED, name
    assert f(dh=A[0]) == f(dw=A[1]) == f(dw=A[3]) == f(sl=A[2]) == f(tot=A[5]) == f(ws=A[0]) == OVERLAP
    assert f(ws=A[3] + 64 * 64 * 2 - 16) == OVERLAP
    need = uly.load().ulysses_sharded_linear_ce_workspace_size
    assert need(1, 64, 64, 100, 4, 1, BF16) > need(1, 64, 64, 100, 4, 0, BF16) > 0
    assert need(1, 65, 64, 100, 4, 1, BF16) == need(1, 64, 60, 100, 4, 1, BF16) == need(1, 64, 64, 100, 4, 2, BF16) == 0
    assert f(wsb=need(1, 64, 64, 100, 4, 1, BF16) - 1) == WORKSPACE
    assert f(dh=None, dw=None, wsb=need(1, 64, 64, 100, 4, 0, BF16) - 1) == WORKSPACE


# ---------------------------------------------------------- Python binding

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _args(**over):
    P, B, Np, d = 2, 1, 4, 128
    a = dict(q_seq=_t(P, B, Np, 4, d), k_seq=_t(P, B, Np, 2, d), v_seq=_t(P, B, Np, 2, d), q_out=_t(P, B, 8, 2, d),
             k_out=_t(P, B, 8, 1, d), v_out=_t(P, B, 8, 1, d), P=P, inv_freq=np.ones(64), q_weight=_t(d),
             k_weight=_t(d))
    a.update(over)
    return a


@pytest.mark.parametrize("over,msg", [
    ({}, "CUDA device"),
    ({"k_seq": _t(2, 1, 5, 2, 128)}, "k_seq must be"),
    ({"v_seq": _t(2, 1, 4, 2, 128, dtype=torch.float32)}, "v_seq must be"),
    ({"q_out": _t(2, 1, 4, 4, 128)}, "q_out must be"),
    ({"P": 4}, "leading dimension"),
    ({"q_weight": None}, "go together"),
    ({"v_out": None}, "go together"),
    ({"q_out": None}, "required"),
    ({"q_weight": _t(64)}, "q_weight must be"),
    ({"q_seq": _t(2, 4, 4, 128)}, "5-D"),
])
def test_binding_forward(over, msg):
    with pytest.raises(ValueError, match=msg):
        uly_py.ulysses_qkv_norm_rope_fwd(**_args(**over))


def test_binding_rotation_arguments():
    shape = (2, 1, 4)
    d, _ = uly_py._rope_desc(np.ones(32), None, None, False, shape)
    assert (d.rot_dim, d.num_axes, d.positions) == (64, 1, None)
    d, _ = uly_py._rope_desc([1.0] * 32, torch.zeros(3, 2, 1, 4, dtype=torch.int64), [0] * 16 + [2] * 16, True, shape)
    assert (d.rot_dim, d.num_axes, d.interleaved) == (64, 3, 1)
    assert uly_py._rope_desc(None, None, None, False, shape)[0].rot_dim == 0
    for bad in (dict(positions=torch.zeros(2, 1, 4, dtype=torch.int32)),
                dict(positions=torch.zeros(2, 1, 5, dtype=torch.int64)),
                dict(axis_of_freq=[0] * 31), dict(inv_freq=np.ones((2, 16)))):
        args = dict(inv_freq=np.ones(32), positions=None, axis_of_freq=None, interleaved=False, shape=shape)
        args.update(bad)
        with pytest.raises(ValueError):
            uly_py._rope_desc(**args)


def test_binding_token_strides():
    x = torch.zeros(2, 3, 4, 8, 64)
    stride = lambda t: uly_py._token_stride("x", t, 64)
    assert stride(x) == 512 and stride(x[:, :, :, 2:4]) == 512 and stride(x[..., 4:5, :]) == 512
    assert stride(torch.zeros(1, 1, 1, 8, 64)) == 512
    assert stride(torch.zeros(2, 1, 1, 8, 64)[:, :, :, :2]) == 512
    assert stride(x[:, :, ::2]) == 1024  # every second token is evenly spaced too
    for bad in (x.transpose(0, 1), x[:, :, :, ::2], x[:, :2], torch.zeros(2, 3, 4, 8, 128)[..., ::2]):
        with pytest.raises(ValueError, match="evenly spaced"):
            stride(bad)


def test_binding_backward():
    a = _args()
    dq, dk, dv = (torch.zeros_like(a[n]) for n in ("q_seq", "k_seq", "v_seq"))
    call = lambda **k: uly_py.ulysses_qkv_norm_rope_bwd(
        **{**dict(q_seq=a["q_seq"], k_seq=a["k_seq"], dq_out=a["q_out"], dk_out=a["k_out"], dv_out=a["v_out"],
                  dq_seq=dq, dk_seq=dk, dv_seq=dv, P=2, inv_freq=np.ones(64), q_weight=a["q_weight"],
                  k_weight=a["k_weight"]), **k})
    for over, msg in (({}, "CUDA device"), ({"q_seq": None}, "needs q_seq"), ({"dv_seq": None}, "go together"),
                      ({"q_weight": None, "k_weight": None, "dq_weight": _t(128)}, "no weight gradients"),
                      ({"dq_out": _t(2, 1, 4, 4, 128)}, "dq_out must be"), ({"dk_weight": _t(64)}, "dk_weight must be")):
        with pytest.raises(ValueError, match=msg):
            call(**over)


def test_binding_linear_ce():
    h, w, y = _t(2, 1, 8, 64), _t(100, 64), torch.zeros(2, 1, 8, dtype=torch.int64)
    f = uly_py.ulysses_sharded_linear_ce_loss
    for args, kw, msg in (((h, w, y, 2), {}, "CUDA device"), ((h, w, y, 4), {}, "hidden must be"),
                          ((h, _t(100, 72), y, 2), {}, "weight must be"), ((h, w.float(), y, 2), {}, "weight must be"),
                          ((h, w, y.int(), 2), {}, "labels"), ((h, w, y, 2), {"dhidden": _t(2, 1, 8, 72)}, "dhidden"),
                          ((h, w, y, 2), {"dweight": w.float()}, "dweight"),
                          ((h, w, y, 2), {"outputs": (torch.zeros(2), torch.zeros(2), torch.zeros(1))}, "outputs")):
        with pytest.raises(ValueError, match=msg):
            f(*args, **kw)
