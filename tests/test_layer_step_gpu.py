"""A training step around the attention path with the calls a user makes:
packed QKV projection, norm + rotation + move, attention, move back, output
projection, LM-head loss, and everything backward again, against torch's
autograd in fp64 on the CPU.

Tolerance: eight stages round their outputs to the tensors' type (Q/K/V, their
norm and rotation, attention, its output's projection, and the same backward),
each by at most eps/2 of the value, so relative Frobenius errors stay below
8 * 2^-8 in bf16; in fp32 each stage is within 1e-5 (the attention path's own
bound), together 8e-5.
"""
import numpy as np
import pytest
import torch

from parity_utils import log_errors, rel_fro

pytestmark = pytest.mark.gpu
EPS = 1e-6


def reference(x, wqkv, wq, wk, wo, w_lm, labels, pos, inv, P, Hq, Hkv, d, cu):
    """[B][N] of everything, unsharded, fp64, by autograd; returns the total and the gradients."""
    leaves = [t.double().requires_grad_(True) for t in (x, wqkv, wq, wk, wo, w_lm)]
    x, wqkv, wq, wk, wo, w_lm = leaves
    B, N, _ = x.shape
    q, k, v = (x @ wqkv.T).reshape(B, N, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], dim=2)
    t = (pos.double()[..., None] * torch.from_numpy(inv))[:, :, None]

    def turn(h, w):
        h = h / (h.square().mean(-1, keepdim=True) + EPS).sqrt() * w
        z = torch.complex(h[..., :d // 2], h[..., d // 2:]) * torch.polar(torch.ones_like(t), t)
        return torch.cat([z.real, z.imag], -1)

    q, k = turn(q, wq), turn(k, wk)
    k, v = (h.repeat_interleave(Hq // Hkv, dim=2) for h in (k, v))
    s = torch.einsum("bihd,bjhd->bhij", q, k) / d ** 0.5
    doc = torch.searchsorted(torch.tensor(cu[1:]), torch.arange(N), right=True)
    allowed = (torch.arange(N)[:, None] >= torch.arange(N)) & (doc[:, None] == doc)
    o = torch.einsum("bhij,bjhd->bihd", s.masked_fill(~allowed, -torch.inf).softmax(-1), v)
    h = x + o.reshape(B, N, Hq * d) @ wo.T
    logits = (h[:, :-1] @ w_lm.T).reshape(-1, w_lm.shape[0])
    total = torch.nn.functional.cross_entropy(logits, labels[:, 1:].reshape(-1), ignore_index=-100)
    total.backward()
    return total.item(), [t.grad for t in leaves]


@pytest.mark.parametrize("dtype,P,N,Hq,Hkv,d,V,cu", [
    (torch.float32, 2, 48, 4, 2, 64, 300, [0, 20, 48]),
    (torch.bfloat16, 2, 256, 4, 2, 128, 700, [0, 100, 256]),
    (torch.bfloat16, 4, 320, 8, 4, 128, 1111, [0, 320]),
])
def test_step(uly, dtype, P, N, Hq, Hkv, d, V, cu):
    B, E, Np, H = 1, 128, N // P, Hq + 2 * Hkv
    g = torch.Generator().manual_seed(N)
    rand = lambda *s: torch.randn(*s, generator=g)
    x = rand(B, N, E).to(dtype)
    wqkv, wo = (rand(H * d, E) / E ** 0.5).to(dtype), (rand(E, Hq * d) / (Hq * d) ** 0.5).to(dtype)
    wq, wk = [(1 + 0.2 * rand(d)).to(dtype) for _ in range(2)]
    w_lm = (rand(V, E) / E ** 0.5 * 3).to(dtype)
    labels = torch.randint(0, V, (B, N), generator=g)
    labels[torch.rand(B, N, generator=g) < 0.2] = -100
    pos = torch.arange(N)[None] - torch.tensor(cu)[torch.searchsorted(torch.tensor(cu[1:]), torch.arange(N), right=True)][None]
    inv = 1e4 ** (-np.arange(d // 2) / (d // 2))
    total, want = reference(x, wqkv, wq, wk, wo, w_lm, labels, pos, inv, P, Hq, Hkv, d, cu)

    shard = lambda t: t.reshape(B, P, Np, *t.shape[2:]).transpose(0, 1).contiguous().cuda()
    full = lambda t: t.transpose(0, 1).reshape(B, N, *t.shape[3:])
    mm = lambda a, b: (a.float() @ b.float()).to(dtype)
    xs, ys, ps = shard(x), shard(labels), shard(pos)
    wqkv, wo, wq, wk, w_lm = (t.cuda() for t in (wqkv, wo, wq, wk, w_lm))
    rope = dict(inv_freq=inv, q_weight=wq, k_weight=wk, positions=ps, eps=EPS)
    new = lambda h: torch.empty(P, B, N, h // P, d, dtype=dtype, device="cuda")
    seq = lambda h: torch.empty(P, B, Np, h, d, dtype=dtype, device="cuda")
    # forward
    qkv = mm(xs, wqkv.T).reshape(P, B, Np, H, d)
    q, k, v = new(Hq), new(Hkv), new(Hkv)
    uly.ulysses_qkv_norm_rope_fwd(*qkv.split([Hq, Hkv, Hkv], dim=3), q, k, v, P, **rope)
    o, lse = new(Hq), torch.empty(P, B, Hq // P, N, device="cuda")
    uly.ulysses_attn_fwd(q, k, v, o, lse, cu_seqlens=cu)
    o_seq = seq(Hq)
    uly.ulysses_head_to_seq(o, o_seq, P)
    h = (xs.float() + o_seq.reshape(P, B, Np, Hq * d).float() @ wo.T.float()).to(dtype)
    dh, dw_lm = torch.empty_like(h), torch.empty_like(w_lm)
    _, _, got_total = uly.ulysses_sharded_linear_ce_loss(h, w_lm, ys, P, dhidden=dh, dweight=dw_lm)
    # backward
    do_seq = mm(dh, wo).reshape(P, B, Np, Hq, d)
    dwo = dh.reshape(-1, E).T.float() @ o_seq.reshape(-1, Hq * d).float()
    do = new(Hq)
    uly.ulysses_seq_to_head(do_seq, do, P)
    dq, dk, dv = new(Hq), new(Hkv), new(Hkv)
    uly.ulysses_attn_bwd(q, k, v, o, lse, do, dq, dk, dv, cu_seqlens=cu)
    dqkv, dwq, dwk = torch.empty_like(qkv), torch.empty_like(wq), torch.empty_like(wk)
    uly.ulysses_qkv_norm_rope_bwd(*qkv.split([Hq, Hkv, Hkv], dim=3)[:2], dq, dk, dv,
                                  *dqkv.split([Hq, Hkv, Hkv], dim=3), P, **rope, dq_weight=dwq, dk_weight=dwk)
    dqkv = dqkv.reshape(P, B, Np, H * d)
    dx = dh.float() + dqkv.float() @ wqkv.float()
    dwqkv = dqkv.reshape(-1, H * d).T.float() @ xs.reshape(-1, E).float()
    torch.cuda.synchronize()
    assert uly.ulysses_get_device_status()[0] == 0
    tol = 8 * 2.0 ** -8 if dtype == torch.bfloat16 else 8e-5
    got = [full(dx), dwqkv, dwq, dwk, dwo, dw_lm]
    errs = {n: rel_fro(a, b) for n, a, b in zip(("x", "wqkv", "wq", "wk", "wo", "w_lm"), got, want)}
    errs["total"] = abs(float(got_total) - total) / total
    log_errors(f"layer step {dtype} N{N}", **errs)
    assert all(e <= tol for e in errs.values()), errs
