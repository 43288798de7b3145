"""A windowed decoder block with the calls a user makes: the first norm, packed QKV
projection, norm + rotation + move, sliding-window attention with sinks, move
back, output projection, norm behind the block with its gate and residual scale,
LM-head loss, and everything backward again, against torch's autograd in fp64 on
the CPU; and one token more through the same block over a cache.

Tolerance: ten stages round their outputs to the tensors' type (both norms, Q/K/V,
their norm and rotation, attention, its output's projection, and the same
backward), each by at most eps/2 of the value, so relative Frobenius errors stay
below 10 * 2^-8 in bf16; in fp32 each stage is within 1e-5 (the attention path's
own bound), together 1e-4.
"""
import numpy as np
import pytest
import torch

from parity_utils import log_errors, rel_fro

pytestmark = pytest.mark.gpu
EPS = 1e-6


def rms(t):
    return t / (t.square().mean(-1, keepdim=True) + EPS).sqrt()


def reference(leaves, labels, pos, inv, Hq, Hkv, d, cu, window, sinks, scale):
    """[B][N] of everything, unsharded, fp64, by autograd; returns the total, the gradients and the block's output."""
    x, w0, wqkv, wq, wk, wo, w1, w2, gate, w_lm = leaves = [t.double().requires_grad_(True) for t in leaves]
    B, N, _ = x.shape
    q, k, v = ((rms(x) * w0) @ wqkv.T).reshape(B, N, Hq + 2 * Hkv, d).split([Hq, Hkv, Hkv], dim=2)
    t = (pos.double()[..., None] * torch.from_numpy(inv))[:, :, None]

    def turn(h, w):
        h = rms(h) * w
        z = torch.complex(h[..., :d // 2], h[..., d // 2:]) * torch.polar(torch.ones_like(t), t)
        return torch.cat([z.real, z.imag], -1)

    q, k = turn(q, wq), turn(k, wk)
    k, v = (h.repeat_interleave(Hq // Hkv, dim=2) for h in (k, v))
    s = torch.einsum("bihd,bjhd->bhij", q, k) / d ** 0.5
    i = torch.arange(N)
    start = torch.tensor(cu)[torch.searchsorted(torch.tensor(cu[1:]), i, right=True)]
    i, j = i[:, None], i[None]
    allowed = (j <= i) & (j >= start[:, None]) & ((i - j < window) | (j - start[:, None] < sinks))
    o = torch.einsum("bhij,bjhd->bihd", s.masked_fill(~allowed, -torch.inf).softmax(-1), v)
    y = o.reshape(B, N, Hq * d) @ wo.T
    h = x + scale * gate[:, None] * (rms(y) * w2)
    z = rms(h) * w1
    logits = (z[:, :-1] @ w_lm.T).reshape(-1, w_lm.shape[0])
    total = torch.nn.functional.cross_entropy(logits, labels[:, 1:].reshape(-1), ignore_index=-100)
    # the stream goes on to the next block, too: a gradient of its own
    (total + (h * h.detach().sign()).sum() / 1e3).backward()
    return total.item(), [t.grad for t in leaves], h.detach(), z.detach()


def weights(E, Hq, Hkv, d, V, B, dtype, g):
    rand = lambda *s: torch.randn(*s, generator=g)
    H = Hq + 2 * Hkv
    return [t.to(dtype) for t in (
        1 + 0.2 * rand(E), rand(H * d, E) / E ** 0.5, 1 + 0.2 * rand(d), 1 + 0.2 * rand(d),
        rand(E, Hq * d) / (Hq * d) ** 0.5, 1 + 0.2 * rand(E), 1 + 0.2 * rand(E), 0.5 + 0.5 * rand(B, E),
        rand(V, E) / E ** 0.5 * 3)]


CASES = [
    (torch.float32, 2, 2, 96, 4, 2, 64, 300, [0, 40, 96], 20, 3),
    (torch.bfloat16, 2, 1, 384, 4, 2, 128, 700, [0, 100, 384], 60, 4),
    (torch.bfloat16, 4, 2, 512, 8, 4, 128, 1111, [0, 512], 130, 2),
]


@pytest.mark.parametrize("dtype,P,B,N,Hq,Hkv,d,V,cu,window,sinks", CASES)
def test_training_step(uly, dtype, P, B, N, Hq, Hkv, d, V, cu, window, sinks):
    E, Np, H, scale = 128, N // P, Hq + 2 * Hkv, 0.5
    g = torch.Generator().manual_seed(N)
    x = torch.randn(B, N, E, generator=g).to(dtype)
    ws = weights(E, Hq, Hkv, d, V, B, dtype, g)
    labels = torch.randint(0, V, (B, N), generator=g)
    labels[torch.rand(B, N, generator=g) < 0.2] = -100
    start = torch.tensor(cu)[torch.searchsorted(torch.tensor(cu[1:]), torch.arange(N), right=True)]
    pos = (torch.arange(N) - start)[None].expand(B, N)
    inv = 1e4 ** (-np.arange(d // 2) / (d // 2))
    total, want, ref_h, _ = reference([x] + ws, labels, pos, inv, Hq, Hkv, d, cu, window, sinks, scale)

    shard = lambda t: t.reshape(B, P, Np, *t.shape[2:]).transpose(0, 1).contiguous().cuda()
    full = lambda t: t.transpose(0, 1).reshape(B, N, *t.shape[3:])
    mm = lambda a, b: (a.float() @ b.float()).to(dtype)
    new = lambda h: torch.empty(P, B, N, h // P, d, dtype=dtype, device="cuda")
    seq = lambda h: torch.empty(P, B, Np, h, d, dtype=dtype, device="cuda")
    like = torch.empty_like
    w0, wqkv, wq, wk, wo, w1, w2, gate, w_lm = (t.cuda() for t in ws)
    xs, ys, ps = shard(x), shard(labels), shard(pos)
    rope = dict(inv_freq=inv, q_weight=wq, k_weight=wk, positions=ps, eps=EPS)
    rstd = [torch.empty(2, P, B, Np, device="cuda") for _ in range(2)]
    # forward
    z0 = like(xs)
    uly.ulysses_residual_norm_fwd(xs, None, None, z0, P, w0, rstd=rstd[0], eps=EPS)
    qkv = mm(z0, wqkv.T).reshape(P, B, Np, H, d)
    q, k, v = new(Hq), new(Hkv), new(Hkv)
    uly.ulysses_qkv_norm_rope_fwd(*qkv.split([Hq, Hkv, Hkv], dim=3), q, k, v, P, **rope)
    o, lse = new(Hq), torch.empty(P, B, Hq // P, N, device="cuda")
    uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks, cu_seqlens=cu)
    o_seq = seq(Hq)
    uly.ulysses_head_to_seq(o, o_seq, P)
    y = mm(o_seq.reshape(P, B, Np, Hq * d), wo.T)
    h, z = like(xs), like(xs)
    uly.ulysses_residual_norm_fwd(xs, y, h, z, P, w1, post_weight=w2, gate=gate, residual_scale=scale, rstd=rstd[1],
                                  eps=EPS)
    dz, dw_lm = like(z), like(w_lm)
    _, _, got_total = uly.ulysses_sharded_linear_ce_loss(z, w_lm, ys, P, dhidden=dz, dweight=dw_lm)
    # backward
    dh = (shard(ref_h.sign()) / 1e3).to(dtype)
    dx1, dy, dw1, dw2, dgate = like(xs), like(y), like(w1), like(w2), like(gate)
    uly.ulysses_residual_norm_bwd(xs, y, dh, dz, dx1, dy, P, w1, rstd[1], post_weight=w2, gate=gate,
                                  residual_scale=scale, dweight=dw1, dpost_weight=dw2, dgate=dgate)
    do_seq = mm(dy, wo).reshape(P, B, Np, Hq, d)
    dwo = dy.reshape(-1, E).T.float() @ o_seq.reshape(-1, Hq * d).float()
    do = new(Hq)
    uly.ulysses_seq_to_head(do_seq, do, P)
    dq, dk, dv = new(Hq), new(Hkv), new(Hkv)
    uly.ulysses_window_attn_bwd(q, k, v, o, lse, do, dq, dk, dv, window, sinks, cu_seqlens=cu)
    dqkv, dwq, dwk = like(qkv), like(wq), like(wk)
    uly.ulysses_qkv_norm_rope_bwd(*qkv.split([Hq, Hkv, Hkv], dim=3)[:2], dq, dk, dv,
                                  *dqkv.split([Hq, Hkv, Hkv], dim=3), P, **rope, dq_weight=dwq, dk_weight=dwk)
    dqkv = dqkv.reshape(P, B, Np, H * d)
    dz0 = mm(dqkv, wqkv)
    dwqkv = dqkv.reshape(-1, H * d).T.float() @ z0.reshape(-1, E).float()
    dx, dw0 = like(xs), like(w0)
    uly.ulysses_residual_norm_bwd(xs, None, dx1, dz0, dx, None, P, w0, rstd[0], dweight=dw0)
    torch.cuda.synchronize()
    assert uly.ulysses_get_device_status()[0] == 0
    tol = 10 * 2.0 ** -8 if dtype == torch.bfloat16 else 1e-4
    got = [full(dx), dw0, dwqkv, dwq, dwk, dwo, dw1, dw2, dgate, dw_lm]
    names = ("x", "w0", "wqkv", "wq", "wk", "wo", "w1", "w2", "gate", "w_lm")
    errs = {n: rel_fro(a, b) for n, a, b in zip(names, got, want)}
    errs["total"] = abs(float(got_total) - total) / total
    log_errors(f"window block {dtype} N{N}", **errs)
    assert all(e <= tol for e in errs.values()), errs


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [(torch.float32, 4, 2, 64), (torch.bfloat16, 8, 2, 128)])
def test_tokens_over_a_rolling_cache(uly, dtype, Hq, Hkv, d):
    """A prompt through the block's forward, then token by token over a rolling cache: the rows of the whole
    sequence's forward, by the same calls with one token a sequence."""
    B, N, steps, E, window, sinks, scale = 2, 70, 5, 128, 24, 3, 0.5
    H, C = Hq + 2 * Hkv, sinks + window + 1
    g = torch.Generator().manual_seed(4)
    x = torch.randn(B, N + steps, E, generator=g).to(dtype)
    ws = weights(E, Hq, Hkv, d, 8, B, dtype, g)
    inv = 1e4 ** (-np.arange(d // 2) / (d // 2))
    pos = torch.arange(N + steps)[None].expand(B, N + steps)
    labels = torch.zeros(B, N + steps, dtype=torch.int64)
    _, _, ref_h, ref_z = reference([x] + ws, labels, pos, inv, Hq, Hkv, d, [0, N + steps], window, sinks, scale)
    w0, wqkv, wq, wk, wo, w1, w2, gate, _ = (t.cuda() for t in ws)
    mm = lambda a, b: (a.float() @ b.float()).to(dtype)
    new = lambda n, h: torch.empty(1, B, n, h, d, dtype=dtype, device="cuda")

    def block(x, pos, attend):
        """x [1][B][n][E] through the block; attend(q, k, v) -> [1][B][n][Hq][d]."""
        n = x.shape[2]
        z0, h, z = (torch.empty_like(x) for _ in range(3))
        uly.ulysses_residual_norm_fwd(x, None, None, z0, 1, w0, eps=EPS)
        q, k, v = new(n, Hq), new(n, Hkv), new(n, Hkv)
        uly.ulysses_qkv_norm_rope_fwd(*mm(z0, wqkv.T).reshape(1, B, n, H, d).split([Hq, Hkv, Hkv], dim=3), q, k, v, 1,
                                      inv_freq=inv, q_weight=wq, k_weight=wk, positions=pos, eps=EPS, to_head=False)
        y = mm(attend(q, k, v).reshape(1, B, n, Hq * d), wo.T)
        uly.ulysses_residual_norm_fwd(x, y, h, z, 1, w1, post_weight=w2, gate=gate, residual_scale=scale, eps=EPS)
        return h, z

    kc, vc = (torch.full((1, B, C, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    slots = lambda at: torch.where(at < sinks, at, sinks + (at - sinks) % (C - sinks))

    def prompt(q, k, v):
        keep = torch.cat([torch.arange(sinks), torch.arange(N - window, N)]).cuda()
        kc[:, :, slots(keep)], vc[:, :, slots(keep)] = k[:, :, keep], v[:, :, keep]
        o, lse = torch.empty_like(q), torch.empty(1, B, Hq, N, device="cuda")
        return uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks)[0]

    def one(n):
        def attend(q, k, v):
            at = slots(torch.tensor([n], device="cuda"))
            kc[:, :, at], vc[:, :, at] = k, v
            o, lse = torch.empty_like(q), torch.empty(1, B, Hq, 1, device="cuda")
            lens = torch.full((B,), n + 1, dtype=torch.int64, device="cuda")
            return uly.ulysses_window_attn_decode(q, kc, vc, lens, o, lse, window, sinks)[0]
        return attend

    xs, ps = x[None].cuda(), pos[None].cuda()
    parts = [block(xs[:, :, :N].contiguous(), ps[:, :, :N].contiguous(), prompt)]
    for n in range(N, N + steps):
        parts.append(block(xs[:, :, n:n + 1].contiguous(), ps[:, :, n:n + 1].contiguous(), one(n)))
    assert uly.ulysses_get_device_status()[0] == 0
    tol = 6 * 2.0 ** -8 if dtype == torch.bfloat16 else 6e-5  # six stages, as above
    for got, want in ((torch.cat([p[0] for p in parts], 2)[0], ref_h), (torch.cat([p[1] for p in parts], 2)[0], ref_z)):
        assert rel_fro(got, want) <= tol
        assert rel_fro(got[:, N:], want[:, N:]) <= tol
