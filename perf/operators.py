"""Cases and plain forms of the operators on either side of the attention path.

Two operators, each with its gradient:

* ``qkv_norm_rope``: RMS norm of every query and key head, the rotary position
  embedding (one position axis or several) and the seq->head move of Q, K and
  V; its backward takes dQ, dK and dV back to the sequence layout.
* ``linear_ce``: the LM head's product, the shifted next-token cross entropy
  and the good-token-weighted total, without keeping the logits, with the
  gradients of the hidden states and of the head's weight.

``run`` computes the plain form (elementary torch operations in 32 bits), or,
with ``own`` set, makes the framework's calls on the same state.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IGNORE = -100
VOCAB = 151936  # the vocabulary of the benchmark's loss measurement
HIDDEN = 2560
LARGEST_CE = 16384 * HIDDEN * VOCAB  # tokens x hidden x vocabulary of the largest listed case


# ------------------------------------------------------------------- cases

def _rope(name, direction, B, N, P, Hq, Hkv, d, dtype="bf16", axes=1, rot=None, interleaved=False, norm=True,
          packed=False, to_head=True, positions="none"):
    return {"name": name, "op": "qkv_norm_rope", "direction": direction, "B": B, "N": N, "P": P, "Hq": Hq,
            "Hkv": Hkv, "d": d, "dtype": dtype, "axes": axes, "rot": d if rot is None else rot,
            "interleaved": interleaved, "norm": norm, "packed": packed, "to_head": to_head, "positions": positions}


def _ce(name, B, N, P, D, V, dtype="bf16", grad=True, ignore=0.0):
    return {"name": name, "op": "linear_ce", "B": B, "N": N, "P": P, "D": D, "V": V, "dtype": dtype, "grad": grad,
            "ignore": ignore}


def listed():
    return [
        # one new token of each of eight sequences, far into a long context: latency alone
        _rope("rope_fwd_new_token", "fwd", 8, 1, 1, 32, 8, 128, to_head=False, positions="far"),
        # a training layer at 8K tokens, Q, K and V as views of one projection's output
        _rope("rope_fwd_8k_packed", "fwd", 1, 8192, 4, 32, 8, 128, packed=True),
        # the long-context training layer: 64K tokens on four shards, forward and backward
        _rope("rope_fwd_64k", "fwd", 1, 65536, 4, 32, 8, 128),
        _rope("rope_bwd_64k", "bwd", 1, 65536, 4, 32, 8, 128),
        # video and text tokens: positions on three axes, an odd number of tokens per shard
        _rope("rope_bwd_video", "bwd", 2, 10002, 2, 12, 4, 128, axes=3, packed=True, positions="grid"),
        # the fp32 path, packed documents, half of every head rotated, left in the sequence layout
        _rope("rope_bwd_fp32_docs", "bwd", 1, 4095, 3, 12, 6, 64, dtype="fp32", rot=32, to_head=False,
              positions="docs"),
        # a toy model's step: latency alone
        _ce("ce_grad_tiny", 1, 32, 2, 256, 1000, ignore=0.1),
        # the loss of a short text under a full-size head (evaluation): one read of the weight
        _ce("ce_loss_short", 1, 64, 1, HIDDEN, VOCAB, grad=False),
        # a training step's loss at 8K tokens, a third of them prompt tokens without a label
        _ce("ce_grad_8k", 1, 8192, 4, HIDDEN, VOCAB, ignore=0.3),
        # twice the tokens, all with labels
        _ce("ce_grad_16k", 1, 16384, 4, HIDDEN, VOCAB),
        # a smaller model whose sizes fill no tile: odd vocabulary, ragged tokens, batch of two
        _ce("ce_grad_ragged", 2, 3021, 3, 776, 50257, ignore=0.2),
        # the fp32 path
        _ce("ce_grad_fp32", 1, 2048, 4, 1024, 32000, dtype="fp32", ignore=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "bwd", "ce", "ce"])
    if kind != "ce":
        P = rng.choice([1, 1, 2, 4, 8])
        Hkv = P * rng.choice([1, 2])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        d = rng.choice([64, 128, 128])
        B = rng.choice([1, 1, 2, 5])
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        # no more values than the largest listed case, half of that in 32 bits
        most = 65536 * 48 * 128 // (B * P * (Hq + 2 * Hkv) * d * (2 if dtype == "fp32" else 1))
        N = P * _log_int(rng, 1, max(1, min(65536 // P, most)))
        axes = rng.choice([1, 1, 3])
        return _rope("", kind, B, N, P, Hq, Hkv, d, dtype=dtype, axes=axes, rot=rng.choice([d, d, d // 2, 16]),
                     interleaved=rng.random() < 0.25, norm=rng.random() < 0.85, packed=rng.random() < 0.5,
                     to_head=rng.random() < 0.7,
                     positions="grid" if axes == 3 else rng.choice(["none", "far", "docs"]))
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    P, B = rng.choice([1, 2, 3, 4]), rng.choice([1, 1, 2])
    D = 8 * _log_int(rng, 8, 512)
    V = _log_int(rng, 100, 160000)
    # no more products than the largest listed case, a sixteenth of that in 32 bits
    most = LARGEST_CE // (D * V * (16 if dtype == "fp32" else 1))
    N = P * max(1, _log_int(rng, 2, max(2, min(16384, most))) // (P * B))
    return _ce("", B, N, P, D, V, dtype=dtype, grad=rng.random() < 0.7, ignore=rng.choice([0.0, 0.1, 0.5]))


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (_prepare_rope if case["op"] == "qkv_norm_rope" else _prepare_ce)(case, g)


def _positions(case, g):
    """int64 [axes][P][B][N/P], or None for every token's index in its sequence."""
    B, N, P, axes = (case[k] for k in ("B", "N", "P", "axes"))
    if case["positions"] == "none":
        return None
    n = torch.arange(N, device="cuda").expand(axes, B, N)
    if case["positions"] == "far":  # later chunks of a long context, another place for each sequence
        pos = n + torch.randint(500_000, 1_000_000, (1, B, 1), device="cuda", generator=g)
    elif case["positions"] == "docs":  # packed documents: positions start again at every document
        starts = (torch.rand(1, B, N, device="cuda", generator=g) < 4.0 / (N + 4)).long() * n
        pos = n - starts.cummax(dim=2).values
    else:  # "grid": frames of 24 x 36 patches (time, height, width), then text where all axes agree
        video, rows, cols = N * 3 // 4, 24, 36
        frame = n[0, 0] // (rows * cols)
        at = torch.stack([frame, n[0, 0] // cols % rows, n[0, 0] % cols])[:axes].view(axes, 1, N)
        pos = torch.where(n < video, at, n - video + video // (rows * cols) + cols)
    return pos.reshape(axes, B, P, N // P).transpose(1, 2).contiguous()


def _views(case, x):
    """Q, K and V heads of [P][B][N/P][Hq + 2 Hkv][d]: views of one packed buffer, or tensors of their own."""
    parts = x.split([case["Hq"], case["Hkv"], case["Hkv"]], dim=3)
    return list(parts) if case["packed"] else [p.contiguous() for p in parts]


def _prepare_rope(case, g):
    B, N, P, Hq, Hkv, d = (case[k] for k in ("B", "N", "P", "Hq", "Hkv", "d"))
    dt = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    # a projection's output: heads of different scales
    x = rand(P, B, N // P, Hq + 2 * Hkv, d) * (0.5 + 2 * torch.rand(Hq + 2 * Hkv, 1, device="cuda", generator=g))
    state = {"case": case, "x": _views(case, x.to(dt)), "positions": _positions(case, g), "weights": (None, None)}
    del x
    if case["norm"]:
        state["weights"] = tuple((1 + 0.2 * rand(d)).to(dt) for _ in range(2))
    half = case["rot"] // 2
    state["inv_freq"] = (1e6 ** (-torch.arange(half, dtype=torch.float64) / half)).numpy()
    # frequencies in runs of one axis each, as (16, 24, 24) of 64
    cut = [half // 4, half // 4 + (half - half // 4) // 2]
    axis = (torch.arange(half) >= cut[0]).int() + (torch.arange(half) >= cut[1]).int()
    state["axis"] = axis.numpy() if case["axes"] == 3 else None
    shape = lambda H: (P, B, N, H // P, d) if case["to_head"] else (P, B, N // P, H, d)  # noqa: E731
    state["y"] = [torch.empty(shape(H), dtype=dt, device="cuda") for H in (Hq, Hkv, Hkv)]
    if case["direction"] == "bwd":
        state["y"] = [rand(*shape(H)).to(dt) for H in (Hq, Hkv, Hkv)]
        state["dx"] = _views(case, torch.empty(P, B, N // P, Hq + 2 * Hkv, d, dtype=dt, device="cuda"))
        state["dw"] = tuple(None if w is None else torch.empty_like(w) for w in state["weights"])
    return state


def _prepare_ce(case, g):
    B, N, P, D, V = (case[k] for k in ("B", "N", "P", "D", "V"))
    dt = DTYPES[case["dtype"]]
    weight = (torch.randn(V, D, device="cuda", generator=g) / math.sqrt(D)).to(dt)
    full = torch.randint(0, V, (B, N), device="cuda", generator=g)
    # hidden states as after a final norm, leaning to the next token's row: some tokens are well predicted
    lean = 12 * torch.rand(B, N, 1, device="cuda", generator=g)
    hidden = torch.randn(B, N, D, device="cuda", generator=g) + lean * weight[full.roll(-1, 1)].float()
    if case["ignore"]:  # prompts: runs of sixteen tokens without a label
        runs = torch.rand(B, N // 16 + 1, device="cuda", generator=g) < case["ignore"]
        full = full.masked_fill(runs.repeat_interleave(16, 1)[:, :N], IGNORE)
    shard = lambda t: t.reshape(B, P, N // P, *t.shape[2:]).transpose(0, 1).contiguous()  # noqa: E731
    state = {"case": case, "hidden": shard(hidden.to(dt)), "weight": weight, "labels": shard(full)}
    if case["grad"]:
        state["dhidden"], state["dweight"] = torch.empty_like(state["hidden"]), torch.empty_like(weight)
    return state


# --------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["op"] == "linear_ce":
        return _own_ce(state) if own else _plain_ce(state)
    if own:
        return _own_rope(state)
    return _plain_rope_fwd(state) if case["direction"] == "fwd" else _plain_rope_bwd(state)


def _own_rope(state):
    import long_context_sequence_head_gb300 as uly
    case = state["case"]
    common = dict(inv_freq=state["inv_freq"], q_weight=state["weights"][0], k_weight=state["weights"][1],
                  positions=state["positions"], axis_of_freq=state["axis"], interleaved=case["interleaved"],
                  to_head=case["to_head"])
    if case["direction"] == "fwd":
        return uly.ulysses_qkv_norm_rope_fwd(*state["x"], *state["y"], case["P"], **common)
    if "workspace" not in state:
        state["workspace"] = torch.empty(uly.ulysses_qkv_norm_rope_workspace_size(case["d"]), dtype=torch.uint8,
                                         device="cuda")
    dx = uly.ulysses_qkv_norm_rope_bwd(*state["x"][:2], *state["y"], *state["dx"], case["P"], **common,
                                       dq_weight=state["dw"][0], dk_weight=state["dw"][1],
                                       workspace=state["workspace"])
    return dx, state["dw"]


def _own_ce(state):
    import long_context_sequence_head_gb300 as uly
    case = state["case"]
    if "workspace" not in state:
        need = uly.ulysses_sharded_linear_ce_workspace_size(
            *(case[k] for k in ("B", "N", "D", "V", "P")), case["grad"], state["hidden"].dtype)
        state["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    grads = (state["dhidden"], state["dweight"]) if case["grad"] else (None, None)
    loss = uly.ulysses_sharded_linear_ce_loss(state["hidden"], state["weight"], state["labels"], case["P"],
                                              dhidden=grads[0], dweight=grads[1], workspace=state["workspace"])
    return loss, grads


def _cos_sin(state):
    """cos and sin of [P][B][N/P][rot/2] angles, formed in 64 bits."""
    case = state["case"]
    B, N, P = case["B"], case["N"], case["P"]
    inv = torch.from_numpy(state["inv_freq"]).cuda()
    pos = state["positions"]
    if pos is None:
        pos = torch.arange(N, device="cuda").view(1, P, 1, N // P).expand(1, P, B, N // P)
    pos = pos.permute(1, 2, 3, 0)
    if state["axis"] is not None:
        pos = pos[..., torch.from_numpy(state["axis"]).cuda().long()]
    angle = (pos.double() * inv).unsqueeze(3)
    return angle.cos().float(), angle.sin().float()


def _pairs(case, x):
    r = case["rot"]
    return (x[..., 0:r:2], x[..., 1:r:2]) if case["interleaved"] else (x[..., :r // 2], x[..., r // 2:r])


def _rotate(case, x, cos, sin):
    a, b = _pairs(case, x)
    y, (a_out, b_out) = x.clone(), (None, None)
    a_out, b_out = _pairs(case, y)
    a_out.copy_(a * cos - b * sin)
    b_out.copy_(b * cos + a * sin)
    return y


def _to_head(x, P):
    _, B, Np, H, d = x.shape
    return x.reshape(P, B, Np, P, H // P, d).permute(3, 1, 0, 2, 4, 5).reshape(P, B, P * Np, H // P, d)


def _to_seq(y, P):
    _, B, N, Hp, d = y.shape
    return y.reshape(P, B, P, N // P, Hp, d).permute(2, 1, 3, 0, 4, 5).reshape(P, B, N // P, P * Hp, d)


def _plain_rope_fwd(state):
    case, P = state["case"], state["case"]["P"]
    cos, sin = _cos_sin(state)

    def one(x, w):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        return _rotate(case, y, cos, sin).to(x.dtype)

    q, k, v = one(state["x"][0], state["weights"][0]), one(state["x"][1], state["weights"][1]), state["x"][2]
    return [_to_head(t, P) if case["to_head"] else t.clone() for t in (q, k, v)]


def _plain_rope_bwd(state):
    case, P = state["case"], state["case"]["P"]
    cos, sin = _cos_sin(state)

    def one(x, dy, w):
        g = _rotate(case, dy.float(), cos, -sin)
        if w is None:
            return g.to(x.dtype), None
        x32 = x.float()
        rstd = torch.rsqrt(x32.square().mean(-1, keepdim=True) + 1e-6)
        xhat = x32 * rstd
        dw = (g * xhat).sum(dim=(0, 1, 2, 3))
        g = g * w.float()
        dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        return dx.to(x.dtype), dw.to(w.dtype)

    dy = [_to_seq(t, P) if case["to_head"] else t for t in state["y"]]
    dq, dqw = one(state["x"][0], dy[0], state["weights"][0])
    dk, dkw = one(state["x"][1], dy[1], state["weights"][1])
    return (dq, dk, dy[2].clone()), (dqw, dkw)


def _targets(labels):
    """The label of each row's next token, in the sharded order [P][B][N/P]."""
    P, B, Np = labels.shape
    full = labels.transpose(0, 1).reshape(B, P * Np)
    nxt = torch.full_like(full, IGNORE)
    nxt[:, :-1] = full[:, 1:]
    return nxt.reshape(B, P, Np).transpose(0, 1)


def _plain_ce(state):
    h, w = state["hidden"], state["weight"]
    P, D = h.shape[0], h.shape[3]
    y = _targets(state["labels"]).reshape(P, -1)
    good = y >= 0
    n_good = good.sum(1)
    total_good = n_good.sum().clamp(min=1)
    rows, w32 = h.reshape(-1, D).float(), w.float()
    logits = rows @ w32.T
    top = logits.max(1, keepdim=True).values
    e = (logits - top).exp()
    s = e.sum(1, keepdim=True)
    at = y.reshape(-1, 1).clamp(min=0)
    ce = (s.log() + top - logits.gather(1, at)).reshape(P, -1) * good
    shard_loss = ce.sum(1) / n_good.clamp(min=1)
    total = ((shard_loss * n_good).sum() / total_good).reshape(1)
    if not state["case"]["grad"]:
        return (shard_loss, n_good, total), (None, None)
    del logits
    d = e.div_(s)
    d.scatter_add_(1, at, torch.full_like(s, -1.0))
    d.mul_((good.reshape(-1, 1) / total_good).float())
    return (shard_loss, n_good, total), ((d @ w32).to(h.dtype).reshape(h.shape), (d.T @ rows).to(w.dtype))


# ------------------------------------------------------------------- work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    tokens = case["B"] * case["N"]
    if case["op"] == "qkv_norm_rope":
        rotated = tokens * (case["Hq"] + case["Hkv"]) * case["d"]
        moved = tokens * case["Hkv"] * case["d"]
        at = 0 if case["positions"] == "none" else tokens * case["axes"] * 8
        bwd = case["direction"] == "bwd"
        # backward: the projection's output is read again, for the norm alone
        reads = rotated * ((2 if case["norm"] else 1) if bwd else 1) + moved
        return {"bytes": (reads + rotated + moved) * es + at, "flops": rotated * (16 if bwd else 8)}
    T, D, V = tokens * (1 - case["ignore"]), case["D"], case["V"]
    sides = 2 if case["grad"] else 1
    return {"bytes": sides * (tokens + V) * D * es + tokens * 8, "flops": (6 if case["grad"] else 2) * T * D * V}


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    state = prepare(case, seed)
    return _exact_rope(state) if case["op"] == "qkv_norm_rope" else _exact_ce(state)


def _exact_rope(state):
    case = state["case"]
    P, B, N, rot = case["P"], case["B"], case["N"], case["rot"]
    pos = state["positions"]
    if pos is None:
        pos = torch.arange(N, device="cuda").reshape(P, N // P)[None, :, None].expand(1, P, B, -1)
    axis = torch.zeros(rot // 2, dtype=torch.int64) if state["axis"] is None else torch.tensor(state["axis"]).long()
    turn = torch.tensor(state["inv_freq"], device="cuda")[None, None, None] * torch.index_select(
        pos, 0, axis.cuda()).movedim(0, -1)
    turn = torch.polar(torch.ones_like(turn), turn)[..., None, :]

    def forward(x, w):
        if w is not None:
            x = x / ((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w
        head, tail = x[..., :rot], x[..., rot:]
        pair = (-1, 2) if case["interleaved"] else (2, -1)
        last = -1 if case["interleaved"] else -2
        z = head.unflatten(-1, pair)
        z = torch.complex(z.select(last, 0), z.select(last, 1)) * turn
        return torch.cat([torch.stack([z.real, z.imag], last).flatten(-2), tail], -1)

    def move(x):
        if not case["to_head"]:
            return x
        heads = torch.cat(list(x.unbind(0)), 1)  # every token of a sequence
        return torch.stack(heads.chunk(P, 2))

    with torch.enable_grad():
        x = [t.double().requires_grad_(case["direction"] == "bwd") for t in state["x"]]
        w = [None if t is None else t.double().requires_grad_(case["direction"] == "bwd") for t in state["weights"]]
        y = [move(forward(x[0], w[0])), move(forward(x[1], w[1])), move(x[2])]
        if case["direction"] == "fwd":
            return y
        leaves = x + [t for t in w if t is not None]
        grads = torch.autograd.grad(y, leaves, [t.double() for t in state["y"]])
    return tuple(grads[:3]), (tuple(grads[3:]) if case["norm"] else (None, None))


def _exact_ce(state):
    case = state["case"]
    if case["B"] * case["N"] * case["D"] * case["V"] > 4e11:  # over about 20 seconds in 64 bits
        return None
    P, B, Np, D = state["hidden"].shape
    labels = torch.cat(list(state["labels"].unbind(0)), 1)
    nxt = torch.cat([labels[:, 1:], torch.full_like(labels[:, :1], IGNORE)], 1)
    nxt = torch.stack(nxt.chunk(P, 1)).flatten(1)
    keep = nxt != IGNORE
    counts = keep.sum(1)
    with torch.enable_grad():
        h = state["hidden"].double().requires_grad_(case["grad"])
        w = state["weight"].double().requires_grad_(case["grad"])
        logits = h.reshape(P * B * Np, D)[keep.flatten()] @ w.mT
        losses = logits.logsumexp(1) - logits[torch.arange(len(logits), device="cuda"), nxt[keep]]
        sums = torch.stack([p.sum() for p in losses.split(counts.tolist())])
        total = (sums.sum() / max(1, int(counts.sum()))).reshape(1)
        grads = torch.autograd.grad(total, (h, w)) if case["grad"] else (None, None)
    return (sums.detach() / counts.clamp(min=1), counts, total.detach()), tuple(grads)
