"""Cases and plain forms of a windowed decoder block's operators.

Two operators, each with its gradient, and the first with its form for one
new token:

* ``window_attn``: causal attention over a sliding window of each token's last
  keys, plus the first tokens of its document, which stay visible (sinks);
  forward and backward over head shards, with packed documents, and for one
  token of each sequence over a key/value cache.
* ``residual_norm``: what stands between two blocks of a model: the norm behind
  a block, its gate and residual scale, the sum with the residual stream and
  the norm before the next block; forward and backward.

``run`` computes the plain form (elementary torch operations in 32 bits), or,
with ``own`` set, makes the framework's calls on the same state.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
HIDDEN = 2560


# ------------------------------------------------------------------- cases

def _attn(name, direction, S, B, N, Hq, Hkv, window, sinks, d=128, dtype="bf16", docs=False):
    """S head shards of Hq query and Hkv key/value heads each."""
    return {"name": name, "op": "window_attn", "direction": direction, "S": S, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv,
            "d": d, "window": window, "sinks": sinks, "dtype": dtype, "docs": docs}


def _decode(name, S, B, Hq, Hkv, window, sinks, capacity, longest, shortest=1, d=128, dtype="bf16"):
    """One new token of each of B sequences of shortest..longest tokens; a cache of `capacity` slots."""
    return {"name": name, "op": "window_attn", "direction": "decode", "S": S, "B": B, "Hq": Hq, "Hkv": Hkv, "d": d,
            "window": window, "sinks": sinks, "capacity": capacity, "longest": longest, "shortest": shortest,
            "dtype": dtype}


def _norm(name, direction, B, N, P, D, gate="none", post=True, first=False, dtype="bf16"):
    """gate: none, shared (one vector [D]) or sequence (one for each sequence [B][D])."""
    return {"name": name, "op": "residual_norm", "direction": direction, "B": B, "N": N, "P": P, "D": D, "gate": gate,
            "post": post, "first": first, "dtype": dtype}


def listed():
    return [
        # a windowed layer of long-context training: 64K tokens on four head shards
        _attn("window_fwd_64k", "fwd", 4, 1, 65536, 8, 2, 4096, 4),
        _attn("window_bwd_64k", "bwd", 4, 1, 65536, 8, 2, 4096, 4),
        # a shorter sequence under a narrow window: few key tiles for every row
        _attn("window_fwd_8k", "fwd", 4, 1, 8192, 8, 2, 1024, 4),
        # packed documents, each with first tokens of its own
        _attn("window_bwd_docs", "bwd", 4, 1, 32768, 8, 2, 1024, 4, docs=True),
        # sizes that fill no tile: an odd group, a window and sinks that end inside tiles
        _attn("window_fwd_ragged", "fwd", 2, 2, 5003, 6, 2, 777, 130),
        # the fp32 path
        _attn("window_bwd_fp32", "bwd", 2, 1, 509, 4, 2, 100, 3, d=64, dtype="fp32"),
        # one new token of each of eight sequences over a rolling cache: latency alone
        _decode("window_decode_rolling", 1, 8, 32, 8, 1024, 4, capacity=1028, longest=9000),
        # serving: 32 long sequences whose caches hold every token
        _decode("window_decode_long", 1, 32, 32, 8, 4096, 4, capacity=40960, longest=40960, shortest=8192),
        # one new token of each of eight sequences: latency alone
        _norm("norm_fwd_new_token", "fwd", 8, 1, 1, HIDDEN),
        # the long-context training layer, a learned gate
        _norm("norm_fwd_64k", "fwd", 1, 65536, 4, HIDDEN, gate="shared"),
        _norm("norm_bwd_64k", "bwd", 1, 65536, 4, HIDDEN, gate="shared"),
        # a smaller model, ragged tokens, every sequence with a gate of its own
        _norm("norm_bwd_ragged", "bwd", 2, 3021, 3, 776, gate="sequence"),
    ]


LARGEST = 65536 * 4100 * 32 * 10 * 128  # operations of the largest attention pass


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    kind = rng.choice(["fwd", "bwd", "decode", "norm_fwd", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    d = 128 if dtype == "bf16" else rng.choice([64, 128])
    if kind.startswith("norm"):
        D = 8 * _log_int(rng, 8, 1024)
        P, B = rng.choice([1, 2, 4]), rng.choice([1, 1, 2, 5])
        # no more values than the largest listed case, half of that in 32 bits
        most = 65536 * HIDDEN // (D * (2 if dtype == "fp32" else 1))
        N = P * max(1, _log_int(rng, 1, min(131072, most)) // (P * B))
        return _norm("", kind[5:], B, N, P, D, gate=rng.choice(["none", "shared", "sequence"]),
                     post=rng.random() < 0.7, first=rng.random() < 0.1, dtype=dtype)
    S, Hkv, G = rng.choice([1, 1, 2, 4]), rng.choice([1, 2, 8]), rng.choice([1, 2, 3, 4, 8])
    sinks = rng.choice([0, 1, 4, 4, 60, 130, 300])
    window = _log_int(rng, 1, 8192)
    if kind == "decode":
        B = _log_int(rng, 1, 64)
        # no more slots than the largest listed case
        most = 32 * 4100 * 8 * 128 // (S * B * Hkv * d * (2 if dtype == "fp32" else 1))
        window = min(window, max(1, most - sinks))
        longest = _log_int(rng, 1, 20000)
        rolling = rng.random() < 0.5
        return _decode("", S, B, Hkv * G, Hkv, window, sinks,
                       sinks + window + rng.choice([0, 1, 17]) if rolling else longest + rng.choice([0, 5]), longest,
                       d=d, dtype=dtype)
    B = rng.choice([1, 1, 2])
    # no more products than the largest listed case, a 2000th of that in 32 bits
    ops = LARGEST / (2000 if dtype == "fp32" else 1) / (10 if kind == "bwd" else 4) / (S * B * Hkv * G * d)
    N = _log_int(rng, 1, min(65536, ops / (window + sinks) + math.sqrt(ops)))
    return _attn("", kind, S, B, N, Hkv * G, Hkv, window, sinks, d=d, dtype=dtype, docs=N >= 8 and rng.random() < 0.3)


def _cu_seqlens(case):
    """Bounds of the packed documents, the same for every seed: lengths from N/64 to N/4; None without."""
    if not case["docs"]:
        return None
    rng, N, cu = random.Random(case["N"]), case["N"], [0]
    while cu[-1] < N:
        cu.append(min(N, cu[-1] + rng.randint(max(1, N // 64), max(1, N // 4))))
    return cu


def _lens(case):
    """Tokens of each sequence, the new one included; the same for every seed."""
    rng = random.Random(case["B"] * 100003 + case["longest"])
    return [rng.randint(case["shortest"], case["longest"]) for _ in range(case["B"])]


def _pairs(case):
    """Allowed (query, key) pairs of one head."""
    W, S = case["window"], case["sinks"]
    cu = _cu_seqlens(case) or [0, case["N"]]
    total = 0
    for a, b in zip(cu, cu[1:]):
        i = torch.arange(1, b - a + 1)
        total += int((i.clamp(max=W) + (i - W).clamp(min=0, max=S)).sum())
    return total


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "residual_norm":
        return _prepare_norm(case, g)
    return _prepare_decode(case, g) if case["direction"] == "decode" else _prepare_attn(case, g)


def _qkv(case, g, n_q, n_k, sink_at):
    """Normed queries and keys with a direction that all queries share and the first keys answer to."""
    S, B, Hq, Hkv, d = (case[k] for k in ("S", "B", "Hq", "Hkv", "d"))
    dt = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    common = rand(Hkv, 1, d)
    q = (rand(S, B, n_q, Hkv, Hq // Hkv, d) + 0.5 * common).flatten(3, 4).to(dt)
    k = torch.randn(S, B, n_k, Hkv, d, device="cuda", generator=g, dtype=dt)
    v = torch.randn(S, B, n_k, Hkv, d, device="cuda", generator=g, dtype=dt)
    if len(sink_at):
        k[:, :, sink_at] = (k[:, :, sink_at].float() + 0.5 * common[:, 0]).to(dt)
    return q, k, v


def _prepare_attn(case, g):
    N = case["N"]
    cu = _cu_seqlens(case)
    starts = torch.zeros(N, dtype=torch.int64, device="cuda")  # of each token's document
    for a, b in zip(cu or [], (cu or [])[1:]):
        starts[a:b] = a
    first = torch.arange(N, device="cuda") - starts < case["sinks"]
    q, k, v = _qkv(case, g, N, N, first.nonzero().flatten())
    state = {"case": case, "q": q, "k": k, "v": v, "cu": cu, "starts": starts, "o": torch.empty_like(q),
             "lse": torch.empty(case["S"], case["B"], case["Hq"], N, dtype=torch.float32, device="cuda")}
    if case["direction"] == "bwd":
        o, lse = _plain_attn_fwd(state)
        state["o"].copy_(o)
        state["lse"].copy_(lse)
        state["dout"] = torch.randn(q.shape, device="cuda", generator=g).to(q.dtype)
        state["grads"] = [torch.empty_like(t) for t in (q, k, v)]
    return state


def _prepare_decode(case, g):
    q, k, v = _qkv(case, g, 1, case["capacity"], torch.arange(min(case["sinks"], case["capacity"])))
    return {"case": case, "q": q, "k": k, "v": v, "lens": torch.tensor(_lens(case), device="cuda"),
            "o": torch.empty_like(q),
            "lse": torch.empty(case["S"], case["B"], case["Hq"], 1, dtype=torch.float32, device="cuda")}


def _prepare_norm(case, g):
    B, N, P, D = (case[k] for k in ("B", "N", "P", "D"))
    dt = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    tokens = (P, B, N // P, D)
    # a residual stream: a few channels far larger than the others
    x = rand(*tokens) * (1 + 20 * (torch.rand(D, device="cuda", generator=g) < 0.01))
    state = {"case": case, "x": x.to(dt), "y": None, "weight": (1 + 0.2 * rand(D)).to(dt), "post": None, "gate": None,
             "scale": 1.0, "h": None, "z": torch.empty(tokens, dtype=dt, device="cuda"),
             "rstd": torch.empty(2, *tokens[:3], dtype=torch.float32, device="cuda")}
    if not case["first"]:
        state["y"] = (2 * rand(*tokens)).to(dt)
        state["scale"] = 0.5
        state["h"] = torch.empty_like(state["z"])
        if case["post"]:
            state["post"] = (1 + 0.2 * rand(D)).to(dt)
        if case["gate"] != "none":
            state["gate"] = (0.5 + 0.5 * rand(*((D,) if case["gate"] == "shared" else (B, D)))).to(dt)
    if case["direction"] == "bwd":
        state["rstd"].copy_(_plain_norm_fwd(state)[-1])
        state["dz"] = (1e-3 * rand(*tokens)).to(dt)
        state["dh"] = None if case["first"] else (1e-3 * rand(*tokens)).to(dt)
        state["dx"] = torch.empty_like(state["x"])
        state["dy"] = None if case["first"] else torch.empty_like(state["x"])
        state["dweights"] = [None if t is None else torch.empty_like(t)
                             for t in (state["weight"], state["post"], state["gate"])]
    return state


# --------------------------------------------------------------- one pass

def run(state):
    case = state["case"]
    if case["op"] == "residual_norm":
        forms = {"fwd": (_plain_norm_fwd, _own_norm_fwd), "bwd": (_plain_norm_bwd, _own_norm_bwd)}
    else:
        forms = {"fwd": (_plain_attn_fwd, _own_attn_fwd), "bwd": (_plain_attn_bwd, _own_attn_bwd),
                 "decode": (_plain_decode, _own_decode)}
    return forms[case["direction"]][1 if own else 0](state)


def _workspace(state, nbytes):
    if "workspace" not in state:
        state["workspace"] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device="cuda")
    return state["workspace"]


def _attn_workspace(state, for_bwd):
    import long_context_sequence_head_gb300 as uly
    if "workspace" in state:
        return state["workspace"]
    case = state["case"]
    return _workspace(state, uly.ulysses_window_attn_workspace_size(
        *(case[k] for k in ("B", "N", "Hq", "Hkv", "d", "S", "window", "sinks")),
        len(state["cu"]) - 1 if state["cu"] else 0, for_bwd, state["q"].dtype))


def _own_attn_fwd(state):
    import long_context_sequence_head_gb300 as uly
    case = state["case"]
    return uly.ulysses_window_attn_fwd(state["q"], state["k"], state["v"], state["o"], state["lse"], case["window"],
                                       case["sinks"], cu_seqlens=state["cu"], workspace=_attn_workspace(state, False))


def _own_attn_bwd(state):
    import long_context_sequence_head_gb300 as uly
    case = state["case"]
    return uly.ulysses_window_attn_bwd(state["q"], state["k"], state["v"], state["o"], state["lse"], state["dout"],
                                       *state["grads"], case["window"], case["sinks"], cu_seqlens=state["cu"],
                                       workspace=_attn_workspace(state, True))


def _own_decode(state):
    import long_context_sequence_head_gb300 as uly
    case = state["case"]
    if "workspace" not in state:
        _workspace(state, uly.ulysses_window_attn_decode_workspace_size(
            *(case[k] for k in ("B", "capacity", "Hq", "Hkv", "d", "S", "window", "sinks")), state["q"].dtype))
    return uly.ulysses_window_attn_decode(state["q"], state["k"], state["v"], state["lens"], state["o"], state["lse"],
                                          case["window"], case["sinks"], workspace=state["workspace"])


def _own_norm_fwd(state):
    import long_context_sequence_head_gb300 as uly
    return uly.ulysses_residual_norm_fwd(state["x"], state["y"], state["h"], state["z"], state["case"]["P"],
                                         state["weight"], post_weight=state["post"], gate=state["gate"],
                                         residual_scale=state["scale"], rstd=state["rstd"], eps=EPS)


def _own_norm_bwd(state):
    import long_context_sequence_head_gb300 as uly
    case = state["case"]
    if "workspace" not in state:
        _workspace(state, uly.ulysses_residual_norm_workspace_size(*(case[k] for k in ("B", "N", "D", "P"))))
    dw, dpost, dgate = state["dweights"]
    dx, dy = uly.ulysses_residual_norm_bwd(state["x"], state["y"], state["dh"], state["dz"], state["dx"], state["dy"],
                                           case["P"], state["weight"], state["rstd"], post_weight=state["post"],
                                           gate=state["gate"], residual_scale=state["scale"], dweight=dw,
                                           dpost_weight=dpost, dgate=dgate, workspace=state["workspace"])
    return dx, dy, dw, dpost, dgate


# ------------------------------------------------- plain form: attention

def _blocks(state):
    """Blocks of query rows: (r0, r1, key indices, allowed pairs [rows][keys])."""
    case = state["case"]
    N, W, S = case["N"], case["window"], case["sinks"]
    heads = case["S"] * case["B"] * case["Hq"]
    rows = 2048
    while rows > 16 and heads * rows * (rows + min(W, N) + S) > 1 << 29:
        rows //= 2
    cu = state["cu"] or [0, N]
    starts = state["starts"]
    for r0 in range(0, N, rows):
        r1 = min(N, r0 + rows)
        start = max(c for c in cu if c <= r0)
        lo = max(start, r0 - W + 1)
        j = torch.cat([torch.arange(start, min(start + S, lo), device="cuda"), torch.arange(lo, r1, device="cuda")])
        i = torch.arange(r0, r1, device="cuda")[:, None]
        s = starts[r0:r1, None]
        yield r0, r1, j, (j >= s) & (j <= i) & ((i - j < W) | (j - s < S))


def _grouped(t, Hkv):
    """[S][B][rows][Hq][d] -> [S][B][Hkv][group * rows][d]."""
    S, B, R, H, d = t.shape
    return t.float().view(S, B, R, Hkv, H // Hkv, d).permute(0, 1, 3, 4, 2, 5).reshape(S, B, Hkv, H // Hkv * R, d)


def _ungrouped(t, Hq, R):
    S, B, Hkv, _, d = t.shape
    return t.view(S, B, Hkv, Hq // Hkv, R, d).permute(0, 1, 4, 2, 3, 5).reshape(S, B, R, Hq, d)


def _probabilities(state, r0, r1, j, allowed):
    """Queries, keys and values of a block in 32 bits, its probabilities and their log-sum-exp."""
    case = state["case"]
    q = _grouped(state["q"][:, :, r0:r1], case["Hkv"])
    k, v = (state[n][:, :, j].float().transpose(2, 3) for n in ("k", "v"))
    s = (q @ k.transpose(3, 4)).mul_(1 / math.sqrt(case["d"]))
    s.masked_fill_(~allowed.repeat(case["Hq"] // case["Hkv"], 1), -math.inf)
    top = s.max(-1, keepdim=True).values
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return q, k, v, p.div_(total), top + total.log()


def _plain_attn_fwd(state):
    case = state["case"]
    o, lse = torch.empty_like(state["q"]), torch.empty_like(state["lse"])
    for r0, r1, j, allowed in _blocks(state):
        _, _, v, p, l = _probabilities(state, r0, r1, j, allowed)
        o[:, :, r0:r1] = _ungrouped(p @ v, case["Hq"], r1 - r0)
        lse[..., r0:r1] = l.view(case["S"], case["B"], case["Hq"], r1 - r0)
    return o, lse


def _plain_attn_bwd(state):
    case = state["case"]
    scale = 1 / math.sqrt(case["d"])
    dq = torch.empty_like(state["q"])
    dk, dv = (torch.zeros(state["k"].transpose(2, 3).shape, device="cuda") for _ in range(2))
    for r0, r1, j, allowed in _blocks(state):
        q, k, v, p, _ = _probabilities(state, r0, r1, j, allowed)
        do = _grouped(state["dout"][:, :, r0:r1], case["Hkv"])
        ds = do @ v.transpose(3, 4)
        ds = ds.sub_((p * ds).sum(-1, keepdim=True)).mul_(p)
        dq[:, :, r0:r1] = _ungrouped(ds @ k, case["Hq"], r1 - r0) * scale
        dk.index_add_(3, j, ds.transpose(3, 4) @ q)
        dv.index_add_(3, j, p.transpose(3, 4) @ do)
    return dq, (dk * scale).transpose(2, 3).to(dq.dtype).contiguous(), dv.transpose(2, 3).to(dq.dtype).contiguous()


def _plain_decode(state):
    case = state["case"]
    S, B, Hq, Hkv, d, W, sinks, C = (case[k] for k in ("S", "B", "Hq", "Hkv", "d", "window", "sinks", "capacity"))
    lens = state["lens"][:, None]
    recent = lens - W + torch.arange(W, device="cuda")  # the window's tokens
    first = torch.arange(sinks, device="cuda").expand(B, sinks)
    token = torch.cat([first, recent], 1)
    valid = torch.cat([first < lens - W, recent >= 0], 1)
    slot = torch.where(token < sinks, token, sinks + (token - sinks) % max(C - sinks, 1)).clamp(0, C - 1)
    rows = torch.arange(B, device="cuda")[:, None]
    k, v = (state[n][:, rows, slot].float().transpose(2, 3) for n in ("k", "v"))
    q = state["q"].float().view(S, B, Hkv, Hq // Hkv, d)
    s = (q @ k.transpose(3, 4)) / math.sqrt(d)
    s = s.masked_fill(~valid[:, None, None, :], -math.inf)
    top = s.max(-1, keepdim=True).values
    p = (s - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p / total) @ v
    return o.reshape(S, B, 1, Hq, d).to(state["q"].dtype), (top + total.log()).reshape(S, B, Hq, 1)


# ------------------------------------------------------ plain form: norms

def _gate32(state):
    """The gate, to be multiplied with [P][B][N/P][D]."""
    g = state["gate"]
    return 1.0 if g is None else g.float()[:, None] if g.dim() == 2 else g.float()


def _normed(t, w):
    r = torch.rsqrt(t.square().mean(-1, keepdim=True) + EPS)
    return t * r * w.float(), r[..., 0]


def _plain_norm_fwd(state):
    h, ones = state["x"].float(), torch.ones(state["x"].shape[:3], device="cuda")
    r2 = ones
    if state["y"] is not None:
        u = state["y"].float()
        if state["post"] is not None:
            u, r2 = _normed(u, state["post"])
        h = h + state["scale"] * _gate32(state) * u
    z, r1 = _normed(h, state["weight"])
    dt = state["x"].dtype
    return None if state["y"] is None else h.to(dt), z.to(dt), torch.stack([r1, r2])


def _plain_norm_bwd(state):
    x, w = state["x"].float(), state["weight"].float()
    dt, (r1, r2) = state["x"].dtype, state["rstd"][..., None]
    gate, scale, h = _gate32(state), state["scale"], x
    if state["y"] is not None:
        yhat = state["y"].float() * r2
        u = yhat if state["post"] is None else yhat * state["post"].float()
        h = x + scale * gate * u
    hhat, dz = h * r1, state["dz"].float()
    dw = (dz * hhat).sum(dim=(0, 1, 2)).to(dt)
    dz = dz * w
    t = r1 * (dz - hhat * (dz * hhat).mean(-1, keepdim=True))
    if state["dh"] is not None:
        t = t + state["dh"].float()
    if state["y"] is None:
        return t.to(dt), None, dw, None, None
    dgate, dpost = None, None
    if state["gate"] is not None:
        dgate = (scale * t * u).sum(dim=(0, 2) if state["gate"].dim() == 2 else (0, 1, 2)).to(dt)
    dy = scale * gate * t
    if state["post"] is not None:
        dpost = (dy * yhat).sum(dim=(0, 1, 2)).to(dt)
        dy = dy * state["post"].float()
        dy = r2 * (dy - yhat * (dy * yhat).mean(-1, keepdim=True))
    return t.to(dt), dy.to(dt), dw, dpost, dgate


# ------------------------------------------------------------------- work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "residual_norm":
        values = case["B"] * case["N"] * case["D"]
        tensors = (2 if case["first"] else 4) if case["direction"] == "fwd" else (3 if case["first"] else 6)
        return {"bytes": values * tensors * es, "flops": values * (8 if case["direction"] == "fwd" else 20)}
    S, B, Hq, Hkv, d = (case[k] for k in ("S", "B", "Hq", "Hkv", "d"))
    if case["direction"] == "decode":
        keys = sum(min(n, case["window"] + min(case["sinks"], max(0, n - case["window"]))) for n in _lens(case))
        return {"bytes": S * es * d * (2 * keys * Hkv + 2 * B * Hq), "flops": 4 * S * keys * Hq * d}
    rows, pairs = S * B * case["N"], S * B * Hq * _pairs(case)
    if case["direction"] == "fwd":
        return {"bytes": rows * (2 * (Hq + Hkv) * d * es + Hq * 4), "flops": 4 * d * pairs}
    return {"bytes": rows * (4 * (Hq + Hkv) * d * es + Hq * 4), "flops": 10 * d * pairs}


# ------------------------------------------------------- 64-bit definition

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "residual_norm":
        return _exact_norm(state)
    return _exact_decode(state) if case["direction"] == "decode" else _exact_attn(state)


def _exact_attn(state):
    case = state["case"]
    if work(case)["flops"] > 5e11:  # over about 20 seconds in 64 bits
        return None
    S, B, N, W, sinks, Hq, Hkv = (case[k] for k in ("S", "B", "N", "window", "sinks", "Hq", "Hkv"))
    bwd = case["direction"] == "bwd"
    at = torch.arange(N, device="cuda")
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(state["lse"].shape, dtype=torch.float64, device="cuda")
    grads = [torch.zeros(state[n].shape, dtype=torch.float64, device="cuda") for n in ("q", "k", "v")]
    step = 512
    while step > 8 and S * B * Hq * step * (step + W + sinks) > 1 << 27:
        step //= 2
    for a in range(0, N, step):
        rows = at[a:a + step]
        begin = state["starts"][rows]
        # every key that any of these rows sees, by the definition
        sees = (at <= rows[:, None]) & (at >= begin[:, None])
        sees &= (at > rows[:, None] - W) | (at < begin[:, None] + sinks)
        used = sees.any(0).nonzero().flatten()
        sees = sees[:, used]
        with torch.enable_grad():
            q, k, v = (t.double().requires_grad_(bwd) for t in (
                state["q"][:, :, rows], state["k"][:, :, used], state["v"][:, :, used]))
            heads = q.unflatten(3, (Hkv, Hq // Hkv))
            scores = torch.einsum("sbihgd,sbjhd->sbhgij", heads, k) / case["d"] ** 0.5
            scores = torch.where(sees, scores, -math.inf)
            out = torch.einsum("sbhgij,sbjhd->sbihgd", scores.softmax(-1), v).flatten(3, 4)
            if bwd:
                got = torch.autograd.grad(out, (q, k, v), state["dout"][:, :, rows].double())
                grads[0][:, :, rows] = got[0]
                grads[1][:, :, used] += got[1]
                grads[2][:, :, used] += got[2]
            else:
                o[:, :, rows], lse[..., rows] = out, scores.logsumexp(-1).flatten(2, 3)
    return tuple(grads) if bwd else (o, lse)


def _exact_decode(state):
    case = state["case"]
    S, C, W, sinks, G = case["S"], case["capacity"], case["window"], case["sinks"], case["Hq"] // case["Hkv"]
    o = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(state["lse"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        seen = [j for j in range(n) if j >= n - W or j < sinks]
        at = torch.tensor([j if j < sinks else sinks + (j - sinks) % (C - sinks) for j in seen], device="cuda")
        k, v = (state[t][:, b, at].double() for t in ("k", "v"))
        for h in range(case["Hq"]):
            s = torch.einsum("sd,sjd->sj", state["q"][:, b, 0, h].double(), k[:, :, h // G]) / case["d"] ** 0.5
            lse[:, b, h, 0] = s.logsumexp(1)
            o[:, b, 0, h] = torch.einsum("sj,sjd->sd", s.softmax(1), v[:, :, h // G])
    return o, lse


def _exact_norm(state):
    case = state["case"]
    bwd = case["direction"] == "bwd"
    with torch.enable_grad():
        x, y, w, post, gate = (None if t is None else t.double().requires_grad_(bwd) for t in (
            state["x"], state["y"], state["weight"], state["post"], state["gate"]))
        rms = lambda t: (t.pow(2).sum(-1, keepdim=True) / case["D"] + EPS).sqrt()  # noqa: E731
        h, after = x, torch.ones_like(x[..., :1])
        if y is not None:
            block = y
            if post is not None:
                after = rms(y)
                block = y / after * post
            if gate is not None:
                block = block * (gate.unsqueeze(1) if gate.dim() == 2 else gate)
            h = x + block * state["scale"]
        before = rms(h)
        z = h / before * w
        if not bwd:
            return None if y is None else h, z, torch.cat([1 / before, 1 / after], -1).movedim(-1, 0)
        leaves = [t for t in (x, y, w, post, gate) if t is not None]
        outs, cots = [z], [state["dz"].double()]
        if state["dh"] is not None:
            outs, cots = outs + [h], cots + [state["dh"].double()]
        grads = iter(torch.autograd.grad(outs, leaves, cots))
    return tuple(None if t is None else next(grads) for t in (x, y, w, post, gate))
