"""The LM head and sharded loss in one, on the GPU against the fp64 oracle.

Tolerances count roundings, u = 2^-24.  A product over K terms in fp32 is off
by at most 2 K u of the sum of its absolute terms (2: an accumulation may
truncate).  So a logit is off by d_r <= 2 D u max_v <|h_r|, |w_v|>, and
by 2 u of itself more where it is taken in units of log2; a probability by the
factor exp(2 d_r) and a row's loss by 2 d_r, plus 32 u of the values themselves
(exponential, sums of tile partials, logarithm).  The operands of the gradient
products are rounded: in bf16 the gradient of the logits times the softmax's
denominator S by 2^-8, with a scale in place of 1 / S that is off by 2^-8 at
most and makes up for it at the label, and for dW h times that scale by 2^-8 too
(calls of up to 128 rows: 2^-16);
in fp32 by less than 8 u altogether.  Each gradient adds its product's error and
its own rounding.
"""
import numpy as np
import pytest
import torch

import oracle.norm_rope as nr
from oracle import shift_labels_batched
from parity_utils import REL_TOL, Guards, bytes_equal, log_errors, rel_fro

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def make(P, B, N, D, V, dtype, ignore=0.2, lean=8.0, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(V, D, generator=g) / D ** 0.5 * scale).to(dtype)
    labels = torch.randint(0, V, (B, N), generator=g)
    h = torch.randn(B, N, D, generator=g)
    h = h + lean * torch.rand(B, N, 1, generator=g) * w[labels.roll(-1, 1)].float()
    labels[torch.rand(B, N, generator=g) < ignore] = -100
    shard = lambda t: t.reshape(B, P, N // P, *t.shape[2:]).transpose(0, 1).contiguous()
    return shard(h.to(dtype)), w, shard(labels)


def full(x):
    return x.transpose(0, 1).reshape(x.shape[1], -1, *x.shape[3:])


def run(uly, h, w, labels, dh=True, dw=True, **more):
    g = Guards()
    P, B, Np, D = h.shape
    outs = (g.empty((P,), FP32, float("nan")), g.empty((P,), torch.int64), g.empty((1,), FP32, float("nan")))
    grads = [g.empty(t.shape, t.dtype, float("nan")) if on else None for t, on in ((h, dh), (w, dw))]
    need = uly.ulysses_sharded_linear_ce_workspace_size(B, Np * P, D, w.shape[0], P, dh or dw, h.dtype)
    ws = g.workspace(need)
    ws.fill_(0xFF)  # NaN in every type where nothing is written
    uly.ulysses_sharded_linear_ce_loss(h.cuda(), w.cuda(), labels.cuda(), P, dhidden=grads[0], dweight=grads[1],
                                       workspace=ws, outputs=outs, **more)
    torch.cuda.synchronize()
    g.check()
    return outs, grads


def compare(outs, grads, h, w, labels, what, norm=True):
    P = h.shape[0]
    h64, w64 = full(h).double().numpy(), w.double().numpy()
    sh = shift_labels_batched(full(labels).numpy())
    per, counts, total, dh, dw, g = nr.linear_ce(h64, w64, sh, P)
    sl, sg, tot = (t.cpu().double().numpy() for t in outs)
    assert sg.astype(np.int64).tolist() == counts.tolist()
    good = (sh != -100).reshape(-1)
    rows = np.where(good[:, None], h64.reshape(-1, h64.shape[-1]), 0.0)
    D, V = w64.shape[1], w64.shape[0]
    size = (np.abs(rows) @ np.abs(w64).T).max(1)          # of a logit's terms
    d = (2 * D + 2) * U * size                            # of a logit
    tol_row = 2 * d + 32 * U * (1 + size)
    tol_loss = tol_row[good].max() if good.any() else 0.0
    assert np.abs(sl - per).max() <= tol_loss + 2 * U * np.abs(per).max(), (what, sl, per, tol_loss)
    assert abs(tot[0] - total) <= tol_loss + 4 * U * abs(total), (what, tot, total, tol_loss)
    T = max(int(good.sum()), 1)
    y = sh.reshape(-1)
    p = np.abs(g * T)
    p[np.arange(len(y))[good], y[good]] = 1 - p[good, y[good]]
    half = torch.finfo(h.dtype).eps / 2
    tag = "bf16" if h.dtype == BF16 else "fp32"
    # g's error: the probability's, then its rounding
    rounded = np.full(g.shape, 2.0 ** -7 + 2.0 ** -14 if tag == "bf16" else 8 * U)
    rounded[np.arange(len(y))[good], y[good]] = 8 * U
    dg0 = p * np.expm1(2 * d + 16 * U)[:, None] / T
    dg0 += rounded * (np.abs(g) + dg0)
    errs = {}
    for name, got, ref, side in (("dh", grads[0], dh.reshape(-1, D), lambda q: q @ np.abs(w64)),
                                 ("dw", grads[1], dw, lambda q: q.T @ np.abs(rows))):
        if got is None:
            continue
        got = (full(got.cpu()) if name == "dh" else got.cpu()).double().numpy().reshape(ref.shape)
        K = V if name == "dh" else T
        scaled = 2.0 ** (-16 if len(y) <= 128 else -8)  # h / S
        dg = dg0 + (scaled * (np.abs(g) + dg0) if name == "dw" and tag == "bf16" else 0.0)
        before = side(dg) + 2 * K * U * side(np.abs(g) + dg)
        tol = half * (np.abs(ref) + before) + before + 2.0 ** -133  # the last: below the smallest subnormal step
        assert np.isfinite(got).all(), (what, name)
        over = np.abs(got - ref) - tol
        assert (over <= 0).all(), (what, name, float(over.max()), np.unravel_index(over.argmax(), over.shape))
        errs[name] = rel_fro(got, ref)
        if norm and np.linalg.norm(ref) > 0:
            assert errs[name] <= REL_TOL[tag], (what, name, errs[name])
    log_errors(f"linear ce {what} {tag}", total=abs(tot[0] - total), **errs)


CASES = [
    # P, B, N, D, V, dtype
    (1, 1, 2, 8, 1, BF16),          # one row, one word: loss 0
    (1, 1, 2, 8, 3, FP32),
    (2, 1, 64, 64, 100, BF16),
    (4, 2, 64, 128, 1000, BF16),
    (4, 2, 64, 128, 1000, FP32),
    (3, 1, 99, 72, 257, BF16),      # nothing a multiple of a tile
    (2, 3, 150, 200, 513, BF16),
    (1, 1, 300, 100, 255, FP32),
    (1, 2, 260, 520, 777, FP32),
    (2, 1, 700, 264, 2049, BF16),   # several row tiles, column tiles and products of 64
    (1, 1, 65, 1032, 4099, BF16),
    (1, 1, 513, 256, 256, BF16),    # whole tiles and one row more
    (2, 1, 128, 328, 1500, BF16),   # the most rows whose h / S has two parts, and one more
    (1, 1, 129, 328, 1500, BF16),
]


@pytest.mark.parametrize("P,B,N,D,V,dtype", CASES)
def test_loss_and_gradients(uly, P, B, N, D, V, dtype):
    h, w, labels = make(P, B, N, D, V, dtype, seed=N + V)
    outs, grads = run(uly, h, w, labels)
    assert uly.ulysses_get_device_status()[0] == 0
    compare(outs, grads, h, w, labels, f"P{P} B{B} N{N} D{D} V{V}")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_one_gradient_or_none_gives_the_same_results(uly, dtype):
    h, w, labels = make(2, 1, 130, 136, 700, dtype, seed=5)
    outs, grads = run(uly, h, w, labels)
    for dh, dw in ((True, False), (False, True), (False, False)):
        o2, g2 = run(uly, h, w, labels, dh=dh, dw=dw)
        assert all(bytes_equal(a, b) for a, b in zip(outs, o2))
        for a, b in zip(grads, g2):
            assert b is None or bytes_equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_no_label_at_all(uly, dtype):
    h, w, labels = make(2, 1, 40, 64, 300, dtype, ignore=0.0)
    labels[:] = -100
    h[:] = float("nan")  # rows without a label are not read
    outs, grads = run(uly, h, w, labels)
    assert outs[0].cpu().tolist() == [0, 0] and outs[1].cpu().tolist() == [0, 0] and float(outs[2]) == 0.0
    assert float(grads[0].abs().max()) == 0.0 and float(grads[1].abs().max()) == 0.0
    assert uly.ulysses_get_device_status()[0] == 0


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_nan_rows_without_a_label_touch_nothing(uly, dtype):
    P, B, N = 2, 2, 90
    h, w, labels = make(P, B, N, 72, 333, dtype, ignore=0.4, seed=9)
    sh = torch.from_numpy(shift_labels_batched(full(labels).numpy())).reshape(B, P, N // P).transpose(0, 1)
    clean_outs, clean = run(uly, h, w, labels)
    h2 = h.clone()
    h2[sh == -100] = float("nan")
    outs, grads = run(uly, h2, w, labels)
    assert all(bytes_equal(a, b) for a, b in zip(list(clean_outs) + clean, list(outs) + grads))
    assert float(grads[0].cpu()[sh == -100].abs().max()) == 0.0


@pytest.mark.parametrize("N", [24, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_row_that_is_not_finite_stays_one_row(uly, dtype, bad, N):
    """A NaN or an infinity in a row with a label: its loss, its shard's and the total are NaN, and so
    are its dh and dW; the other rows' dh are as without it."""
    h, w, labels = make(2, 1, N, 72, 333, dtype, ignore=0.0, seed=23)
    _, clean = run(uly, h, w, labels)
    h[1, 0, 3, 5] = bad
    outs, grads = run(uly, h, w, labels)
    assert torch.isfinite(outs[0][0]) and torch.isnan(outs[0][1]) and torch.isnan(outs[2]).all()
    dh, dw = grads[0].cpu().reshape(N, -1), grads[1].cpu()
    row = N // 2 + 3
    assert torch.isnan(dh[row]).all()
    others = [i for i in range(N) if i != row]
    assert bytes_equal(dh[others], clean[0].cpu().reshape(N, -1)[others])
    assert torch.isnan(dw[:, 5]).all()
    assert uly.ulysses_get_device_status()[0] == 0


def test_a_shard_without_labels_and_invalid_labels(uly):
    h, w, labels = make(4, 1, 64, 64, 100, BF16, ignore=0.0, seed=11)
    labels[1] = -100
    labels[2, 0, 0] = -100  # the target of shard 1's last token
    outs, grads = run(uly, h, w, labels)
    assert uly.ulysses_get_device_status()[0] == 0
    assert outs[1].cpu().tolist()[1] == 0
    compare(outs, grads, h, w, labels, "empty shard")
    bad = labels.clone()
    bad[0, 0, 5] = 100  # out of range: ignored and reported
    bad[3, 0, 5] = -7
    outs, grads = run(uly, h, w, bad)
    assert uly.ulysses_get_device_status()[0] == 1
    bad[0, 0, 5] = bad[3, 0, 5] = -100
    compare(outs, grads, h, w, bad, "invalid labels")


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_logits_and_certain_rows(uly, dtype):
    """Logits in the hundreds: the maximum is taken out before any exponential; p reaches 1 and 0.
    A logit's own rounding moves a probability by percents there, so only the element-wise bound holds."""
    h, w, labels = make(1, 1, 80, 64, 600, dtype, lean=40.0, seed=13, scale=8.0)
    outs, grads = run(uly, h, w, labels)
    compare(outs, grads, h, w, labels, "large logits", norm=False)
    h, w, labels = make(1, 1, 80, 64, 600, dtype, lean=0.0, seed=14, scale=30.0)
    outs, grads = run(uly, h, w, labels)
    compare(outs, grads, h, w, labels, "large logits, wrong labels", norm=False)


@pytest.mark.parametrize("level", [[20, 60, -80, 0], [-70, -70, -71, -90], [120, 119.5, 40, -300], [30, -40, 32, 34],
                                   [0, -200, 0, -50]])
@pytest.mark.parametrize("N,dtype", [(100, BF16), (200, BF16), (100, FP32)])
def test_logits_that_differ_between_columns(uly, level, N, dtype):
    """Every 64 columns at a level of their own, from rows that scale it by 0 to 1.2: exponentials
    within e^33 are kept as they are, others relative to their columns' largest."""
    D = 64
    g = torch.Generator().manual_seed(17)
    u = torch.ones(D) / 8
    at = torch.tensor(level, dtype=torch.float32).repeat_interleave(64)[:, None]
    w = (at * u + torch.randn(len(at), D, generator=g) / 8)[:250].to(dtype)
    h = (torch.linspace(0, 1.2, N)[:, None] * u + torch.randn(N, D, generator=g) / 8)[None, None].to(dtype)
    labels = torch.randint(0, 250, (1, 1, N), generator=g)
    outs, grads = run(uly, h, w, labels)
    compare(outs, grads, h, w, labels, f"levels {level}", norm=False)
    for dh, dw in ((True, False), (False, True), (False, False)):
        o2, g2 = run(uly, h, w, labels, dh=dh, dw=dw)
        assert all(bytes_equal(a, b) for a, b in zip(outs, o2))
        assert all(b is None or bytes_equal(a, b) for a, b in zip(grads, g2))


@pytest.mark.parametrize("rows,dtype", [(8192, BF16), (8193, BF16), (8194, BF16), (20000, BF16), (9000, FP32),
                                        (65537, BF16), (65538, BF16), (140000, BF16), (70000, FP32)])
def test_pieces(uly, rows, dtype):
    """More rows with labels than one piece holds; the last row of a sequence has none."""
    h, w, labels = make(1, 1, rows, 24, 70, dtype, ignore=0.0, seed=rows)
    outs, grads = run(uly, h, w, labels)
    compare(outs, grads, h, w, labels, f"{rows} rows")
    # enough rows for three pieces, labels for one
    if rows >= 20000:
        labels[:, :, 2000:] = -100
        outs, grads = run(uly, h, w, labels)
        compare(outs, grads, h, w, labels, "one piece of three")


def test_same_bits_on_every_run_and_stream_and_graph(uly):
    h, w, labels = make(2, 2, 300, 264, 1111, BF16, seed=21)
    outs, grads = run(uly, h, w, labels)
    want = list(outs) + grads
    for _ in range(2):
        o, g = run(uly, h, w, labels)
        assert all(bytes_equal(a, b) for a, b in zip(want, list(o) + g))
    P, B, Np, D = h.shape
    hc, wc, lc = h.cuda(), w.cuda(), labels.cuda()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    dh, dw = torch.empty_like(hc), torch.empty_like(wc)
    got = uly.ulysses_sharded_linear_ce_loss(hc, wc, lc, P, dhidden=dh, dweight=dw, stream=side)
    side.synchronize()
    assert all(bytes_equal(a, b) for a, b in zip(want, list(got) + [dh, dw]))
    ws = torch.empty(uly.ulysses_sharded_linear_ce_workspace_size(B, Np * P, D, len(w), P, True, BF16),
                     dtype=torch.uint8, device="cuda")
    held, lab = torch.zeros_like(hc), torch.full_like(lc, -100)
    out = (torch.empty(P, device="cuda"), torch.empty(P, dtype=torch.int64, device="cuda"),
           torch.empty(1, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uly.ulysses_sharded_linear_ce_loss(held, wc, lab, P, dhidden=dh, dweight=dw, workspace=ws, outputs=out)
    held.copy_(hc)
    lab.copy_(lc)  # the number of good rows is read on the device
    graph.replay()
    torch.cuda.synchronize()
    assert all(bytes_equal(a, b) for a, b in zip(want, list(out) + [dh, dw]))


def test_agrees_with_the_loss_over_kept_logits(uly):
    """The same total as ulysses_sharded_ce_loss on logits formed first (fp32)."""
    h, w, labels = make(4, 1, 128, 64, 500, FP32, seed=31)
    outs, _ = run(uly, h, w, labels, dh=False, dw=False)
    logits = (h.double() @ w.double().T).float().cuda()
    sl, sg, tot = uly.ulysses_sharded_ce_loss(logits, labels.cuda(), 4)
    torch.cuda.synchronize()
    assert bytes_equal(outs[1], sg)
    assert abs(float(outs[2]) - float(tot)) <= 1e-5 * float(tot)


def _random_cases(n, seed=77):
    rng = np.random.default_rng(seed)
    out = []
    for _ in range(n):
        P = int(rng.choice([1, 2, 3, 4]))
        N = P * int(rng.integers(1, 400 // P))
        D = 8 * int(rng.integers(1, 60))
        V = int(rng.choice([int(rng.integers(2, 300)), int(rng.integers(300, 3000))]))
        out.append((P, int(rng.integers(1, 3)), N, D, V, BF16 if rng.integers(0, 2) else FP32))
    return out


@pytest.mark.parametrize("P,B,N,D,V,dtype", _random_cases(10))
def test_random_shapes(uly, P, B, N, D, V, dtype):
    test_loss_and_gradients(uly, P, B, N, D, V, dtype)


def test_two_calls_at_once(uly):
    """Two calls with workspaces of their own on two streams, attention on a third."""
    streams = [torch.cuda.Stream() for _ in range(3)]
    cases = []
    for seed in (1, 2):
        h, w, labels = (t.cuda() for t in make(2, 1, 1500, 264, 3001, BF16, seed=seed))
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        total = uly.ulysses_sharded_linear_ce_loss(h, w, labels, 2, dhidden=dh, dweight=dw)[2]
        cases.append((h, w, labels, [total.clone(), dh.clone(), dw.clone()]))
    q = torch.randn(2, 1, 1024, 8, 128, device="cuda").to(BF16)
    k = torch.randn(2, 1, 1024, 2, 128, device="cuda").to(BF16)
    o, lse = torch.empty_like(q), torch.empty(2, 1, 8, 1024, device="cuda")
    for _ in range(5):
        torch.cuda.synchronize()
        got = []
        for (h, w, labels, _), s in zip(cases, streams):
            dh, dw = torch.zeros_like(h), torch.zeros_like(w)
            s.wait_stream(torch.cuda.current_stream())
            total = uly.ulysses_sharded_linear_ce_loss(h, w, labels, 2, dhidden=dh, dweight=dw, stream=s)[2]
            got.append([total, dh, dw])
        uly.ulysses_attn_fwd(q, k, k, o, lse, stream=streams[2])
        torch.cuda.synchronize()
        assert uly.ulysses_get_device_status()[0] == 0
        for (_, _, _, want), g in zip(cases, got):
            assert all(bytes_equal(a, b) for a, b in zip(want, g))


def test_first_call_of_a_process_captured():
    """Nothing has to run before a capture: the kernels are set up on the host."""
    import os
    import subprocess
    import sys
    code = """
import torch, numpy as np, long_context_sequence_head_gb300 as uly
h, w = (torch.randn(*s, device="cuda").bfloat16() for s in ((2, 1, 100, 136), (500, 136)))
y = torch.randint(0, 500, (2, 1, 100), device="cuda")
grads = dict(dhidden=torch.empty_like(h), dweight=torch.empty_like(w))
ws = torch.empty(uly.ulysses_sharded_linear_ce_workspace_size(1, 200, 136, 500, 2, True, torch.bfloat16),
                 dtype=torch.uint8, device="cuda")
out = tuple(torch.empty(n, dtype=t, device="cuda") for n, t in ((2, torch.float32), (2, torch.int64), (1, torch.float32)))
x = [torch.randn(1, 1, 8, 4, 128, device="cuda").bfloat16() for _ in range(3)]
o = [torch.empty_like(t) for t in x]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    uly.ulysses_sharded_linear_ce_loss(h, w, y, 2, **grads, workspace=ws, outputs=out)
    uly.ulysses_qkv_norm_rope_fwd(*x, *o, 1, inv_freq=np.ones(64))
g.replay()
torch.cuda.synchronize()
total = uly.ulysses_sharded_linear_ce_loss(h, w, y, 2)[2]
assert torch.equal(total, out[2]) and uly.ulysses_get_device_status()[0] == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]


def test_the_longest_vocabulary(uly):
    """2^21 words, targets among the last; against fp64 on the GPU (tolerances as the bf16 norm bound)."""
    V, D = 1 << 21, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    h = torch.randn(1, 1, 40, D, device="cuda", generator=g).to(BF16)
    w = (torch.randn(V, D, device="cuda", generator=g) / 4).to(BF16)
    y = torch.randint(V - 10, V, (1, 1, 40), device="cuda", generator=g)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    total = uly.ulysses_sharded_linear_ce_loss(h, w, y, 1, dhidden=dh, dweight=dw)[2]
    rows, t = h[0, 0, :-1].double(), y[0, 0, 1:]
    x = rows @ w.double().T
    want = (x.logsumexp(1) - x[torch.arange(39), t]).mean()
    p = x.softmax(1)
    p[torch.arange(39), t] -= 1
    p /= 39
    assert abs(float(total) - float(want)) <= 1e-5 * float(want)
    assert rel_fro(dh[0, 0, :-1], (p @ w.double()).cpu()) <= REL_TOL["bf16"]
    assert rel_fro(dw, (p.T @ rows).cpu()) <= REL_TOL["bf16"]
