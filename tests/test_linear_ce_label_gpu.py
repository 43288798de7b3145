"""The labels' terms of the fused LM-head loss, on the GPU against fp64.

The gradient of a row's logits is p - 1 at its label, most of it, and p at the
other words.  In bf16 the label's term is held in 32 bits and meets the weight's
and the hidden row as they were given; only the other words' terms have rounded
operands.  Tolerances count that, with u = 2^-24 (a rounding to bf16 is off by
2^-8 of the value at most):

* a logit is off by d_r <= (2 D + 2) u max_v <|h_r|, |w_v|> (products of bf16
  values are exact in fp32, their sum may truncate), a probability by the factor
  exp(2 d_r + 16 u) (exponential and sum);
* others: p is rounded once for dh, 2^-8; for dW h / S is rounded besides,
  (1 + 2^-8)^2 - 1;  in fp32 8 u altogether;
* label: 1 - p by the factor above and 8 u for its own steps; and since it is
  formed as a difference, 32 u of p;
* each gradient adds 2 K u of its terms for a sum of K and its own rounding.
"""
import pytest
import torch

from parity_utils import Guards, bytes_equal, log_errors
from test_linear_ce_gpu import BF16, FP32, U, full, make

pytestmark = pytest.mark.gpu


def run(uly, h, w, labels, **more):
    g = Guards()
    P, B, Np, D = h.shape
    dh, dw = g.empty(h.shape, h.dtype, float("nan")), g.empty(w.shape, w.dtype, float("nan"))
    ws = g.workspace(uly.ulysses_sharded_linear_ce_workspace_size(B, Np * P, D, len(w), P, True, h.dtype))
    ws.fill_(0xFF)  # NaN in every type where nothing is written
    loss = uly.ulysses_sharded_linear_ce_loss(h, w, labels, P, dhidden=dh, dweight=dw, workspace=ws, **more)
    torch.cuda.synchronize()
    g.check()
    return loss, dh, dw


def check(uly, h, w, labels, what):
    h, w, labels = h.cuda(), w.cuda(), labels.cuda()
    loss, dh, dw = run(uly, h, w, labels)
    assert uly.ulysses_get_device_status()[0] == 0
    y = torch.full_like(full(labels), -100)
    y[:, :-1] = full(labels)[:, 1:]
    y = y.reshape(-1)
    good = y >= 0
    y, rows, w64 = y[good], full(h).reshape(len(good), -1)[good].double(), w.double()
    T, D, V = max(len(y), 1), w.shape[1], len(w)
    at = torch.arange(len(y), device="cuda")
    x = rows @ w64.T
    total = (x.logsumexp(1) - x[at, y]).sum() / T
    d = (2 * D + 2) * U * (rows.abs() @ w64.abs().T).amax(1)
    tol = float((2 * d).max() + 32 * U * (1 + x.abs().max())) + 4 * U * float(total)
    assert abs(float(loss[2]) - float(total)) <= tol
    grow = torch.expm1(2 * d + 16 * U)[:, None]
    p = x.softmax(1)
    del x
    py = p[at, y]
    eps = torch.finfo(h.dtype).eps / 2
    errs = {}
    for name, got in (("dh", full(dh).reshape(len(good), -1)), ("dw", dw)):
        rounded = 8 * U if h.dtype == FP32 else (2.0 ** -8 if name == "dh" else (1 + 2.0 ** -8) ** 2 - 1)
        off = p * (grow + rounded * (1 + grow))
        off[at, y] = (1 - py) * (grow[:, 0] + 8 * U) + 32 * U * py
        g = p.clone()
        g[at, y] -= 1
        side = (lambda q: q @ w64 / T) if name == "dh" else (lambda q: q.T @ rows / T)
        size = (lambda q: q @ w64.abs() / T) if name == "dh" else (lambda q: q.T @ rows.abs() / T)
        ref = side(g)
        before = size(off) + 2 * (V if name == "dh" else T) * U * size(g.abs_() + off)
        if name == "dh":
            assert float(got[~good].abs().sum()) == 0.0
            got = got[good]
        over = (got.double() - ref).abs() - (eps * (ref.abs() + before) + before + 2.0 ** -133)
        assert float(over.max()) <= 0, (what, name, float(over.max()), int(over.argmax()))
        errs[name] = float((got.double() - ref).norm() / ref.norm())
    log_errors(f"linear ce labels {what}", **errs)
    return dh, dw


@pytest.mark.parametrize("P,B,N,D,V", [(1, 1, 2, 8, 3), (2, 1, 128, 328, 1500), (1, 1, 129, 328, 1500),
                                       (4, 2, 64, 128, 1000), (2, 3, 150, 200, 513), (1, 2, 260, 520, 777),
                                       (2, 1, 700, 264, 2049), (1, 1, 65, 1032, 4099), (1, 1, 3000, 72, 33),
                                       (3, 1, 4500, 136, 70), (1, 1, 600, 776, 50257)])
def test_label_terms(uly, P, B, N, D, V):
    """The same accuracy whatever the number of rows, tiles and runs of the contraction."""
    h, w, labels = make(P, B, N, D, V, BF16, seed=N + V)
    check(uly, h, w, labels, f"P{P} B{B} N{N} D{D} V{V}")


@pytest.mark.parametrize("kind", ["one word", "half one word", "ten words", "neighbours", "pairs", "certain"])
@pytest.mark.parametrize("N,D,V", [(1500, 136, 3001), (300, 264, 300), (4500, 1032, 300)])
def test_frequent_words(uly, kind, N, D, V):
    """Words that are the label of one, two, a few or all of 256 rows, whose terms go alone or summed."""
    h, w, labels = make(1, 1, N, D, V, BF16, ignore=0.05, seed=N + len(kind), lean=40.0 if kind == "certain" else 8.0)
    g = torch.Generator().manual_seed(3)
    kept = labels >= 0
    if kind == "one word":
        labels[kept] = V - 1
    elif kind == "half one word":
        labels[kept & (torch.rand(labels.shape, generator=g) < 0.5)] = 31
    elif kind == "ten words":
        labels[kept] = labels[kept] % 10 * 29
    elif kind == "neighbours":
        labels[kept] = 32 + labels[kept] % 33
    elif kind == "pairs":
        labels[0, 0] = torch.where(kept[0, 0], torch.arange(N) // 2 % V, labels[0, 0])
    one = check(uly, h, w, labels, f"{kind} N{N} D{D}")
    two = run(uly, h.cuda(), w.cuda(), labels.cuda())[1:]
    assert all(bytes_equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("V,N,dtype", [(300_000, 4500, BF16), (300_000, 4353, BF16), (300_000, 1400, FP32)])
def test_several_pieces_of_many_tiles(uly, V, N, dtype):
    """More rows than a piece holds, and more tiles of dW than CTA pairs: dW's tiles are carried in fp32
    from the first piece, some done whole and some in two runs, to the second, where all are done whole."""
    h, w, labels = make(1, 1, N, 24, V, dtype, ignore=0.0, seed=V + N)
    one = check(uly, h, w, labels, f"pieces V{V} N{N}")
    two = run(uly, h.cuda(), w.cuda(), labels.cuda())[1:]
    assert all(bytes_equal(a, b) for a, b in zip(one, two))
