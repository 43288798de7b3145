"""Pins of the fp64 norm/rotation and LM-head-loss oracle: closed forms,
finite differences and torch's autograd (CPU)."""
import numpy as np
import pytest
import torch

from oracle import norm_rope as nr
from oracle import aggregate_sharded_loss, per_rank_losses_batched, shift_labels_batched


def test_rotation_keeps_lengths_and_composes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 16))
    inv = 10.0 ** -np.arange(8)
    t1 = nr.angles(rng.integers(-10, 10, (1, 5)), inv)
    for inter in (False, True):
        y = nr.rotate(x, t1, inter)
        np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
        np.testing.assert_allclose(nr.rotate(y, t1, inter, back=True), x, atol=1e-13)
        # turning by p and then by q is turning by p + q
        t2 = nr.angles(np.full((1, 5), 7), inv)
        t12 = t1 + t2
        np.testing.assert_allclose(nr.rotate(y, t2, inter), nr.rotate(x, t12, inter), atol=1e-12)


def test_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8))
    inv = [1.0, 0.3, 0.05, 0.001]
    at = lambda x, p: nr.rotate(x, nr.angles(np.array([[p]]), inv), False)
    a = (at(q, 1_000_003) * at(k, 1_000_000)).sum()
    b = (at(q, 3) * at(k, 0)).sum()
    np.testing.assert_allclose(a, b, atol=1e-9)


def test_angles_at_far_and_negative_positions():
    p = np.array([[0, 1, -1, 10 ** 6, -10 ** 6, 2 ** 40]])
    t = nr.angles(p, [1.0, 0.1])
    big = np.longdouble(10) ** 6
    np.testing.assert_allclose(np.cos(t[3, 0]), float(np.cos(big)), atol=1e-9)
    np.testing.assert_allclose(t[1], [1.0, 0.1], atol=1e-12)
    np.testing.assert_allclose(t[2], [-1.0, -0.1], atol=1e-12)
    np.testing.assert_allclose(np.sin(t[4]), -np.sin(t[3]), atol=1e-9)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_gradient_against_differences(inter):
    rng = np.random.default_rng(2)
    x, w, dy = rng.standard_normal((4, 2, 16)), 1 + 0.3 * rng.standard_normal(16), rng.standard_normal((4, 2, 16))
    t = nr.angles(rng.integers(0, 100, (1, 4)), 10.0 ** -np.arange(6))  # 12 of 16 values turn
    f = lambda x, w: (nr.norm_rope(x, w, t, inter, 1e-6) * dy).sum()
    dx, dw = nr.norm_rope_bwd(x, w, t, dy, inter, 1e-6)
    h = 1e-6
    for i in [(0, 0, 0), (1, 1, 5), (3, 0, 15), (2, 1, 11)]:
        e = np.zeros_like(x)
        e[i] = h
        np.testing.assert_allclose((f(x + e, w) - f(x - e, w)) / (2 * h), dx[i], rtol=1e-6, atol=1e-8)
    for i in (0, 7, 15):
        e = np.zeros_like(w)
        e[i] = h
        np.testing.assert_allclose((f(x, w + e) - f(x, w - e)) / (2 * h), dw[i], rtol=1e-6, atol=1e-8)


def test_linear_ce_against_autograd_and_the_logits_oracle():
    rng = np.random.default_rng(3)
    B, N, D, V, P = 2, 12, 8, 21, 3
    h, w = rng.standard_normal((B, N, D)), rng.standard_normal((V, D))
    labels = rng.integers(0, V, (B, N))
    labels[rng.random((B, N)) < 0.3] = -100
    sh = shift_labels_batched(labels)
    per, counts, total, dh, dw, _ = nr.linear_ce(h, w, sh, P)
    losses, goods = per_rank_losses_batched(h @ w.T, sh, P)
    np.testing.assert_allclose(per, losses, rtol=1e-12)
    assert counts.tolist() == list(goods)
    np.testing.assert_allclose(total, aggregate_sharded_loss(losses, goods), rtol=1e-12)
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    loss = torch.nn.functional.cross_entropy((th @ tw.T).reshape(-1, V), torch.tensor(sh).reshape(-1),
                                             ignore_index=-100)
    loss.backward()
    np.testing.assert_allclose(float(loss), total, rtol=1e-12)
    np.testing.assert_allclose(th.grad.numpy(), dh, atol=1e-14)
    np.testing.assert_allclose(tw.grad.numpy(), dw, atol=1e-14)


def test_linear_ce_without_any_label():
    h, w = np.full((1, 4, 8), np.nan), np.ones((5, 8))
    per, counts, total, dh, dw, _ = nr.linear_ce(h, w, np.full((1, 4), -100), 2)
    assert per.tolist() == [0, 0] and counts.tolist() == [0, 0] and total == 0
    assert not dw.any()
