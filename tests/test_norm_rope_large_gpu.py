"""The normed forward and backward over more values than 32 bits count: the weight
gradients against fp64 sums, the last tokens as a call of their own gives them.

dw = sum of dy x r over R rows, with dy = x so that every term is positive and a
row that is left out shows.  A warp adds its share of the rows one by one and the
shares are joined in a few dozen steps: (R / 2432 + 128) u of the sum (2432: the
warps of the backward's fp32 launch on 152 SMs), 32 u for a term."""
import pytest
import torch

from parity_utils import bytes_equal

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_weight_gradients_past_32_bits(uly):
    n, heads, d = 1_500_000, (16, 4, 4), 128  # 4.6e9 values
    x = torch.empty(1, 1, n, sum(heads), d, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(2))
    parts = x.split(list(heads), dim=3)
    w = [torch.ones(d, device="cuda") for _ in range(2)]
    dy = [t.contiguous() for t in parts]
    dx, dw = torch.empty_like(x), [torch.empty(d, device="cuda") for _ in range(2)]
    common = dict(q_weight=w[0], k_weight=w[1])
    uly.ulysses_qkv_norm_rope_bwd(*parts[:2], *dy, *dx.split(list(heads), dim=3), 1, **common, dq_weight=dw[0],
                                  dk_weight=dw[1])
    tail = [t[:, :, -5:].contiguous() for t in parts]
    want = [torch.empty_like(t) for t in tail]
    uly.ulysses_qkv_norm_rope_bwd(*tail[:2], *tail, *want, 1, **common)
    assert all(bytes_equal(a[:, :, -5:], b) for a, b in zip(dx.split(list(heads), dim=3), want))
    assert uly.ulysses_get_device_status()[0] == 0
    for got, t, H in zip(dw, parts, heads):
        ref = torch.zeros(d, device="cuda", dtype=torch.float64)
        for c in t[0, 0].split(100_000):
            c = c.double()
            ref += (c * c * torch.rsqrt(c.square().mean(-1, keepdim=True) + 1e-6)).sum((0, 1))
        off = (got.double() - ref).abs()
        assert bool((off <= (n * H / 2432 + 160) * U * ref).all()), float((off / ref).max())
        assert n * H / 2432 * U < 1e-3  # a thousandth of the rows would show
    out = [torch.empty_like(t) for t in dy]
    del dx, dy
    uly.ulysses_qkv_norm_rope_fwd(*parts, *out, 1, **common)
    uly.ulysses_qkv_norm_rope_fwd(*tail, *want, 1, **common)
    assert all(bytes_equal(a[:, :, -5:], b) for a, b in zip(out, want))
