"""Several position axes without positions: the token's index stands on every
axis, so that a text alone runs through a model whose frequencies have axes."""
import numpy as np
import pytest
import torch

import long_context_sequence_head_gb300 as uly_py
from parity_utils import bytes_equal

SHAPE = (2, 1, 4)


@pytest.mark.parametrize("axis,axes", [([0, 1, 2, 0], 3), ([0, 0, 0, 0], 1), ([7, 0, 0, 0], 8)])
def test_axes_without_positions(axis, axes):
    desc, _ = uly_py._rope_desc(np.ones(4), None, axis, False, SHAPE)
    assert (desc.positions, desc.num_axes) == (None, axes)


def test_axes_that_are_not_there():
    """Positions say how many axes there are; without them the library refuses more than eight, and negative ones."""
    one = torch.zeros(SHAPE, dtype=torch.int64)
    assert uly_py._rope_desc(np.ones(4), one, [0, 1, 2, 0], False, SHAPE)[0].num_axes == 1
    assert uly_py._rope_desc(np.ones(4), None, [8, 0, 0, 0], False, SHAPE)[0].num_axes == 9
    assert uly_py._rope_desc(np.ones(4), None, [-1, -1, -1, -1], False, SHAPE)[0].num_axes == 1
    assert uly_py._rope_desc([], None, [], False, SHAPE)[0].num_axes == 1


@pytest.mark.gpu
@pytest.mark.parametrize("axes", [2, 3, 8])
def test_as_with_the_index_on_every_axis(uly, axes):
    P, B, Np, H, d = 2, 2, 21, 4, 128
    g = torch.Generator(device="cuda").manual_seed(axes)
    x = [torch.randn(P, B, Np, H, d, device="cuda", generator=g).to(torch.bfloat16) for _ in range(3)]
    w = dict(q_weight=torch.ones(d, device="cuda", dtype=torch.bfloat16),
             k_weight=torch.ones(d, device="cuda", dtype=torch.bfloat16))
    common = dict(inv_freq=1e4 ** (-np.arange(64) / 64), axis_of_freq=np.arange(64) % axes, **w)
    pos = torch.arange(P * Np, device="cuda").view(1, P, 1, Np).expand(axes, P, B, Np).contiguous()
    far = lambda: [torch.empty(P, B, P * Np, H // P, d, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    out = [far(), far()]
    back = [[torch.empty_like(t) for t in x] for _ in range(2)]
    for i, positions in enumerate((None, pos)):
        uly.ulysses_qkv_norm_rope_fwd(*x, *out[i], P, positions=positions, **common)
        uly.ulysses_qkv_norm_rope_bwd(*x[:2], *out[0], *back[i], P, positions=positions, **common)
    torch.cuda.synchronize()
    assert all(bytes_equal(a, b) for a, b in zip(out[0] + back[0], out[1] + back[1]))
    plain = [torch.empty_like(t) for t in out[0]]
    uly.ulysses_qkv_norm_rope_fwd(*x, *plain, P, inv_freq=common["inv_freq"], **w)  # one axis: the same angles
    assert all(bytes_equal(a, b) for a, b in zip(out[0], plain))
