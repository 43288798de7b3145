"""Rows of a few elements in ulysses_residual_norm_*: their sizes and refusals on the
host (CPU; a plan for a type whose rows have no whole 16 bytes divided by zero), and
the shortest rows there are against fp64."""
import pytest
import torch

import test_residual_norm_gpu as whole
from test_window_norm_refusals import BF16, FP32, UNSUPPORTED, WORKSPACE, _norm_bwd, _norm_fwd


@pytest.mark.parametrize("N,P", [(1, 1), (64, 2), (4096, 4)])
def test_sizes(uly, N, P):
    """A row is a multiple of 16 bytes: 4 elements in fp32, 8 in bf16."""
    size = lambda D: uly.ulysses_residual_norm_workspace_size(3, N, D, P)
    for D in (1, 2, 3, 5, 6, 7, 9, 10, 11, 13, 8193, 8194, 8196, 16385, 16388):
        assert size(D) == 0, D
    for D in (4, 8, 12, 16, 20, 8192, 8200, 16384):
        assert size(D) >= 2 * 4 * D, D


def test_calls(uly):
    """What the types do not have rows for is refused; what they have gets as far as its workspace."""
    for D in (1, 2, 3, 4, 5, 6, 7, 12):
        for dt in (BF16, FP32):
            if dt == FP32 and D % 4 == 0:
                assert _norm_bwd(uly, D=D, dt=dt, wsb=0) == WORKSPACE
            else:
                assert _norm_fwd(uly, D=D, dt=dt) == _norm_bwd(uly, D=D, dt=dt) == UNSUPPORTED


CASES = [
    # B, N, P, D, gate, post, first
    (1, 1, 1, 4, "shared", True, False),
    (3, 10, 2, 4, "sequence", True, False),
    (2, 30000, 3, 4, "shared", True, False),
    (40, 70, 7, 4, "sequence", False, False),
    (1, 333, 1, 4, None, False, True),
    (3, 10, 2, 8, "sequence", True, False),
    (1, 40000, 2, 8, "shared", True, False),
    (5, 90, 3, 8, None, False, False),
    (2, 300, 2, 12, "sequence", True, False),
    (1, 7, 1, 20, "shared", True, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,N,P,D,gate,post,first", CASES)
def test_values(uly, B, N, P, D, gate, post, first, dtype):
    if D * dtype.itemsize % 16 == 0:
        whole.test_values_and_gradients(uly, B, N, P, D, gate, post, first, dtype)
        return
    t = torch.zeros(P, B, N // P, D, dtype=dtype, device="cuda")
    w, rstd = t[0, 0, 0].clone(), torch.zeros(2, P, B, N // P, device="cuda")
    with pytest.raises(RuntimeError, match="ULY_ERR_UNSUPPORTED"):
        uly.ulysses_residual_norm_fwd(t, None, None, t.clone(), P, w, rstd=rstd)
    with pytest.raises(RuntimeError, match="ULY_ERR_UNSUPPORTED"):
        uly.ulysses_residual_norm_bwd(t, None, None, t.clone(), t.clone(), None, P, w, rstd, dweight=w.clone())

