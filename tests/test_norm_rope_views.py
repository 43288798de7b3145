"""Views that ulysses_qkv_norm_rope_* refuse in the binding (CPU only): an
expanded tensor's tokens share their memory, so neither may its stride 0 reach
the library, for which 0 means contiguous, nor may tokens overlap."""
import pytest
import torch

import long_context_sequence_head_gb300 as uly

D = 64


@pytest.mark.parametrize("small,shape", [
    ((1, 1, 1, 4, D), (1, 1, 8, 4, D)),   # one token for all
    ((1, 1, 1, 4, D), (1, 8, 1, 4, D)),   # one start token for every sequence
    ((1, 1, 1, 4, D), (8, 1, 1, 4, D)),
    ((1, 1, 1, 4, D), (2, 3, 8, 4, D)),
    ((1, 1, 1, 1, D), (1, 1, 8, 1, D)),
])
def test_expanded_tokens_are_refused(small, shape):
    with pytest.raises(ValueError, match="memory of its own"):
        uly._token_stride("q_seq", torch.zeros(small).expand(shape), D)


def test_overlapping_tokens_are_refused():
    x = torch.zeros(8 * 128 + 256)
    with pytest.raises(ValueError, match="memory of its own"):
        uly._token_stride("q_seq", x.as_strided((1, 1, 8, 4, D), (1024, 1024, 128, D, 1)), D)


def test_partly_expanded_views_are_refused():
    for t in (torch.zeros(2, 1, 8, 4, D).expand(2, 3, 8, 4, D), torch.zeros(2, 3, 1, 4, D).expand(2, 3, 8, 4, D),
              torch.zeros(2, 3, 8, 1, D).expand(2, 3, 8, 4, D)):
        with pytest.raises(ValueError):
            uly._token_stride("q_seq", t, D)


def test_what_is_expanded_to_its_own_shape_passes():
    x = torch.zeros(1, 1, 8, 12, D)[:, :, :, :4]
    assert uly._token_stride("q_seq", x.expand(1, 1, 8, 4, D), D) == 12 * D
    assert uly._token_stride("q_seq", torch.zeros(1, 1, 1, 4, D).expand(1, 1, 1, 4, D), D) == 4 * D


class _Cuda(torch.Tensor):
    """A CPU tensor that says it lives on a device, so that a call gets as far as the strides."""

    def get_device(self):
        return 0


class _NoLaunch:
    def __init__(self, device, stream):
        pass

    __enter__ = lambda self: self
    __exit__ = lambda self, *exc: None
    raw = lambda self: 0
    scratch = lambda self, workspace, nbytes: torch.zeros(1)


class _Library:
    """Stands for the loaded library: no call may reach it."""

    def __getattr__(self, name):
        if name.endswith("workspace_size"):
            return lambda *a: 256
        return lambda *a: pytest.fail(f"{name} was called")


def _t(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16).as_subclass(_Cuda)


@pytest.mark.parametrize("direction,which", [("fwd", 0), ("fwd", 1), ("fwd", 2), ("bwd inputs", 0), ("bwd inputs", 1),
                                             ("bwd gradients", 0), ("bwd gradients", 1), ("bwd gradients", 2)])
def test_calls_with_expanded_views_do_not_reach_the_library(monkeypatch, direction, which):
    monkeypatch.setattr(uly, "load", lambda *a: _Library())
    monkeypatch.setattr(uly, "_Launch", _NoLaunch)
    B, heads = 4, (4, 2, 2)
    near = [_t(1, B, 1, H, D) for H in heads]
    far = [_t(1, B, 1, H, D) for H in heads]
    w = dict(q_weight=_t(D), k_weight=_t(D))
    bad = list(near)
    bad[which] = _t(1, 1, 1, heads[which], D).expand(1, B, 1, heads[which], D)  # one token for a batch
    with pytest.raises(ValueError, match="memory of its own"):
        if direction == "fwd":
            uly.ulysses_qkv_norm_rope_fwd(*bad, *far, 1, **w)
        elif direction == "bwd inputs":
            uly.ulysses_qkv_norm_rope_bwd(*bad[:2], *far, *near, 1, **w)
        else:
            uly.ulysses_qkv_norm_rope_bwd(*near[:2], *far, *bad, 1, **w)
