"""ulysses_window_attn_decode where few heads share a long list of tokens, so that more
blocks than a cluster holds join their sums through the workspace, and where two calls
see the same tokens.  Tolerances: window_ref.py's, row by row."""
import math

import pytest
import torch

from test_window_decode_gpu import make, reference_row, run, seen, slot_of, verify
from window_ref import check

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32

CASES = [
    # S, B, C, Hq, Hkv, lens, window, sinks
    (1, 1, 4200, 32, 8, [4200], 4096, 4),             # one sequence
    (1, 2, 4100, 32, 8, [9001, 4100], 4096, 4),       # two, rolling
    (1, 2, 4100, 8, 8, [1, 17], 4096, 4),             # most blocks without a token
    (2, 1, 5000, 4, 1, [4999], 5000, 0),              # one KV head a shard: 64 blocks
    (1, 1, 3001, 16, 1, [2999], 2500, 130),           # two groups of query heads
    (1, 3, 4000, 3, 1, [0, 4000, 130], 3000, 33),     # an empty sequence between
    (1, 2, 4200, 5, 1, [4200, 4077], 1, 4000),        # sinks alone but for the token
]


@pytest.mark.parametrize("S,B,C,Hq,Hkv,lens,window,sinks", CASES)
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_through_the_workspace(uly, S, B, C, Hq, Hkv, lens, window, sinks, dtype):
    size = uly.ulysses_window_attn_decode_workspace_size(B, C, Hq, Hkv, 128, S, window, sinks, dtype)
    assert size >= 9 * S * B * Hq * (128 + 2) * 4  # sums of more blocks than a cluster's eight
    q, k, v, kc, vc, n = make(S, B, C, Hq, Hkv, 128, lens, window, sinks, dtype)
    verify(run(uly, q, kc, vc, n, window, sinks), q, k, v, lens, window, sinks)
    assert uly.ulysses_get_device_status()[0] == 0


def test_replayed_with_other_lengths(uly):
    """A captured call, its workspace full of something else each time; the same bits as an eager one's."""
    C, window, sinks = 4100, 4096, 4
    q, k, v, kc, vc, n = make(1, 1, C, 32, 8, 128, [C], 10 ** 6, sinks, BF16)
    o, lse = torch.empty_like(q), torch.empty(1, 1, 32, 1, device="cuda")
    ws = torch.empty(uly.ulysses_window_attn_decode_workspace_size(1, C, 32, 8, 128, 1, window, sinks, BF16),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uly.ulysses_window_attn_decode(q, kc, vc, n, o, lse, window, sinks, workspace=ws)
    for m in (C, 3, 0, 2000):
        n.fill_(m)
        ws.fill_(0x7f)
        graph.replay()
        torch.cuda.synchronize()
        verify((o, lse), q, k, v, [m], window, sinks)
        again = run(uly, q, kc, vc, n, window, sinks)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,lens,window,sinks,rolled", [(8, 2, [900, 517, 1], 128, 4, 140),
                                                             (32, 8, [4300], 4000, 100, 4100)])
def test_whole_and_rolling_caches_give_the_same_bits(uly, Hq, Hkv, lens, window, sinks, rolled, dtype):
    """Blocks are cut by min(C, sinks + window) tokens, the same for both caches, and see the
    same tokens in the same order."""
    C, B = max(lens), len(lens)
    q, k, v, kc, vc, n = make(1, B, C, Hq, Hkv, 128, lens, window, sinks, dtype)
    roll = [torch.full((1, B, rolled, Hkv, 128), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    for b, m in enumerate(lens):
        at = seen(m, window, sinks)
        to = [slot_of(j, sinks, rolled) for j in at]
        for whole, r in zip((kc, vc), roll):
            r[:, b, to] = whole[:, b, at]
    o, lse = run(uly, q, kc, vc, n, window, sinks)
    o2, lse2 = run(uly, q, *roll, n, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    verify((o, lse), q, k, v, lens, window, sinks)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_forward_and_decode_of_the_last_token(uly, dtype):
    """Each within its bounds of the exact row."""
    N, window, sinks = 700, 150, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(2, 2, N, H, 128, device="cuda", generator=g).to(dtype) for H in (4, 2, 2))
    o, lse = torch.empty_like(q), torch.empty(2, 2, 4, N, device="cuda")
    uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks)
    n = torch.tensor([N, N], device="cuda")
    last = q[:, :, -1:].contiguous()
    got, glse = run(uly, last, k, v, n, window, sinks)
    at = torch.tensor(seen(N, window, sinks), device="cuda")
    val, err = reference_row(last, k[:, :, at], v[:, :, at], torch.ones(1, len(at), dtype=torch.bool, device="cuda"),
                             1 / math.sqrt(128), dtype == BF16)
    for name, a, b in (("decode", got, glse), ("forward", o[:, :, -1:], lse[..., -1:])):
        check(name + " o", a, val["o"], err["o"])
        check(name + " lse", b, val["lse"], err["lse"])
