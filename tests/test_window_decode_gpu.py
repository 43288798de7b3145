"""ulysses_window_attn_decode against fp64, with whole and rolling caches.

Tolerances: window_ref.py's for O and lse (scores in fp32, P rounded to bf16 for
the second product, one rounding of the output), row by row."""
import math

import pytest
import torch

from parity_utils import Guards
from window_ref import check, reference

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32


def slot_of(j, sinks, C):
    return j if j < sinks else sinks + (j - sinks) % (C - sinks)


def seen(n, window, sinks):
    return [j for j in range(n) if j >= n - window or j < sinks]


def make(S, B, C, Hq, Hkv, d, lens, window, sinks, dtype, seed=0):
    """Queries, every token's key and value, and a cache whose unseen slots hold NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * C)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dtype)
    most = max(max(lens), 1)
    q, k, v = rand(S, B, 1, Hq, d), rand(S, B, most, Hkv, d), rand(S, B, most, Hkv, d)
    kc, vc = (torch.full((S, B, C, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    for b, n in enumerate(lens):
        for j in seen(n, window, sinks):
            kc[:, b, slot_of(j, sinks, C)] = k[:, b, j]
            vc[:, b, slot_of(j, sinks, C)] = v[:, b, j]
    return q, k, v, kc, vc, torch.tensor(lens, dtype=torch.int64, device="cuda")


def run(uly, q, kc, vc, lens, window, sinks, **kw):
    g = Guards()
    S, B, _, Hq, d = q.shape
    o, lse = g.full_like(q, float("nan")), g.empty((S, B, Hq, 1), FP32, float("nan"))
    ws = g.workspace(uly.ulysses_window_attn_decode_workspace_size(B, kc.shape[2], Hq, kc.shape[3], d, S, window, sinks,
                                                                   q.dtype))
    uly.ulysses_window_attn_decode(q, kc, vc, lens, o, lse, window, sinks, workspace=ws, **kw)
    g.check()
    return o, lse


def verify(got, q, k, v, lens, window, sinks):
    o, lse = got
    d = q.shape[4]
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[:, b] == 0).all() and (lse[:, b] == -math.inf).all()
            continue
        at = torch.tensor(seen(n, window, sinks), device="cuda")
        mask = torch.ones(1, len(at), dtype=torch.bool, device="cuda")
        one = slice(b, b + 1)
        val, err = reference_row(q[:, one], k[:, one][:, :, at], v[:, one][:, :, at], mask, 1 / math.sqrt(d),
                                 q.dtype == BF16)
        check(f"o of sequence {b}", o[:, one], val["o"], err["o"])
        check(f"lse of sequence {b}", lse[:, one], val["lse"], err["lse"])


def reference_row(q, k, v, mask, scale, rounded):
    """window_ref.reference for one query row over all given keys."""
    val, err = reference(q, k, v, torch.zeros_like(q), mask, scale, rounded)
    return val, err


CASES = [
    # S, B, C, Hq, Hkv, lens, window, sinks
    (1, 1, 1, 1, 1, [1], 1, 0),
    (1, 3, 40, 4, 2, [0, 1, 40], 10, 2),
    (1, 2, 5, 8, 2, [5, 3], 100, 300),                  # fewer tokens than sinks
    (2, 2, 300, 6, 2, [300, 130], 77, 3),
    (1, 4, 33, 4, 1, [33, 34, 500, 7], 30, 3),          # rolling, exactly sinks + window slots
    (1, 3, 40, 3, 1, [41, 1000003, 37], 20, 4),         # rolling with room to spare
    (1, 3, 5, 2, 1, [100, 6, 5], 1, 4),                 # a window of the token itself
    (1, 2, 9, 2, 2, [50, 9], 9, 0),                     # no sinks
    (1, 1, 2000, 32, 8, [1999], 1500, 4),
    (1, 2, 700, 16, 1, [700, 650], 700, 0),             # two groups of eight query heads
    (1, 1, 600, 20, 1, [580], 300, 130),                # three, the last half full
    (4, 2, 1030, 8, 2, [5000, 1029], 1024, 4),
]


@pytest.mark.parametrize("S,B,C,Hq,Hkv,lens,window,sinks", CASES)
@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP32, 128), (FP32, 64)], ids=["bf16", "fp32-128", "fp32-64"])
def test_against_reference(uly, S, B, C, Hq, Hkv, lens, window, sinks, dtype, d):
    if max(lens) > 10000:  # keep the tokens' values few: only those that are seen are made
        return long_sequence(uly, S, B, C, Hq, Hkv, lens, window, sinks, dtype, d)
    q, k, v, kc, vc, n = make(S, B, C, Hq, Hkv, d, lens, window, sinks, dtype)
    verify(run(uly, q, kc, vc, n, window, sinks), q, k, v, lens, window, sinks)
    assert uly.ulysses_get_device_status()[0] == 0


def long_sequence(uly, S, B, C, Hq, Hkv, lens, window, sinks, dtype, d):
    g = torch.Generator(device="cuda").manual_seed(C)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dtype)
    q = rand(S, B, 1, Hq, d)
    kc, vc = (torch.full((S, B, C, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
    kept = []
    for b, n in enumerate(lens):
        js = sorted(set(range(min(n, sinks))) | set(range(max(0, n - window), n)))
        k, v = rand(S, len(js), Hkv, d), rand(S, len(js), Hkv, d)
        for i, j in enumerate(js):
            kc[:, b, slot_of(j, sinks, C)], vc[:, b, slot_of(j, sinks, C)] = k[:, i], v[:, i]
        kept.append((k, v))
    o, lse = run(uly, q, kc, vc, torch.tensor(lens, device="cuda"), window, sinks)
    for b, (k, v) in enumerate(kept):
        one, mask = slice(b, b + 1), torch.ones(1, k.shape[1], dtype=torch.bool, device="cuda")
        val, err = reference_row(q[:, one], k[:, None], v[:, None], mask, 1 / math.sqrt(d), dtype == BF16)
        check("o", o[:, one], val["o"], err["o"])
        check("lse", lse[:, one], val["lse"], err["lse"])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_rolling_and_whole_caches_agree(uly, dtype):
    """The same tokens in a whole cache and in a rolling one."""
    lens, window, sinks = [900, 517, 1], 128, 4
    q, _, _, kc, vc, n = make(1, 3, 900, 8, 2, 128, lens, window, sinks, dtype)
    rolled = [torch.full((1, 3, 140, 2, 128), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    for b, m in enumerate(lens):
        for j in seen(m, window, sinks):
            for whole, roll in zip((kc, vc), rolled):
                roll[:, b, slot_of(j, sinks, 140)] = whole[:, b, j]
    o, lse = run(uly, q, kc, vc, n, window, sinks)
    o2, lse2 = run(uly, q, *rolled, n, window, sinks)
    # blocks are cut by the cache's size; one block a head here, so the order is the same
    assert torch.allclose(o.float(), o2.float(), atol=2.0 ** -7 if dtype == BF16 else 2.0 ** -20)
    assert torch.allclose(lse, lse2, atol=2.0 ** -18)


def test_last_row_of_the_forward(uly):
    """The decode of a sequence's last token is the forward's last row."""
    N, window, sinks = 700, 150, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn(2, 2, N, H, 128, device="cuda", generator=g).to(BF16) for H in (4, 2, 2))
    o, lse = torch.empty_like(q), torch.empty(2, 2, 4, N, device="cuda")
    uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks)
    n = torch.tensor([N, N], device="cuda")
    got, glse = run(uly, q[:, :, -1:].contiguous(), k, v, n, window, sinks)
    # each is within u |O| + (u + f) sum P|v| of the exact value: sum P|v| < 1.1 for these values, f < 2^-15
    assert (got.float() - o[:, :, -1:].float()).abs().max() <= 2 * (2.0 ** -8 * 1.1 + 2.0 ** -8 * 2)
    assert (glse - lse[..., -1:]).abs().max() <= 2.0 ** -15


def test_lengths_that_cannot_be(uly):
    """A negative length, or tokens that the cache cannot hold: o = 0, lse = -inf, a status; the others are served."""
    lens, window, sinks, C = [-1, 30, 41], 40, 2, 40
    q, k, v, kc, vc, _ = make(1, 3, C, 4, 2, 128, [1, 30, 40], window, sinks, BF16)
    assert uly.ulysses_get_device_status()[0] == 0
    o, lse = run(uly, q, kc, vc, torch.tensor(lens, device="cuda"), window, sinks)
    assert uly.ulysses_get_device_status()[0] == 1  # ULY_ERR_INVALID_ARG
    for b in (0, 2):
        assert (o[:, b] == 0).all() and (lse[:, b] == -math.inf).all()
    verify((o[:, 1:2], lse[:, 1:2]), q[:, 1:2], k[:, 1:2], v[:, 1:2], [30], window, sinks)
    assert uly.ulysses_get_device_status()[0] == 0


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
def test_streams_and_graphs(uly, dtype):
    """A captured step replays with the lengths, queries and cache as they are then."""
    window, sinks, C = 200, 4, 1000
    q, k, v, kc, vc, n = make(1, 2, C, 8, 2, 128, [1000, 900], 10 ** 6, sinks, dtype)
    side = torch.cuda.Stream()
    o, lse = torch.empty_like(q), torch.empty(1, 2, 8, 1, device="cuda")
    ws = torch.empty(uly.ulysses_window_attn_decode_workspace_size(2, C, 8, 2, 128, 1, window, sinks, dtype),
                     dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uly.ulysses_window_attn_decode(q, kc, vc, n, o, lse, window, sinks, workspace=ws)
    for lens in ([1000, 900], [777, 1], [0, 205]):
        n.copy_(torch.tensor(lens))
        ws.fill_(0x7f)
        graph.replay()
        torch.cuda.synchronize()
        verify((o, lse), q, k, v, lens, window, sinks)
        torch.cuda.synchronize()
        again = run(uly, q, kc, vc, n, window, sinks, stream=side)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_far_slots(uly):
    """Offsets past 2^31 elements in the cache."""
    C, Hkv, d = 1 << 21, 8, 128
    kc, vc = (torch.full((1, 2, C, Hkv, d), float("nan"), dtype=BF16, device="cuda") for _ in range(2))
    assert kc.numel() > 1 << 31
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randn(1, 2, 1, 16, d, device="cuda", generator=g).to(BF16)
    lens, window, sinks = [C, C - 5], 100, 3
    kept = []
    for b, n in enumerate(lens):
        at = torch.tensor(sorted(set(range(sinks)) | set(range(n - window, n))), device="cuda")
        rows = [torch.randn(len(at), Hkv, d, device="cuda", generator=g).to(BF16) for _ in range(2)]
        kc[0, b, at], vc[0, b, at] = rows
        kept.append(rows)
    o, lse = run(uly, q, kc, vc, torch.tensor(lens, device="cuda"), window, sinks)
    for b, (k, v) in enumerate(kept):
        mask = torch.ones(1, len(k), dtype=torch.bool, device="cuda")
        val, err = reference_row(q[:, b:b + 1], k[None, None], v[None, None], mask, 1 / math.sqrt(d), True)
        check("o", o[:, b:b + 1], val["o"], err["o"])
        check("lse", lse[:, b:b + 1], val["lse"], err["lse"])
