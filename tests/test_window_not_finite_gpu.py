"""What a key or value that is not finite may spoil in the windowed attention's forward:
the rows that include/ulysses.h names, and no others."""
import pytest
import torch

from test_window_attn_gpu import inputs

pytestmark = pytest.mark.gpu
BF16, FP32 = torch.bfloat16, torch.float32
TILE, NEAR = 128, 384


def may_spoil(j, N, window, sinks, cu):
    rows = set(range(max(0, j - NEAR), min(N, j + window + NEAR)))
    if sinks and window < N:
        for a, b in zip(cu[:-1], cu[1:]):
            first = min(a + max(sinks, 32), N) - 1
            if b > a and a // TILE <= j // TILE <= first // TILE:
                rows |= set(range(a, min(N, b + NEAR)))
    return rows


def forward(uly, q, k, v, window, sinks, cu):
    o, lse = torch.empty_like(q), torch.empty(q.shape[0], q.shape[1], q.shape[3], q.shape[2], device="cuda")
    uly.ulysses_window_attn_fwd(q, k, v, o, lse, window, sinks, cu_seqlens=cu)
    return o, lse


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (3, 3)], ids=["pairs", "singles"])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("window,sinks,cu,bad", [
    (100, 4, None, [10]),                                # behind the sinks, within their tile: every row
    (100, 4, None, [300, 2000]),
    (100, 40, [0, 1500, 3000, 6000], [1470, 4000]),      # in the tile that the next document's sinks begin in
    (64, 4, [0, 1500, 1620, 6000], [1530, 1615]),
    (700, 130, [0, 2500, 6000], [2700, 5999]),
    (1, 1, [0, 3000, 6000], [4500, 0]),
    (300, 0, [0, 2500, 6000], [2499, 3000]),
])
def test_reach(uly, Hq, Hkv, dtype, window, sinks, cu, bad):
    N = 6000
    q, k, v, _ = inputs(4, 2, N, Hq, Hkv, 128, dtype, seed=9)
    o, lse = forward(uly, q, k, v, window, sinks, cu)
    for which in ("k", "v"):
        for j in bad:
            k2, v2 = k.clone(), v.clone()
            (k2 if which == "k" else v2)[:, :, j] = float("nan") if j % 2 else float("inf")
            o2, lse2 = forward(uly, q, k2, v2, window, sinks, cu)
            spoilt = may_spoil(j, N, window, sinks, cu or [0, N])
            rows = torch.tensor([i for i in range(N) if i not in spoilt], dtype=torch.int64, device="cuda")
            assert torch.equal(o[:, :, rows], o2[:, :, rows]), (which, j)
            assert torch.equal(lse[..., rows], lse2[..., rows]), (which, j)
            assert uly.ulysses_get_device_status()[0] == 0
            if which == "v":
                assert not torch.isfinite(o2[:, :, j]).any()  # the row itself sees it
