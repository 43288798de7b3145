"""65 to 320 sinks whose documents have few tokens for each: their dK and dV keep the
precision of P and dS in two bf16 parts, whatever the tokens are (a rule on tokens a
sink once left them to the main kernel's one part)."""
import pytest
import torch

from test_window_attn_gpu import inputs, run
from test_window_sinks_gpu import BF16, sink_sums

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,window,sinks,cu", [
    (24000, 300, 200, None),                       # 120 tokens a sink
    (24000, 100, 300, None),                       # 80
    (24000, 64, 250, [0, 9000, 9050, 24000]),      # documents that share tiles, one shorter than its sinks
    (8192, 128, 130, None),                        # 63
    (8001, 1, 65, [0, 2000, 4100, 8001]),          # 31 to 60, by document
])
def test_few_tokens_a_sink(uly, N, window, sinks, cu):
    """Bounds of test_window_sinks_gpu.sink_sums: fp32 sums of at most 400 additions hold here too."""
    Hq, Hkv = 4, 2
    q, k, v, dout = inputs(1, 1, N, Hq, Hkv, 128, BF16, seed=11)
    shared = torch.randn(Hkv, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)) / 2
    q = (q.float() + shared.repeat_interleave(Hq // Hkv, 0)).to(BF16)
    k = k.float()
    for a, b in zip((cu or [0, N])[:-1], (cu or [0, N])[1:]):
        k[:, :, a:min(a + sinks, b)] += shared
    k = k.to(BF16)
    got = run(uly, q, k, v, dout, window, sinks, cu)
    worst = {}
    for a, b in zip((cu or [0, N])[:-1], (cu or [0, N])[1:]):
        if b - a > window + sinks:
            dk, dv, dk_err, dv_err, _ = sink_sums(q, k, v, dout, window, a, b, sinks)
            for name, want, err in (("dk", dk, dk_err), ("dv", dv, dv_err)):
                off = (got[name][0, 0, a:a + sinks].double().transpose(0, 1) - want).abs()
                worst[name, a] = float((off / err).max())
    print(worst)
    assert max(worst.values()) <= 1, worst
