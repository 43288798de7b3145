"""The limit of a wait in the fused LM-head loss is that of one step's wait, not
of a whole product: a limit below a product's time, but far above a step's (a few
microseconds), reports nothing."""
import pytest
import torch

from parity_utils import bytes_equal

pytestmark = pytest.mark.gpu


def _time_ms(f):
    a, b = torch.cuda.Event(True), torch.cuda.Event(True)
    f()
    torch.cuda.synchronize()
    a.record()
    f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b)


@pytest.mark.parametrize("dtype,N,D,V", [(torch.bfloat16, 4096, 4096, 131072), (torch.float32, 2048, 2048, 65536)])
def test_a_limit_below_a_products_time(uly, dtype, N, D, V):
    g = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(1, 1, N, D, device="cuda", generator=g).to(dtype)
    w = (torch.randn(V, D, device="cuda", generator=g) / D ** 0.5).to(dtype)
    y = torch.randint(0, V, (1, 1, N), device="cuda", generator=g)
    got = []

    def call():
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        got.append((uly.ulysses_sharded_linear_ce_loss(h, w, y, 1, dhidden=dh, dweight=dw)[2], dh, dw))

    ms = _time_ms(call)  # three products and little else
    limit = 500_000
    assert ms / 3 > 2 * limit * 1e-6, ms
    try:
        uly.ulysses_set_wait_limit_ns(limit)
        call()
        torch.cuda.synchronize()
    finally:
        uly.ulysses_set_wait_limit_ns(250_000_000)  # the suite's
    assert uly.ulysses_get_device_status() == (0, 0)
    assert all(bytes_equal(a, b) for a, b in zip(got[0], got[-1]))
