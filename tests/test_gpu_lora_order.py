"""Adapter calls whose kernels' parts have least to do before they meet, over and over: the bits
stay the same, and they are right."""
import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu


def _forward(d, **kw):
    return q8.q8_linear_w8a16_lora(d["x"], d["q"], d["s_w"], d["a"], d["b"], d["scale"], d["ids"],
                                   bias=d["bias"], **kw)


@pytest.mark.parametrize("M,N,K,R", [(1, 8, 16, 8), (5, 16, 16, 24), (16, 8, 16, 8),
                                     (16, 40, 64, 256), (16, 2560, 960, 8)])
@pytest.mark.parametrize("free", [0.0, 0.5, 1.0])
def test_rows_of_up_to_16_with_and_without_adapters(M, N, K, R, free):
    """A row without an adapter has its sums (zeros) at once, before the rest of its cluster may
    have started."""
    d = ref.make(M, N, K, R, 3, seed=60 + M + R, free=free, bias=True)
    y, h = _forward(d, out_dtype=torch.float32)
    wy, wh, by, bh = ref.forward(d)
    ref.near(h, wh, bh, "h")
    ref.near(y, wy, by, "y")
    assert not h[d["ids"] < 0].any()
    yb, hb = torch.empty_like(y), torch.empty_like(h)
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(300):
        yb.fill_(float("nan"))
        hb.fill_(float("nan"))
        if i % 2:                                   # nothing in front of the call, or the fills
            torch.cuda.synchronize()
        _forward(d, out_dtype=torch.float32, y=yb, h=hb)
        wrong += (yb != y).any() | (hb != h).any()
    assert int(wrong) == 0
    assert q8.q8_last_device_status() == q8.Q8_OK
