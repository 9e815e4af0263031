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


@pytest.mark.parametrize("M", [1, 16, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_buffer_written_by_the_call_before(M, dtype):
    """One buffer, written by a call and read by the next one with nothing in between, its values
    other ones each time: checkpoints restored, taken again and used."""
    K, G, n = 960, 32, 4
    ds = [ref.make(M, 136, K, 8, 2, seed=70 + i) for i in range(n)]
    kept = [q8.q8_checkpoint_save(d["x"], G) for d in ds]
    x = torch.empty(M, K, dtype=dtype, device="cuda")
    c, e = torch.empty_like(kept[0][0]), torch.empty_like(kept[0][1])
    back = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    got = [[torch.empty_like(back), None, None] for _ in range(20 * n)]
    args = [ds[0][k] for k in ("q", "s_w", "a", "b", "scale", "ids")]
    want = [q8.q8_linear_w8a16_lora(q8.q8_checkpoint_load(*k), *args)[0] for k in kept]
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        q8.q8_checkpoint_load(*kept[i % n], y=x, out_dtype=dtype)
        q8.q8_checkpoint_save(x, G, codes=c, exps=e)
        q8.q8_checkpoint_load(c, e, y=out[0])
        q8.q8_checkpoint_load(c, e, y=back)
        out[1] = q8.q8_linear_w8a16_lora(back, *args)[0]
    for i, out in enumerate(got):
        assert torch.equal(out[0], q8.q8_checkpoint_load(*kept[i % n])), i
        assert torch.equal(out[1], want[i % n]), i
