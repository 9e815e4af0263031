"""8-bit activation checkpoints against their definition bit for bit, and the weight gradient
from them against 64 bits; a training step of the adapter linear that uses all of it."""
import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu


def _same(x, G):
    codes, exps = q8.q8_checkpoint_save(x, G)
    wc, we = ref.checkpoint(x, G)
    assert torch.equal(exps, we)
    assert torch.equal(codes, wc)
    want = ref.restore(wc, we)
    for dt in (torch.bfloat16, torch.float32):
        got = q8.q8_checkpoint_load(codes, exps, out_dtype=dt)
        assert got.dtype == dt and torch.equal(got.double(), want)
    return codes, exps


@pytest.mark.parametrize("M,K,G", [(1, 32, 32), (1, 960, 64), (3, 256, 256), (7, 96, 32),
                                   (17, 11008, 128), (64, 4096, 256), (129, 1984, 64),
                                   (1000, 65280, 256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_save_and_load(M, K, G, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (M, 1), generator=g, device="cuda").float())
    x[:, :: 97] *= 50.0
    _same(x.to(dtype), G)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_edges(dtype):
    """Zero groups, ties, the borders where the exponent steps, subnormal and the largest
    values."""
    x = torch.zeros(8, 64)
    x[1, :32] = torch.arange(32) - 16.0                       # codes around zero
    x[1, 32:] = (torch.arange(32) - 16.0 + 0.5) * 0.5         # ties
    x[1, 63] = 63.5
    x[2, 0], x[2, 40] = 127.0, 127.5                          # at and above 127 * 2^0
    x[3, 0], x[3, 40] = -254.0, -255.0
    x[4, 0], x[4, 40] = 2.0 ** -126, 2.0 ** -133              # normal and subnormal
    x[5, 0], x[5, 40] = 3.3895e38, -3.3895e38                 # bf16's largest
    x[6, 5] = -0.0
    x[7] = torch.linspace(-1, 1, 64) * 2.0 ** -120
    _same(x.to(dtype).cuda(), 32)


def test_every_bf16_magnitude_as_absmax():
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)         # zero to the largest, all of them
    v = (bits << 16).view(torch.float32)
    x = torch.zeros(bits.numel(), 32)
    x[:, 0], x[:, 1], x[:, 31] = v, -v / 3, v / 2
    _same(x.bfloat16().cuda(), 32)


def test_empty():
    c, e = q8.q8_checkpoint_save(torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda"), 32)
    assert c.shape == (0, 64) and e.shape == (0, 2)
    assert q8.q8_checkpoint_load(c, e).shape == (0, 64)
    dy = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda")
    assert not q8.q8_checkpoint_wgrad(dy, c, e).any()
    w = torch.ones(16, 64, device="cuda")
    assert (q8.q8_checkpoint_wgrad(dy, c, e, dw=w, accumulate=True) == 1).all()


WGRAD = [(1, 8, 32, 32), (2, 16, 64, 64), (7, 24, 96, 32), (63, 264, 128, 128),
         (64, 128, 256, 256), (65, 136, 352, 32), (100, 8, 4096, 64), (129, 520, 640, 128),
         (200, 2560, 960, 64), (333, 256, 288, 32), (1000, 1032, 512, 256), (4096, 264, 384, 128), (2048, 5512, 1056, 32)]


@pytest.mark.parametrize("M,N,K,G", WGRAD)
def test_wgrad(M, N, K, G):
    d = ref.make(M, N, K, 8, 1, seed=M + N)
    codes, exps = q8.q8_checkpoint_save(d["x"], G)
    xs, dy = ref.restore(codes, exps), d["dy"].double()
    want, mag = dy.t() @ xs, dy.abs().t() @ xs.abs()
    dw = q8.q8_checkpoint_wgrad(d["dy"], codes, exps)
    ref.near(dw, want, ref.ACC * mag + 1e-30, "dw")
    for _ in range(3):
        assert torch.equal(dw, q8.q8_checkpoint_wgrad(d["dy"], codes, exps))
    base = torch.randn_like(dw)
    acc = q8.q8_checkpoint_wgrad(d["dy"], codes, exps, dw=base.clone(), accumulate=True)
    assert ((acc - (base + dw)).abs() <= 2.0 ** -23 * (base.abs() + dw.abs())).all()
    big = torch.full((N + 2, K), 7.0, device="cuda")
    q8.q8_checkpoint_wgrad(d["dy"], codes, exps, dw=big[:N])
    assert torch.equal(big[:N], dw) and (big[N:] == 7).all()
    assert q8.q8_last_device_status() == q8.Q8_OK


def test_wgrad_is_exact_on_whole_numbers():
    """Small whole numbers: every product and sum is exact in fp32, so the result is too."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-60, 61, (300, 192), generator=g, device="cuda").float()
    x[:, ::32] = 127.0
    dy = torch.randint(-8, 9, (300, 136), generator=g, device="cuda").float()
    codes, exps = q8.q8_checkpoint_save(x, 32)
    dw = q8.q8_checkpoint_wgrad(dy.bfloat16(), codes, exps)
    assert torch.equal(dw.double(), dy.double().t() @ x.double())


def test_training_step_from_the_checkpoint():
    """Forward, checkpoint, backward and full weight gradient in a row, as a step uses them:
    two microbatches accumulated, against the same step on the restored input."""
    d = ref.make(300, 264, 512, 16, 3, seed=21, mix="runs", free=0.1)
    codes, exps = q8.q8_checkpoint_save(d["x"], 128)
    xr = q8.q8_checkpoint_load(codes, exps)
    assert (xr.double() - d["x"].double()).abs().max() <= d["x"].double().abs().max() / 127
    args = (d["q"], d["s_w"], d["a"], d["b"], d["scale"])
    y, h = q8.q8_linear_w8a16_lora(d["x"], *args, d["ids"])
    full = q8.q8_linear_w8a16_lora_backward(d["dy"], *args, d["ids"], h, codes=codes, exps=exps)
    same = q8.q8_linear_w8a16_lora_backward(d["dy"], *args, d["ids"], h, x=xr)
    for u, v in zip(full, same):
        assert torch.equal(u, v)                     # 8 bits or the same values in bf16
    da, db = torch.zeros_like(full[1]), torch.zeros_like(full[2])
    dw = torch.zeros(264, 512, device="cuda")
    for lo, hi in ((0, 130), (130, 300)):
        part = lambda t: t[lo:hi].contiguous()                       # noqa: E731
        q8.q8_linear_w8a16_lora_backward(part(d["dy"]), *args, part(d["ids"]), part(h),
                                         codes=part(codes), exps=part(exps), want_dx=False,
                                         da=da, db=db, accumulate=True)
        q8.q8_checkpoint_wgrad(part(d["dy"]), part(codes), part(exps), dw=dw, accumulate=True)
    dx_, wa, wb, _, ba, bb = ref.backward(d, h, xr.double())
    ref.near(da, wa, ba + 2.0 ** -23 * wa.abs(), "da")
    ref.near(db, wb, bb + 2.0 ** -23 * wb.abs(), "db")
    dy = d["dy"].double()
    ref.near(dw, dy.t() @ xr.double(), 1.1 * ref.ACC * (dy.abs().t() @ xr.double().abs()), "dw")


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        q8.q8_checkpoint_save(x, 128)
    with pytest.raises(ValueError):
        q8.q8_checkpoint_save(x.half(), 32)
    with pytest.raises(ValueError):
        q8.q8_checkpoint_save(x[:, :32], 32)
    c, e = q8.q8_checkpoint_save(x, 32)
    with pytest.raises(ValueError):
        q8.q8_checkpoint_load(c, e[:3])
    with pytest.raises(q8.Q8Error):
        q8.q8_checkpoint_load(c, torch.zeros(4, 4, dtype=torch.uint8, device="cuda"))  # group 16
    with pytest.raises(ValueError):
        q8.q8_checkpoint_wgrad(torch.zeros(5, 16, dtype=torch.bfloat16, device="cuda"), c, e)
    with pytest.raises(q8.Q8Error):
        q8.q8_checkpoint_wgrad(torch.zeros(4, 12, dtype=torch.bfloat16, device="cuda"), c, e)
