"""What fp32 results of the adapter linear keep of the low-rank term: h is fp32, and so is what
reaches y of it, in calls of every size.

The bound, from the call's own h (so that h's sums are not in it), per output: scale * h is rounded
once (2^-24).  It is a number of 24 bits, all of which three bf16 parts hold.  The tensor core adds 16 products a step and cuts off less
than 2^-23 of the magnitudes added so far: 3 * rank / 16 steps, and one more where the columns
begin in the middle of one.  Base sums are as in test_gpu_lora_uses.py: 33 * 2^-23 and a rounding
for each 1024 terms; scaling, adding the term and the bias round once each (2^-24)."""
import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24


def _bound(R, K, term, base, bias):
    low = (2 * (3 * R / 16 + 2) + 1) * HALF * term
    top = (66 + K / 1024 + 6) * HALF * base
    return low + top + 3 * HALF * (term + base + bias)


@pytest.mark.parametrize("M,N,K,R,L", [(1, 64, 64, 8, 1), (16, 200, 64, 8, 3), (17, 129, 64, 8, 3),
                                       (40, 264, 2064, 8, 2), (77, 640, 128, 16, 8),
                                       (300, 1025, 96, 8, 40), (333, 96, 80, 24, 3),
                                       (700, 264, 4096, 8, 300), (90, 77, 64, 136, 2),
                                       (65, 72, 64, 256, 9), (2600, 2565, 2336, 8, 5)])
@pytest.mark.parametrize("mix", ["each", "runs"])
def test_term_in_fp32(M, N, K, R, L, mix):
    """The term is nearly all of y: the base product is a millionth of its usual size."""
    d = ref.make(M, N, K, R, L, seed=90 + M + R, mix=mix, free=0.1)
    d["s_w"] *= 2.0 ** -20
    d["bias"] = torch.randn(N, device="cuda") * 2.0 ** -20
    y, h = q8.q8_linear_w8a16_lora(d["x"], d["q"], d["s_w"], d["a"], d["b"], d["scale"], d["ids"],
                                   bias=d["bias"], out_dtype=torch.float32)
    wh, bh = ref.forward(d)[1::2]
    ref.near(h, wh, bh, "h")
    x, w = d["x"].double(), d["s_w"].double()[:, None] * d["q"].double()
    want, mag = x @ w.t() + d["bias"].double(), x.abs() @ w.abs().t()
    term = torch.zeros_like(want)
    for i in range(L):
        rows = torch.nonzero(d["ids"] == i).flatten()
        c, hi, b = d["scale"][i].double(), h[rows].double(), d["b"][i].double()
        want[rows] += c * (hi @ b.t())
        term[rows] = c * (hi.abs() @ b.abs().t())
    ref.near(y, want, _bound(R, K, term, mag, d["bias"].double().abs()) + 1e-30, "y")
    assert q8.q8_last_device_status() == q8.Q8_OK


@pytest.mark.parametrize("M", [4, 40, 300])
def test_every_bit_of_h_reaches_y(M):
    """h of 24 significant bits and a b that picks one of them a column: y is h, bit for bit, times
    a power of two."""
    R, K, N, L = 8, 64, 64, 2
    g = torch.Generator("cuda").manual_seed(M)
    d = ref.make(M, N, K, R, L, seed=M, free=0.0)
    d["q"].zero_()
    x = torch.zeros(M, K, device="cuda")
    # x = (1, 2^-8, 2^-16) times bytes, a = 1 at three k: h = a whole number of 24 bits * 2^-16
    part = torch.randint(128, 256, (M, 3), generator=g, device="cuda").float()
    x[:, 0], x[:, 17], x[:, 40] = part[:, 0], part[:, 1] * 2.0 ** -8, part[:, 2] * 2.0 ** -16
    a = torch.zeros(L, R, K, device="cuda")
    a[:, :, 0] = a[:, :, 17] = a[:, :, 40] = 1.0
    b = torch.zeros(L, N, R, device="cuda")
    b[:, torch.arange(N), torch.arange(N) % R] = 2.0
    scale = torch.tensor([0.5, 4.0], device="cuda")
    y, h = q8.q8_linear_w8a16_lora(x.bfloat16(), d["q"], d["s_w"], a.bfloat16(), b.bfloat16(),
                                   scale, d["ids"], out_dtype=torch.float32)
    want = x.double().sum(1)
    # the warp-level sums may cut the last bit off; what h holds is what y has to hold
    assert ((h.double() - want[:, None]).abs() <= 2.0 ** -23 * want[:, None]).all()
    c = 2.0 * scale[d["ids"].long()].double()
    ref.near(y, (c * h[:, 0].double())[:, None].expand(M, N), 2.0 ** -23 * (c * want)[:, None], "y")


@pytest.mark.parametrize("M,N,K,R", [(40, 72, 256, 24), (333, 1025, 2064, 8), (2600, 4096, 2048, 16)])
def test_workspace_of_an_fp32_call(M, N, K, R):
    """The size that q8_workspace_bytes gives is enough for three parts, and nothing behind it is
    written."""
    d = ref.make(M, N, K, R, 3, seed=190 + M)
    args = [d[k] for k in ("x", "q", "s_w", "a", "b", "scale", "ids")]
    want = q8.q8_linear_w8a16_lora(*args, out_dtype=torch.float32)
    need = q8.q8_workspace_bytes(q8.Q8_OP_LINEAR_W8A16_LORA, M, N, K, R)
    for fill in (0xFF, 0x01):
        ws = torch.full((need + 4096,), fill, dtype=torch.uint8, device="cuda")
        got = q8.q8_linear_w8a16_lora(*args, out_dtype=torch.float32, workspace=ws[:need])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (ws[need:] == fill).all()
