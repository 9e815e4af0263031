"""Values that are no numbers in 8-bit checkpoints: a training loop that looks for them in its
gradients has to find them there, and nothing else may change.

A group of a row that holds a NaN or an infinity gets exponent byte 255 (a step of 2^128, infinite in
bf16 and in fp32), codes of 127 and -127 for the infinities and 0 for the rest: infinities are
restored as they were and the group's other values as NaN."""
import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu
BAD = [float("nan"), -float("nan"), float("inf"), -float("inf")]


def _spoil(x, G):
    """x with a value that is no number in some groups, and which groups those are [M, K / G]."""
    M, K = x.shape
    hit = torch.zeros(M, K // G, dtype=torch.bool, device=x.device)
    y = x.clone()
    for i, v in enumerate(BAD * 3):
        m, g, at = (5 * i) % M, (3 * i + 1) % (K // G), (7 * i) % G
        y[m, g * G + at] = v
        hit[m, g] = True
    return y, hit


@pytest.mark.parametrize("M,K,G", [(1, 32, 32), (3, 512, 256), (40, 960, 64), (700, 256, 128)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_save_and_load(M, K, G, dtype):
    g = torch.Generator("cuda").manual_seed(M)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    y, hit = _spoil(x, G)
    codes, exps = q8.q8_checkpoint_save(x, G)
    c2, e2 = q8.q8_checkpoint_save(y, G)
    wide = hit.repeat_interleave(G, dim=1)
    assert (e2[hit] == 255).all() and torch.equal(e2[~hit], exps[~hit])
    assert torch.equal(c2[~wide], codes[~wide])
    want = torch.where(torch.isinf(y), y.sign() * 127, torch.zeros_like(y))[wide]
    assert torch.equal(c2[wide].float(), torch.nan_to_num(want.float()))
    for dt in (torch.bfloat16, torch.float32):
        z = q8.q8_checkpoint_load(c2, e2, out_dtype=dt)
        assert torch.equal(z[~wide], q8.q8_checkpoint_load(codes, exps, out_dtype=dt)[~wide])
        inf = torch.isinf(y)
        assert torch.equal(z[inf].float(), y[inf].float())
        assert torch.isnan(z[wide & ~inf]).all()


@pytest.mark.parametrize("M,N,K,R", [(9, 24, 128, 8), (300, 136, 512, 64), (2600, 2568, 2336, 16)])
def test_gradients_from_them(M, N, K, R):
    """dw is spoilt in the columns of the spoilt groups and da in those of the rows' own adapters,
    both as from the restored values, and every other entry keeps its bits."""
    G = 32
    d = ref.make(M, N, K, R, 3, seed=80 + M, mix="runs", free=0.3)
    d["dy"] = torch.where(d["dy"] == 0, torch.full_like(d["dy"], 2.0 ** -6), d["dy"])
    y, hit = _spoil(d["x"], G)
    args = [d[k] for k in ("q", "s_w", "a", "b", "scale", "ids")]
    h = ref.forward(d)[1].float()
    codes, exps = q8.q8_checkpoint_save(d["x"], G)
    c2, e2 = q8.q8_checkpoint_save(y, G)
    dw, dw2 = q8.q8_checkpoint_wgrad(d["dy"], codes, exps), q8.q8_checkpoint_wgrad(d["dy"], c2, e2)
    cols = hit.any(0).repeat_interleave(G)
    assert torch.equal(dw2[:, ~cols], dw[:, ~cols])
    assert not torch.isfinite(dw2[:, cols]).any()
    grads = [q8.q8_linear_w8a16_lora_backward(d["dy"], *args, h, codes=c, exps=e)
             for c, e in ((codes, exps), (c2, e2))]
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][2], grads[1][2])
    from_bf16 = q8.q8_linear_w8a16_lora_backward(d["dy"], *args, h, x=q8.q8_checkpoint_load(c2, e2),
                                                 want_dx=False, want_db=False)[1]
    for i in range(3):
        rows = d["ids"] == i
        cols = hit[rows].any(0).repeat_interleave(G) if rows.any() else torch.zeros_like(cols)
        da, da2 = grads[0][1][i], grads[1][1][i]
        assert torch.equal(da2[:, ~cols], da[:, ~cols])
        assert not torch.isfinite(da2[:, cols]).any()
        assert torch.equal(torch.isnan(from_bf16[i]), torch.isnan(da2))
    assert q8.q8_last_device_status() == q8.Q8_OK
