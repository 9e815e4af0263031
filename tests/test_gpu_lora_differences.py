"""Gradients of the adapter linear against differences of its own forward passes, with steps large
enough that a wrong gradient cannot pass.

y is linear in x, in a and in b, each alone, so a difference of two forward passes divided by the
step is the gradient, whatever the step.  Only the perturbed row's outputs (x), the adapter's rows
(a) or one column of them (b) can change; the others have the same bits and drop out.  Inputs are
multiples of a power of two that keeps the sum with the step a bf16 number.

Tolerance: what the two sums of each changed output may be off (ref.forward's bound of an fp32 y, times
|dy|, over the step) and the gradient's own bound (ref.backward's: EPS8 of the magnitudes for dx's
rounded weight, and the result's rounding; 3 ACC of the magnitudes for da and db)."""
import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu
STEP = dict(x=32.0, a=2.0, b=2.0)                   # values in multiples of 1 / 4, 1 / 64, 1 / 64


def _inputs(M, N, K, R, L):
    d = ref.make(M, N, K, R, L, seed=170 + M, mix="each", free=0.1)
    d["x"] = (torch.round(d["x"].float() * 4) / 4).clamp(-3.75, 3.75).bfloat16()
    d["a"] = (torch.round(d["a"].float() * 64) / 64).clamp(-0.95, 0.95).bfloat16()
    d["b"] = (torch.round(d["b"].float() * 512) / 64).clamp(-0.95, 0.95).bfloat16()
    return d


def _samples(d, name):
    """Places of the input whose rows have an adapter, 12 of them."""
    g = torch.Generator().manual_seed(7)
    used = torch.unique(d["ids"][d["ids"] >= 0]).tolist()
    rows = torch.nonzero(d["ids"] >= 0).flatten().tolist()
    pick = lambda n: int(torch.randint(0, n, (1,), generator=g))             # noqa: E731
    for _ in range(12):
        first = rows[pick(len(rows))] if name == "x" else used[pick(len(used))]
        yield (first, *(pick(n) for n in d[name].shape[1:]))


def _changed(d, name, at):
    """(rows, columns) of y that the input's place `at` has a part in."""
    every = slice(None)
    if name == "x":
        return at[0], every
    rows = torch.nonzero(d["ids"] == at[0]).flatten()
    return (rows, at[1]) if name == "b" else (rows, every)


@pytest.mark.parametrize("M,N,K,R,L", [(12, 72, 64, 8, 2), (70, 72, 64, 8, 2), (300, 40, 96, 24, 100)])
@pytest.mark.parametrize("name", ["x", "a", "b"])
def test_gradients_are_differences(M, N, K, R, L, name):
    d = _inputs(M, N, K, R, L)
    args = lambda n: [n[k] for k in ("x", "q", "s_w", "a", "b", "scale", "ids")]     # noqa: E731
    y0, h = q8.q8_linear_w8a16_lora(*args(d), out_dtype=torch.float32)
    got = dict(zip("xab", q8.q8_linear_w8a16_lora_backward(
        d["dy"], *args(d)[1:], h, x=d["x"])))[name].double()
    bound = dict(zip("xab", ref.backward(d, h, d["x"].double())[3:]))[name]
    dy, off = d["dy"].double(), ref.forward(d)[2]
    diffs, errs, forceful = [], [], 0
    for at in _samples(d, name):
        n = dict(d, **{name: d[name].clone()})
        n[name][at] += STEP[name]
        assert float(n[name][at]) - float(d[name][at]) == STEP[name]
        y1, _ = q8.q8_linear_w8a16_lora(*args(n), out_dtype=torch.float32)
        where = _changed(d, name, at)
        same = torch.ones_like(y0, dtype=torch.bool)
        same[where] = False
        assert torch.equal(y1[same], y0[same])
        w = dy[where]
        diff = float(((y1.double() - y0.double())[where] * w).sum()) / STEP[name]
        slack = float(((off + ref.forward(n)[2])[where] * w.abs()).sum()) / STEP[name]
        tol = slack + float(bound[at]) + (ref.EPS8 * abs(diff) if name == "x" else 0.0)
        err = abs(float(got[at]) - diff)
        assert err <= tol, (name, at, float(got[at]), diff, tol)
        forceful += tol < 0.1 * abs(diff)
        diffs.append(diff)
        errs.append(err)
    # what the test could not tell from a zero or a sign is the exception
    assert forceful >= 8, forceful
    assert sum(e * e for e in errs) <= (0.02 ** 2) * sum(v * v for v in diffs)
