"""What is measured of the low-rank adapter and 8-bit checkpoint operators.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the
calls a user of this package makes:

  lora      y = s_w * (x q^T) + the low-rank term of each row's own adapter,
            h = x a^T (kept for the backward pass)
  lora_bwd  the gradients of that linear: dx through the frozen int8 weight and the
            adapters, da and db of every adapter; the layer's input comes as bf16 or as an
            8-bit checkpoint
  ckpt      an 8-bit activation checkpoint taken and restored
  wgrad     the weight gradient of a linear from the 8-bit checkpoint of its input

`own` chooses the side; see run().
"""
import math

import torch

own = False

# (K, N) pairs of this repository's decode sweep and Llama-shaped stack.
SHAPES = [(960, 2560), (2048, 8192), (4096, 4096), (4096, 11008), (11008, 4096)]


def listed():
    return [
        # one sequence decoding with one adapter on the smallest layer: launch latency counts
        dict(name="lora M1 960x2560", op="lora", M=1, K=960, N=2560, R=8, L=1, mix="each",
             free=0.0, out="bf16"),
        # a decode batch of 16 requests that use 32 loaded adapters at random
        dict(name="lora M16 4096x11008", op="lora", M=16, K=4096, N=11008, R=16, L=32,
             mix="each", free=0.1, out="bf16"),
        # a ragged decode batch beyond one 16-row pass, rows in no order, fp32 output
        dict(name="lora M77 2048x8192 f32", op="lora", M=77, K=2048, N=8192, R=64, L=8,
             mix="each", free=0.1, out="f32"),
        # prompts of several requests in one prefill batch, each with its own adapter
        dict(name="lora M4096 4096x4096", op="lora", M=4096, K=4096, N=4096, R=16, L=8,
             mix="runs", free=0.1, out="bf16"),
        # a training step's forward pass over three adapters at once, odd token count
        dict(name="lora M2047 4096x11008", op="lora", M=2047, K=4096, N=11008, R=32, L=3,
             mix="runs", free=0.0, out="bf16"),
        # gradients of a small layer, input kept in bf16
        dict(name="bwd M333 960x2560", op="lora_bwd", M=333, K=960, N=2560, R=8, L=3,
             mix="runs", free=0.1, G=0),
        # one adapter of high rank, input kept in 8 bits
        dict(name="bwd M1000 2048x8192", op="lora_bwd", M=1000, K=2048, N=8192, R=64, L=1,
             mix="each", free=0.0, G=64),
        # a full training batch over four adapters, input kept in 8 bits
        dict(name="bwd M4096 4096x11008", op="lora_bwd", M=4096, K=4096, N=11008, R=16, L=4,
             mix="runs", free=0.05, G=128),
        # the checkpoint of a single token
        dict(name="ckpt 1x960", op="ckpt", M=1, K=960, G=32),
        # the checkpoint of a training batch at the widest layer input
        dict(name="ckpt 4096x11008", op="ckpt", M=4096, K=11008, G=128),
        # weight gradients: a short ragged batch, and a full one
        dict(name="wgrad M200 960x2560", op="wgrad", M=200, K=960, N=2560, G=32),
        dict(name="wgrad M4096 4096x11008", op="wgrad", M=4096, K=4096, N=11008, G=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora", "lora_bwd", "lora_bwd", "ckpt", "wgrad"])
    if op == "ckpt":
        G = rng.choice([32, 64, 128, 256])
        return dict(op=op, M=_log_int(rng, 1, 4096), K=G * _log_int(rng, 1, 11008 // G), G=G)
    # K a multiple of 64 up to 4096; N a multiple of 8 up to 11008, odd tile tails among them
    K = 64 * _log_int(rng, 4, 64)
    N = 8 * _log_int(rng, 32, 1376)
    if op == "wgrad":
        G = rng.choice([g for g in (32, 64, 128, 256) if K % g == 0])
        return dict(op=op, M=_log_int(rng, 8, 4096), K=K, N=N, G=G)
    c = dict(op=op, M=_log_int(rng, 1, 4096), K=K, N=N, R=rng.choice([8, 16, 32, 64]),
             L=_log_int(rng, 1, 16), mix=rng.choice(["each", "runs"]),
             free=rng.choice([0.0, 0.1, 0.5]))
    if op == "lora":
        c["out"] = rng.choice(["bf16", "bf16", "f32"])
    else:
        c["G"] = rng.choice([0] + [g for g in (32, 64, 128, 256) if K % g == 0])
    return c


# ------------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activations(g, M, K):
    """bf16 activations with a few channels far larger than the rest."""
    x = _normal(g, (M, K), 1.0)
    cols = torch.randperm(K, generator=g, device="cuda")[: max(1, K // 512)]
    x[:, cols] *= 20.0
    return x.to(torch.bfloat16)


def _pow2(e):
    """2**e of whole numbers -126..127, exact: the exponent bits of an fp32 number."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _group_scales(x, G):
    """8-bit groups of G values of a row: codes and the powers of two they count."""
    M, K = x.shape
    v = x.float().view(M, K // G, G)
    mant, expo = torch.frexp(v.abs().amax(2))
    e = (expo - 7 + (mant > 127.0 / 128.0)).clamp(-126, 121)
    e = torch.where(mant == 0, torch.full_like(e, -126), e)
    c = torch.round(v * _pow2(-e).unsqueeze(2)).clamp(-127, 127)
    return c.view(M, K), e


def _ids(case, g):
    """int32 [M]: each row's adapter, -1 for a row without one.  "each": rows in no order;
    "runs": the rows of a request follow one another."""
    M, L = case["M"], case["L"]
    if case["mix"] == "each":
        ids = torch.randperm(M, generator=g, device="cuda") % L
    else:
        u = torch.rand(max(1, L - 1), generator=g, device="cuda")
        cuts = (u * M).long().sort().values[: L - 1]
        ids = torch.bucketize(torch.arange(M, device="cuda"), cuts, right=True)
    drop = torch.rand(M, generator=g, device="cuda") < case["free"]
    if case["mix"] == "runs":               # rows without an adapter: one run at the end
        drop = torch.arange(M, device="cuda") >= M - int(case["free"] * M)
    return torch.where(drop, torch.full_like(ids, -1), ids).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "ckpt":
        return dict(op="ckpt", G=case["G"], x=_activations(g, case["M"], case["K"]))
    M, K, N = case["M"], case["K"], case["N"]
    st = dict(op=case["op"])
    if case["op"] != "lora":
        st["dy"] = _normal(g, (M, N), 2.0 ** -10).to(torch.bfloat16)
    if case["op"] == "lora":
        st["x"] = _activations(g, M, K)
    else:
        G = st["G"] = case["G"]
        x = _activations(g, M, K)
        if G:
            c, e = _group_scales(x, G)
            st["codes"], st["exps"] = c.to(torch.int8), (e + 127).to(torch.uint8)
        else:
            st["x"] = x
    if case["op"] == "wgrad":
        return st
    W = _normal(g, (N, K), 0.02)
    st["s_w"] = W.abs().amax(1) / 127.0
    st["q"] = torch.round(W / st["s_w"][:, None]).clamp(-127, 127).to(torch.int8)
    del W
    L, R = case["L"], case["R"]
    st["a"] = _normal(g, (L, R, K), K ** -0.5).to(torch.bfloat16)
    st["b"] = _normal(g, (L, N, R), 0.02).to(torch.bfloat16)
    st["scale"] = 16.0 / R * (1.0 + torch.rand(L, generator=g, device="cuda"))
    st["ids"] = _ids(case, g)
    if case["op"] == "lora":
        st["out"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    else:
        st["h"] = _normal(g, (M, R), 1.0) * (st["ids"] >= 0)[:, None]
    return st


# ------------------------------------------------------------------------------ plain forms


def _rows_of(h, ids, L):
    """[M, R] rows into the columns of their adapters: [M, L * R], zero elsewhere."""
    M, R = h.shape
    hot = ids[:, None] == torch.arange(L, device=h.device, dtype=ids.dtype)
    return (hot[:, :, None] * h[:, None, :]).view(M, L * R)


def _mine(hall, ids, L):
    """[M, L * R] products with every adapter -> [M, R] of the row's own, 0 without one."""
    M = hall.shape[0]
    own_col = ids.long().clamp(min=0)
    h = hall.view(M, L, -1)[torch.arange(M, device=hall.device), own_col]
    return torch.where((ids >= 0)[:, None], h, torch.zeros_like(h))


def _plain_lora(st):
    x, a, b, ids = st["x"].float(), st["a"].float(), st["b"].float(), st["ids"]
    L, R, K = a.shape
    h = _mine(x @ a.view(L * R, K).t(), ids, L)
    c = st["scale"][ids.long().clamp(min=0)][:, None]
    low = _rows_of(h * c, ids, L) @ b.permute(1, 0, 2).reshape(-1, L * R).t()
    y = st["s_w"] * (x @ st["q"].float().t()) + low
    return y.to(st["out"]), h


def _plain_input(st):
    if not st["G"]:
        return st["x"].float()
    c, e = st["codes"], st["exps"].int() - 127
    M, K = c.shape
    return (c.float().view(M, -1, st["G"]) * _pow2(e).unsqueeze(2)).view(M, K)


def _plain_lora_bwd(st):
    dy, a, b, ids = st["dy"].float(), st["a"].float(), st["b"].float(), st["ids"]
    L, R, K = a.shape
    N = b.shape[1]
    ball = b.permute(1, 0, 2).reshape(N, L * R)
    c = st["scale"][ids.long().clamp(min=0)][:, None]
    g = _rows_of(_mine(dy @ ball, ids, L) * c, ids, L)
    dx = dy @ (st["q"].float() * st["s_w"][:, None]) + g @ a.view(L * R, K)
    da = (g.t() @ _plain_input(st)).view(L, R, K)
    db = (dy.t() @ _rows_of(st["h"] * c, ids, L)).view(N, L, R).permute(1, 0, 2)
    return dx.to(torch.bfloat16), da, db.contiguous()


def _plain_ckpt(st):
    c, e = _group_scales(st["x"], st["G"])
    M, K = c.shape
    v = c.view(M, -1, st["G"]) * _pow2(e).unsqueeze(2)
    return v.view(M, K).to(torch.bfloat16)


def _plain_wgrad(st):
    return st["dy"].float().t() @ _plain_input(st)


def run(st):
    if own:
        return _own(st)
    return {"lora": _plain_lora, "lora_bwd": _plain_lora_bwd, "ckpt": _plain_ckpt,
            "wgrad": _plain_wgrad}[st["op"]](st)


def _own(st):
    import int8_quantized_linear_q8_b200 as q8

    if st["op"] == "lora":
        return q8.q8_linear_w8a16_lora(st["x"], st["q"], st["s_w"], st["a"], st["b"],
                                       st["scale"], st["ids"], out_dtype=st["out"])
    if st["op"] == "lora_bwd":
        return q8.q8_linear_w8a16_lora_backward(
            st["dy"], st["q"], st["s_w"], st["a"], st["b"], st["scale"], st["ids"], st["h"],
            x=st.get("x"), codes=st.get("codes"), exps=st.get("exps"))
    if st["op"] == "ckpt":
        codes, exps = q8.q8_checkpoint_save(st["x"], st["G"])
        return q8.q8_checkpoint_load(codes, exps)
    return q8.q8_checkpoint_wgrad(st["dy"], st["codes"], st["exps"])


# ------------------------------------------------------------------------------ definitions


def _exact_step(e):
    """2**e in 64 bits, exact: the exponent bits of an fp64 number."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_input(st):
    if not st["G"]:
        return st["x"].double()
    step = _exact_step(st["exps"].long() - 127)
    return st["codes"].double() * step.repeat_interleave(st["G"], dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "ckpt":
        M, K, G = case["M"], case["K"], case["G"]
        v = st["x"].double().view(M, K // G, G)
        top = v.abs().amax(2, keepdim=True)
        # the smallest power of two that counts the largest value in at most 127 steps
        e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 127.0))
        e = torch.where(top > 127.0 * _exact_step(e), e + 1, e)
        e = torch.where(top <= 127.0 * _exact_step(e - 1), e - 1, e).clamp(-126, 121)
        step = _exact_step(e)
        return (torch.round(v / step).clamp(-127, 127) * step).view(M, K)
    if st["op"] == "wgrad":
        return torch.matmul(st["dy"].double().t(), _exact_input(st))
    w = st["s_w"].double()[:, None] * st["q"].double()
    a, b, s, ids = st["a"].double(), st["b"].double(), st["scale"].double(), st["ids"].long()
    if st["op"] == "lora":
        x = st["x"].double()
        y = torch.matmul(x, w.t())
        h = torch.zeros(case["M"], case["R"], dtype=torch.float64, device=x.device)
        for i in range(case["L"]):
            rows = torch.nonzero(ids == i).flatten()
            h[rows] = torch.matmul(x[rows], a[i].t())
            y[rows] += s[i] * torch.matmul(h[rows], b[i].t())
        return y, h
    dy, h, x = st["dy"].double(), st["h"].double(), _exact_input(st)
    dx = torch.matmul(dy, w)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i in range(case["L"]):
        rows = torch.nonzero(ids == i).flatten()
        g = s[i] * torch.matmul(dy[rows], b[i])
        dx[rows] += torch.matmul(g, a[i])
        da[i] = torch.matmul(g.t(), x[rows])
        db[i] = s[i] * torch.matmul(dy[rows].t(), h[rows])
    return dx, da, db


# ------------------------------------------------------------------------------------ work


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "ckpt":
        # x read; codes and exponents written, read again; the restored values written
        return {"bytes": 6 * M * K + 2 * M * K // case["G"], "flops": 4 * M * K}
    N, G = case["N"], case.get("G", 0)
    kept = 2 * M * K if not G else M * K + M * K // G      # the layer's input as it is kept
    if case["op"] == "wgrad":
        return {"bytes": kept + 2 * M * N + 4 * N * K, "flops": 2 * M * N * K}
    R = case["R"]
    rows = M - int(case["free"] * M)                       # rows with an adapter, about
    used = max(1, min(case["L"], rows))                    # adapters that rows use, about
    low = 2 * used * R * (K + N) + 4 * used + 4 * M
    if case["op"] == "lora":
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * M * K + N * K + 4 * N + low + size * M * N + 4 * M * R,
                "flops": 2 * M * N * K + 2 * rows * R * (K + N)}
    return {"bytes": 2 * M * N + N * K + 4 * N + low + 4 * M * R + kept + 2 * M * K
            + 4 * case["L"] * R * (K + N),
            "flops": 2 * M * N * K + 4 * rows * R * (K + N)}
