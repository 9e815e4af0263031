"""Uses of the adapter linear and the 8-bit checkpoint that the other files leave out: large
products in captured graphs, graphs with two branches, host threads, weights made just before
their use, workspaces that hold anything, the longest rows, pools and batches past 2^31 elements."""
import threading

import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu


def _step(d, G, stream=None, codes=None, exps=None, **kw):
    """Forward, checkpoint, every gradient from it."""
    y, h = q8.q8_linear_w8a16_lora(d["x"], d["q"], d["s_w"], d["a"], d["b"], d["scale"], d["ids"],
                                   stream=stream, **kw)
    codes, exps = q8.q8_checkpoint_save(d["x"], G, codes=codes, exps=exps, stream=stream)
    g = q8.q8_linear_w8a16_lora_backward(d["dy"], d["q"], d["s_w"], d["a"], d["b"], d["scale"],
                                         d["ids"], h, codes=codes, exps=exps, stream=stream, **kw)
    dw = q8.q8_checkpoint_wgrad(d["dy"], codes, exps, stream=stream, **kw)
    return y, h, codes, exps, *g, dw


def _check(d, out):
    y, h, codes, exps, dx, da, db, dw = out
    wy, wh, by, bh = ref.forward(d)
    ref.near(h, wh, bh, "h")
    ref.near(y, wy, by + ref.EPS8 * wy.abs(), "y")
    xs, dy = ref.restore(codes, exps), d["dy"].double()
    gx, ga, gb, bx, ba, bb = ref.backward(d, h, xs)
    ref.near(dx, gx, bx + ref.EPS8 * gx.abs(), "dx")
    ref.near(da, ga, ba, "da")
    ref.near(db, gb, bb, "db")
    ref.near(dw, dy.t() @ xs, ref.ACC * (dy.abs().t() @ xs.abs()) + 1e-30, "dw")
    assert q8.q8_last_device_status() == q8.Q8_OK


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("M,L,mix", [(4096, 1024, "each"), (4097, 3, "wild"), (8192, 1023, "runs"),
                                     (9001, 1024, "each"), (13000, 1, "each"), (20011, 40, "each")])
def test_many_rows_sorted(M, L, mix):
    d = ref.make(M, 24, 64, 8, L, seed=29 + M, mix=mix)
    _check(d, _step(d, 32))


@pytest.mark.parametrize("N,K,R", [(10240, 2048, 16), (8192, 2048, 16), (8192, 2048, 64),
                                   (11008, 2816, 32), (8192, 8192, 8), (512, 256, 136)])
@pytest.mark.parametrize("M", [333, 700, 1100])
def test_gradients_split_over_clusters_of_every_size(M, N, K, R):
    d = ref.make(M, N, K, R, 1, seed=45, free=0.0)
    h = ref.forward(d)[1].float()
    codes, exps = ref.checkpoint(d["x"], 256)
    _, da, db = q8.q8_linear_w8a16_lora_backward(d["dy"], d["q"], d["s_w"], d["a"], d["b"],
                                                 d["scale"], d["ids"], h, codes=codes, exps=exps,
                                                 want_dx=False)
    _, ga, gb, _, ba, bb = ref.backward(d, h, ref.restore(codes, exps))
    ref.near(da, ga, ba, "da")
    ref.near(db, gb, bb, "db")


def _expands(M, N, K):
    """Whether all three products expand their int8 operand in the workspace."""
    for op, n in ((q8.Q8_OP_LINEAR_W8A16_LORA, N * K), (q8.Q8_OP_LINEAR_W8A16_LORA_BACKWARD, N * K),
                  (q8.Q8_OP_CHECKPOINT_WGRAD, M * K)):
        assert q8.q8_workspace_bytes(op, M, N, K, 8) >= 2 * n


@pytest.mark.parametrize("M,N,K,G", [(2563, 2568, 2336, 32), (2817, 4104, 1344, 64)])
def test_large_products_of_odd_sizes(M, N, K, G):
    _expands(M, N, K)
    d = ref.make(M, N, K, 24, 5, seed=30, mix="runs")
    _check(d, _step(d, G))
    n = dict(d, q=d["q"][:N - 7].contiguous(), s_w=d["s_w"][:N - 7].contiguous(),
             b=d["b"][:, :N - 7].contiguous(), bias=torch.randn(N - 7, device="cuda"))
    for out in (torch.float32, torch.bfloat16):
        y, _ = q8.q8_linear_w8a16_lora(n["x"], n["q"], n["s_w"], n["a"], n["b"], n["scale"],
                                       n["ids"], bias=n["bias"], out_dtype=out)
        wy, _, by, _ = ref.forward(n)
        ref.near(y, wy, by + (ref.EPS8 * wy.abs() if out == torch.bfloat16 else 0.0), "y")


def test_large_products_captured_and_replayed():
    """Sizes whose int8 operand is expanded beforehand, in one graph of 13 kernels."""
    size = (2600, 4096, 2048, 24, 6)
    _expands(*size[:3])
    d = ref.make(*size, seed=31)
    _step(d, 128)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = _step(d, 128)
    for seed, mix in ((32, "runs"), (33, "wild")):
        n = ref.make(*size, seed=seed, mix=mix)
        for k in ("x", "ids", "dy", "a", "b", "scale", "q", "s_w"):
            d[k].copy_(n[k])
        for _ in range(3):
            g.replay()
        eager = _step(d, 128)
        g.replay()
        torch.cuda.synchronize()
        assert _same(out, eager)
        _check(d, out)


@pytest.mark.parametrize("M", [7, 200])
def test_captured_with_two_branches(M):
    """The forward pass on one branch, the checkpoint and its weight gradient on the other, the
    backward pass where they join."""
    d = ref.make(M, 136, 256, 16, 3, seed=34)
    want = _step(d, 64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            codes, exps = q8.q8_checkpoint_save(d["x"], 64)
            dw = q8.q8_checkpoint_wgrad(d["dy"], codes, exps)
        y, h = q8.q8_linear_w8a16_lora(d["x"], d["q"], d["s_w"], d["a"], d["b"], d["scale"],
                                       d["ids"])
        main.wait_stream(side)
        grads = q8.q8_linear_w8a16_lora_backward(d["dy"], d["q"], d["s_w"], d["a"], d["b"],
                                                 d["scale"], d["ids"], h, codes=codes, exps=exps)
    for _ in range(3):
        for t in (y, h, dw, *grads):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert _same((y, h, codes, exps, *grads, dw), want)


def test_host_threads():
    """Two host threads, a stream and inputs each, small and large products by turns."""
    ds = [[ref.make(M, 264, 512, 16, 4, seed=35 + M + i) for M in (3, 40, 300)] for i in range(2)]
    want = [[_step(d, 32) for d in row] for row in ds]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                got = [_step(d, 32, stream=s) for d in ds[i]]
                s.synchronize()
                if not all(_same(u, v) for u, v in zip(got, want[i])):
                    raise AssertionError("other bits than a single thread's")
        except Exception as e:                                       # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong, wrong


@pytest.mark.parametrize("M", [1, 12, 40, 2600])
def test_operands_made_just_before(M):
    """Weights, checkpoints and gradients made by the calls before, with nothing between them:
    each call reads what the last one wrote."""
    N, K = (4096, 2048) if M == 2600 else (1024, 512)
    ds = [ref.make(M, N, K, 16, 3, seed=36 + i) for i in range(3)]
    Ws = [torch.randn(N, K, device="cuda", generator=torch.Generator("cuda").manual_seed(i)) * 0.02
          for i in range(3)]

    def chain(d, W, wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        q, s, _ = q8.q8_quantize_weight(W)
        sync()
        c = dict(d, q=q, s_w=s)
        out = _step(c, 32)
        sync()
        y2 = q8.q8_linear_w8a16(d["x"], q, s)
        sync()
        c2, e2 = q8.q8_checkpoint_save(out[0], 32)
        sync()
        z = q8.q8_checkpoint_load(c2, e2)
        sync()
        dx = q8.q8_linear_w8a16_lora_backward(z, q, s, d["a"], d["b"], d["scale"], d["ids"],
                                              want_da=False, want_db=False)[0]
        sync()
        return (*out, y2, c2, e2, z, dx)

    want = [chain(d, W, True) for d, W in zip(ds, Ws)]
    for _ in range(4):
        got = [chain(d, W, False) for d, W in zip(ds, Ws)]
        torch.cuda.synchronize()
        assert all(_same(u, v) for u, v in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(5, 72, 256), (90, 72, 256), (2600, 4096, 2048)])
def test_what_a_workspace_held_does_not_matter(M, N, K):
    d = ref.make(M, N, K, 8, 3, seed=37)
    want = _step(d, 64)
    need = max(q8.q8_workspace_bytes(q8.Q8_OP_LINEAR_W8A16_LORA, M, N, K, 8),
               q8.q8_workspace_bytes(q8.Q8_OP_LINEAR_W8A16_LORA_BACKWARD, M, N, K, 8),
               q8.q8_workspace_bytes(q8.Q8_OP_CHECKPOINT_WGRAD, M, N, K, 0))
    for fill in (0xFF, 0x7F, 0x01):
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        got = _step(d, 64, workspace=ws[:need])
        assert _same(got, want)
        assert (ws[need:] == fill).all()


@pytest.mark.parametrize("M", [1, 8, 9, 16, 17, 70])
@pytest.mark.parametrize("K,G", [(65504, 32), (65472, 64)])
def test_longest_rows(M, K, G):
    d = ref.make(M, 40, K, 8, 2, seed=38)
    _check(d, _step(d, G))


@pytest.mark.parametrize("M", [3, 40])
def test_pool_past_2_to_31(M):
    """b has more than 2^31 elements; only the last adapters are used (and initialised)."""
    L, N, R, K = 530, 16384, 256, 64
    d = ref.make(M, N, K, R, 2, seed=39)
    a = torch.empty(L, R, K, dtype=torch.bfloat16, device="cuda")
    b = torch.empty(L, N, R, dtype=torch.bfloat16, device="cuda")
    assert b.numel() > 2 ** 31
    a[-2:], b[-2:] = d["a"], d["b"]
    scale = torch.cat([torch.ones(L - 2, device="cuda"), d["scale"]])
    big = dict(d, a=a, b=b, scale=scale,
               ids=torch.where(d["ids"] >= 0, d["ids"] + (L - 2), d["ids"]))
    y, h, codes, exps, dx, da, db, dw = _step(big, 32)
    assert not da[:-2].any() and not db[:-2].any()
    _check(d, (y, h, codes, exps, dx, da[-2:], db[-2:], dw))


def test_batch_past_2_to_31():
    """x, its checkpoint and dx of more than 2^31 elements: the last rows against the same rows
    alone."""
    M, N, K, R, L = 36000, 8, 65504, 8, 2
    tail = ref.make(50, N, K, R, L, seed=40)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 2 ** 31
    x[-50:] = tail["x"]
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-50:] = tail["ids"]
    dy = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dy[-50:] = tail["dy"]
    y, h, codes, exps, dx, da, db, dw = _step(dict(tail, x=x, ids=ids, dy=dy), 32)
    assert not y[:-50].any() and not h[:-50].any() and not dx[:-50].any()
    assert not codes[:-50].any() and (exps[:-50] == 1).all()
    assert torch.equal(q8.q8_checkpoint_load(codes, exps)[-50:].double(),
                       ref.restore(codes[-50:], exps[-50:]))
    _check(tail, (y[-50:], h[-50:], codes[-50:], exps[-50:], dx[-50:], da, db, dw))


def test_outputs_past_2_to_31():
    """y of more than 2^31 elements, its last rows against the same rows alone."""
    M, N, K = 140000, 16384, 64
    tail = ref.make(40, N, K, 8, 2, seed=41, bias=True)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-40:] = tail["x"]
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    ids[-40:] = tail["ids"]
    y, h = q8.q8_linear_w8a16_lora(x, tail["q"], tail["s_w"], tail["a"], tail["b"], tail["scale"],
                                   ids, bias=tail["bias"])
    assert y.numel() > 2 ** 31 and not h[:-40].any()
    rows = torch.tensor([0, 255, 256, 70001, M - 41], device="cuda")
    assert (y[rows] == tail["bias"].bfloat16()).all()
    wy, wh, by, bh = ref.forward(tail)
    ref.near(h[-40:], wh, bh, "h")
    ref.near(y[-40:], wy, by + ref.EPS8 * wy.abs(), "y")


# A sum of up to 1024 terms is made by the tensor core in 64 steps, each of which cuts off less than
# a unit in the last place (2^-23) of a running sum that is, for terms of one sign, half the sum
# on average; sums are then added up with a rounding (2^-24) each, and the result is scaled.
def _one_sign(terms):
    return 33 * 2.0 ** -23 + (terms / 1024 + 6) * 2.0 ** -24


@pytest.mark.parametrize("M,N,K", [(30000, 2560, 960), (20000, 264, 16384), (2048, 1024, 4096),
                                   (16384, 264, 512), (8192, 2048, 1024), (5000, 1000, 960)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_long_gradient_sums_of_one_sign(M, N, K, accumulate):
    g = torch.Generator("cuda").manual_seed(42)
    codes = torch.randint(1, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    exps = torch.full((M, K // 64), 120, dtype=torch.uint8, device="cuda")
    dy = torch.rand(M, N, device="cuda", generator=g).bfloat16() + 0.125
    want = (dy.double().t() @ codes.double()) * 2.0 ** -7
    base = torch.full((N, K), 3.0, device="cuda") if accumulate else None
    dw = q8.q8_checkpoint_wgrad(dy, codes, exps, dw=base, accumulate=accumulate)
    if accumulate:
        want += 3.0
    ref.near(dw, want, _one_sign(M) * want, "dw")


@pytest.mark.parametrize("M,N,K", [(300, 8192, 65520), (3000, 2064, 16384), (40, 11008, 4096),
                                   (40, 4096, 16384), (300, 4096, 8192), (77, 5000, 4112),
                                   (33, 77, 4080), (4096, 512, 16384)])
def test_long_forward_sums_of_one_sign(M, N, K):
    d = ref.make(M, N, K, 8, 2, seed=43, mix="none", bias=True)
    d["x"] = d["x"].abs()
    d["q"] = d["q"].abs()
    d["bias"] = d["bias"].abs()
    y, _ = q8.q8_linear_w8a16_lora(d["x"], d["q"], d["s_w"], d["a"], d["b"], d["scale"], d["ids"],
                                   bias=d["bias"], out_dtype=torch.float32)
    want = ref.forward(d)[0]
    ref.near(y, want, _one_sign(K) * want, "y")


@pytest.mark.parametrize("M,N,K", [(20000, 264, 16384), (700, 11008, 4096), (9000, 512, 8192)])
def test_converted_products_have_the_same_bits_every_time(M, N, K):
    """Long runs of stages through the rings that convert the int8 operand."""
    d = ref.make(M, N, K, 8, 2, seed=44, mix="runs")
    codes, exps = q8.q8_checkpoint_save(d["x"], 64)
    args = (d["q"], d["s_w"], d["a"], d["b"], d["scale"], d["ids"])
    calls = [lambda: q8.q8_checkpoint_wgrad(d["dy"], codes, exps)]
    if M < 1000:
        h = q8.q8_linear_w8a16_lora(d["x"], *args)[1]
        calls += [lambda: q8.q8_linear_w8a16_lora(d["x"], *args)[0],
                  lambda: q8.q8_linear_w8a16_lora_backward(d["dy"], *args, h, want_da=False,
                                                           want_db=False)[0]]
    for call in calls:
        first = call()
        wrong = sum(not torch.equal(call(), first) for _ in range(40))
        assert wrong == 0, wrong
