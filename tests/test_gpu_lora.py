"""The W8A16 linear with low-rank adapters and its backward pass against their definitions in
64 bits (lora_reference.py derives the bounds), at the sizes, ids and uses where they can go
wrong."""
import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
import lora_reference as ref

pytestmark = pytest.mark.gpu


def _forward(d, **kw):
    return q8.q8_linear_w8a16_lora(d["x"], d["q"], d["s_w"], d["a"], d["b"], d["scale"], d["ids"],
                                   bias=d["bias"], **kw)


def _backward(d, h, **kw):
    return q8.q8_linear_w8a16_lora_backward(d["dy"], d["q"], d["s_w"], d["a"], d["b"], d["scale"],
                                            d["ids"], h, **kw)


def _check_forward(d, out):
    y, h = _forward(d, out_dtype=out)
    wy, wh, by, bh = ref.forward(d)
    ref.near(h, wh, bh, "h")
    ref.near(y, wy, by + (ref.EPS8 * wy.abs() if out == torch.bfloat16 else 0.0), "y")
    assert q8.q8_last_device_status() == q8.Q8_OK
    return y, h


def _check_backward(d, G):
    h = ref.forward(d)[1].float()
    if G:
        codes, exps = ref.checkpoint(d["x"], G)
        xs, kw = ref.restore(codes, exps), dict(codes=codes, exps=exps)
    else:
        xs, kw = d["x"].double(), dict(x=d["x"])
    got = _backward(d, h, **kw)
    dx, da, db, bx, ba, bb = ref.backward(d, h, xs)
    ref.near(got[1], da, ba, "da")
    ref.near(got[2], db, bb, "db")
    ref.near(got[0], dx, bx + ref.EPS8 * dx.abs(), "dx")
    assert (got[0].double() - dx).norm() <= ref.EPS8 * dx.norm() + 1e-30
    assert q8.q8_last_device_status() == q8.Q8_OK
    return got, kw


# (M, N, K, R, L, ids): every tile edge, single rows, odd sizes, the smallest K, ranks that fill
# and cross the rank steps, ids in runs, in no order, none, and naming no adapter
FORWARD = [
    (1, 16, 64, 8, 1, "each"), (1, 2560, 960, 8, 1, "runs"), (2, 7, 16, 8, 3, "each"),
    (3, 1, 32, 16, 2, "wild"), (8, 130, 128, 24, 5, "each"), (9, 257, 320, 16, 4, "runs"),
    (15, 33, 960, 64, 7, "each"), (16, 2560, 960, 16, 32, "each"), (16, 64, 2048, 8, 2, "none"),
    (16, 100, 48, 40, 3, "each"), (17, 129, 80, 8, 3, "wild"), (31, 255, 112, 72, 2, "each"),
    (33, 256, 64, 16, 9, "runs"), (63, 300, 960, 128, 2, "each"), (64, 64, 64, 256, 1, "each"),
    (65, 513, 192, 32, 3, "each"), (77, 640, 512, 64, 8, "each"), (127, 31, 1024, 16, 2, "runs"),
    (128, 384, 256, 8, 128, "each"), (129, 200, 448, 136, 3, "runs"), (200, 96, 48, 8, 4, "none"),
    (255, 65, 96, 32, 5, "wild"), (256, 128, 128, 64, 3, "each"), (257, 1025, 144, 16, 6, "runs"),
    (333, 100, 960, 8, 3, "runs"), (513, 72, 208, 48, 20, "each"), (1000, 520, 320, 16, 1000, "each"),
    (1300, 264, 64, 8, 1024, "each"), (2051, 2561, 2080, 16, 5, "runs"), (2048, 5120, 1024, 40, 3, "each"),
]
BACKWARD = [
    (1, 16, 64, 8, 1, "each", 0), (1, 2560, 960, 8, 1, "runs", 64), (2, 8, 16, 8, 3, "each", 0),
    (3, 8, 32, 16, 2, "wild", 32), (16, 136, 128, 24, 5, "each", 128), (17, 128, 80, 8, 3, "wild", 0),
    (31, 256, 112, 72, 2, "each", 0), (33, 256, 64, 16, 9, "runs", 64), (64, 64, 64, 256, 1, "each", 32),
    (65, 520, 192, 32, 3, "each", 64), (77, 640, 512, 64, 8, "each", 256), (128, 384, 256, 8, 128, "each", 32),
    (129, 200, 448, 136, 3, "runs", 64), (200, 96, 48, 8, 4, "none", 0), (255, 72, 96, 32, 5, "wild", 32),
    (257, 1032, 144, 16, 6, "runs", 0), (333, 104, 960, 8, 3, "runs", 32), (513, 72, 224, 48, 20, "each", 32),
    (1000, 520, 320, 16, 1000, "each", 64), (700, 264, 4096, 64, 2, "runs", 128),
    (2051, 2568, 2080, 16, 5, "runs", 32), (2048, 5120, 1024, 40, 3, "each", 0),
]


@pytest.mark.parametrize("M,N,K,R,L,mix", FORWARD)
def test_forward(M, N, K, R, L, mix):
    d = ref.make(M, N, K, R, L, seed=M * 31 + N, mix=mix, bias=M % 2 == 0)
    _check_forward(d, torch.float32)
    _check_forward(d, torch.bfloat16)


@pytest.mark.parametrize("M,N,K,R,L,mix,G", BACKWARD)
def test_backward(M, N, K, R, L, mix, G):
    _check_backward(ref.make(M, N, K, R, L, seed=M * 37 + N, mix=mix), G)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_rows_without_an_adapter_are_the_plain_linear(M):
    """Their h is 0 and y is q8_linear_w8a16's sum, whatever the pool holds (it is not read)."""
    d = ref.make(M, 96, 128, 16, 3, seed=5, mix="none", bias=True)
    d["a"].fill_(float("nan"))
    d["b"].fill_(float("inf"))
    d["scale"].fill_(float("nan"))
    y, h = _forward(d, out_dtype=torch.float32)
    assert torch.equal(h, torch.zeros_like(h))
    wy, _, by, _ = ref.forward(d)
    ref.near(y, wy, by, "y")
    plain = q8.q8_linear_w8a16(d["x"], d["q"], d["s_w"], out_dtype=torch.float32, bias=d["bias"])
    ref.near(y, plain.double(), 2 * by, "y against the plain linear")
    dx, da, db = _backward(d, h, x=d["x"])
    assert torch.equal(da, torch.zeros_like(da)) and torch.equal(db, torch.zeros_like(db))
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("M", [4, 16, 50, 300])
def test_unused_adapters_are_not_read(M):
    d = ref.make(M, 136, 192, 16, 4, seed=6, mix="each")
    d["ids"][d["ids"] == 2] = 1
    clean = [t.clone() for t in (*_forward(d), *_backward(d, ref.forward(d)[1].float(), x=d["x"]))]
    for k in ("a", "b", "scale"):
        d[k][2] = float("nan")
    d2 = dict(d)
    y, h = _forward(d2)
    wh = torch.where((d["ids"] >= 0)[:, None], h, torch.zeros_like(h))
    dx, da, db = _backward(d2, wh, x=d["x"])
    assert torch.equal(y, clean[0]) and torch.equal(h, clean[1])
    assert torch.isfinite(dx).all() and torch.isfinite(da).all() and torch.isfinite(db).all()
    assert not da[2].any() and not db[2].any()


@pytest.mark.parametrize("M", [3, 16, 70, 400])
def test_rows_do_not_touch_each_other(M):
    """A non-finite activation (a padding row, say) stays in its own row of y, h and dx, and a
    row without an adapter stays out of da and db."""
    d = ref.make(M, 104, 160, 8, 2, seed=7, mix="each")
    d["ids"][1] = -1
    y0, h0 = _forward(d)
    g0 = _backward(d, h0, x=d["x"])
    d["x"][1] = float("inf")
    d["dy"][1] = float("nan")
    y, h = _forward(d)
    rest = torch.arange(M, device="cuda") != 1
    assert torch.equal(y[rest], y0[rest]) and torch.equal(h, h0)
    g = _backward(d, h, x=d["x"])
    assert torch.equal(g[0][rest], g0[0][rest])
    assert torch.equal(g[1], g0[1]) and torch.equal(g[2], g0[2])


def test_extreme_scales_of_weights_and_adapters():
    """Row scales from the smallest normal number up, adapters far larger and smaller than the
    base term: nothing overflows or is lost on the way."""
    d = ref.make(40, 128, 256, 16, 2, seed=8, mix="each", free=0.0)
    d["s_w"] = torch.logspace(-37, 3, 128, device="cuda")
    d["b"][0] *= 2.0 ** 20
    d["b"][1] *= 2.0 ** -20
    _check_forward(d, torch.float32)
    d16 = {k: v if k not in ("x", "dy", "ids") else v[:16].contiguous() for k, v in d.items()}
    _check_forward(d16, torch.float32)


@pytest.mark.parametrize("M,G", [(5, 0), (16, 32), (300, 64)])
def test_accumulate_and_partial_gradients(M, G):
    d = ref.make(M, 200, 320, 24, 3, seed=9, mix="runs")
    (dx, da, db), kw = _check_backward(d, G)
    h = ref.forward(d)[1].float()
    a0, b0 = torch.randn_like(da), torch.randn_like(db)
    a1, b1 = a0.clone(), b0.clone()
    none, a2, b2 = _backward(d, h, want_dx=False, da=a1, db=b1, accumulate=True, **kw)
    assert none is None and a2 is a1 and b2 is b1
    # one fp32 addition of the same gradient, in either order of rounding
    assert ((a1 - (a0 + da)).abs() <= 2.0 ** -23 * (a0.abs() + da.abs())).all()
    assert ((b1 - (b0 + db)).abs() <= 2.0 ** -23 * (b0.abs() + db.abs())).all()
    only = _backward(d, None, want_da=False, want_db=False)
    assert torch.equal(only[0], dx) and only[1] is None and only[2] is None
    only = _backward(d, h, want_dx=False, want_da=False)
    assert torch.equal(only[2], db)
    only = _backward(d, None, want_dx=False, want_db=False, **kw)
    assert torch.equal(only[1], da)


def test_empty_batch():
    d = ref.make(1, 64, 64, 8, 2, seed=10)
    e = {k: (v[:0].contiguous() if k in ("x", "dy", "ids") else v) for k, v in d.items()}
    y, h = _forward(e)
    assert y.shape == (0, 64) and h.shape == (0, 8)
    da, db = torch.ones(2, 8, 64, device="cuda"), torch.ones(2, 64, 8, device="cuda")
    _backward(e, h, x=e["x"], da=da, db=db, accumulate=True)
    assert (da == 1).all() and (db == 1).all()
    dx, da, db = _backward(e, h, x=e["x"])
    assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_outputs_stay_in_their_bounds():
    """Rows behind the batch and columns behind the tile are left as they were."""
    for M, N in ((5, 40), (16, 24), (37, 136), (260, 264)):
        d = ref.make(M, N, 96, 8, 2, seed=11 + M, mix="each")
        big = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
        hb = torch.full((M + 3, 8), 7.0, device="cuda")
        _forward(d, y=big[:M], h=hb[:M])
        assert (big[M:] == 7).all() and (hb[M:] == 7).all()
        dxb = torch.full((M + 3, 96), 7.0, dtype=torch.bfloat16, device="cuda")
        dab = torch.full((3, 8, 96), 7.0, device="cuda")
        dbb = torch.full((3, N, 8), 7.0, device="cuda")
        _backward(d, hb[:M].contiguous(), x=d["x"], dx=dxb[:M], da=dab[:2], db=dbb[:2])
        assert (dxb[M:] == 7).all() and (dab[2] == 7).all() and (dbb[2] == 7).all()
        assert not (big[:M] == 7).all()


@pytest.mark.parametrize("M,mix", [(16, "each"), (300, "runs"), (500, "each")])
def test_same_bits_every_time(M, mix):
    d = ref.make(M, 264, 512, 16, 5, seed=12, mix=mix)
    codes, exps = q8.q8_checkpoint_save(d["x"], 64)
    y0, h0 = _forward(d)
    g0 = _backward(d, h0, codes=codes, exps=exps)
    for _ in range(5):
        y, h = _forward(d)
        g = _backward(d, h, codes=codes, exps=exps)
        assert torch.equal(y, y0) and torch.equal(h, h0)
        assert all(torch.equal(u, v) for u, v in zip(g, g0))


@pytest.mark.parametrize("M", [16, 300])
def test_other_stream_and_two_at_once(M):
    """Calls on two side streams at once, each with its own workspace, and the `stream`
    argument from a stream that is not current."""
    ds = [ref.make(M, 520, 512, 16, 4, seed=13 + s, mix="each") for s in range(2)]
    want = [(*_forward(d), *_backward(d, _forward(d)[1], x=d["x"])) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, (d, s) in enumerate(zip(ds, streams)):
            y, h = _forward(d, stream=s)
            got[i] = (y, h, *_backward(d, h, x=d["x"], stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(w, g))
    with torch.cuda.stream(streams[0]):
        y, h = _forward(ds[0])
    torch.cuda.synchronize()
    assert torch.equal(y, want[0][0])


@pytest.mark.parametrize("M", [1, 16, 130])
def test_captured_and_replayed(M):
    """A forward and backward pass in one graph, replayed on new inputs, next to eager calls."""
    d = ref.make(M, 264, 256, 8, 3, seed=14, mix="each")
    codes, exps = q8.q8_checkpoint_save(d["x"], 32)

    def step():
        y, h = _forward(d)
        q8.q8_checkpoint_save(d["x"], 32, codes=codes, exps=exps)
        return (y, h, *_backward(d, h, codes=codes, exps=exps))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (15, 16):
        n = ref.make(M, 264, 256, 8, 3, seed=seed, mix="runs")
        for k in ("x", "ids", "dy", "a", "b"):
            d[k].copy_(n[k])
        g.replay()
        eager = step()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, eager))


def test_gradients_against_differences():
    """y is linear in x, in a and in b, each alone: a difference of two forward passes is the
    gradient, whatever the step.  Steps are powers of two that keep every input a bf16 number."""
    d = ref.make(70, 72, 64, 8, 2, seed=17, mix="each")
    for k, unit in (("x", 64), ("a", 64), ("b", 64)):
        d[k] = (torch.round(d[k].float() * unit) / unit).clamp(-3.9, 3.9).bfloat16()
    y0, h = _forward(d, out_dtype=torch.float32)
    dx, da, db = _backward(d, h, x=d["x"])
    _, _, by, _ = ref.forward(d)
    dy = d["dy"].double()
    slack = 2 * (by * dy.abs()).sum().item()             # what two sums of y may be off
    for k, grad, step in (("x", dx, 0.25), ("a", da, 0.25), ("b", db, 0.25)):
        flat = grad.reshape(-1)
        for at in range(0, flat.numel(), flat.numel() // 7):
            n = dict(d)
            n[k] = d[k].clone()
            n[k].view(-1)[at] += step
            real = float(n[k].view(-1)[at]) - float(d[k].view(-1)[at])
            y1, _ = _forward(n, out_dtype=torch.float32)
            diff = float(((y1.double() - y0.double()) * dy).sum()) / real
            # dx: rounded weight and result (EPS8 of the magnitudes each); da, db: fp32 sums
            mag = float((dy.abs() @ (d["s_w"].double()[:, None] * d["q"].double()).abs()).max())
            tol = slack / abs(real) + (2 * ref.EPS8 * mag if k == "x" else 1e-4 * abs(diff))
            assert abs(float(flat[at]) - diff) <= tol, (k, at, float(flat[at]), diff, tol)


def test_binding_refusals():
    d = ref.make(4, 64, 64, 8, 2, seed=18)
    with pytest.raises(ValueError):
        _forward(dict(d, ids=d["ids"].long()))
    with pytest.raises(ValueError):
        _forward(dict(d, a=d["a"].float()))
    with pytest.raises(ValueError):
        _forward(dict(d, b=d["b"].transpose(1, 2)))
    with pytest.raises(ValueError):
        _forward(dict(d, x=d["x"].t().contiguous().t()))
    with pytest.raises(ValueError):
        _forward(d, out_dtype=torch.float16)
    with pytest.raises(q8.Q8Error):
        _forward(dict(d, a=d["a"][:, :4].contiguous(), b=d["b"][:, :, :4].contiguous()))
    y, h = _forward(d)
    with pytest.raises(ValueError):
        _backward(d, h)                                          # no input
    with pytest.raises(ValueError):
        _backward(d, None, x=d["x"])                             # no h
    with pytest.raises(ValueError):
        _backward(d, h, x=d["x"], accumulate=True)               # nothing to add to
    with pytest.raises(ValueError):
        _backward(d, h.cpu(), x=d["x"])
