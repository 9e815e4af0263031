"""The adapter linear, its gradients and the 8-bit checkpoint in 64 bits, from their
definitions, with the bounds that the GPU results are held to.

Bounds.  EPS8 = 2^-8 is bf16's largest rounding error relative to the value.  ACC = 1e-5 times the
sum of magnitudes covers fp32 accumulation, as for the other linears (tolerance.py).  A low-rank
term passes through a row of fp32 sums (ACC of their magnitudes), is split into two bf16 parts
(off by at most 2^-17 = 0.76e-5 of the value) and summed again (ACC): 3 ACC of its magnitudes.
dx adds the one rounding of s_w * q to bf16: EPS8 times the magnitudes at most, and, rounding
errors being independent and at most EPS8 / sqrt(3) in the mean square (the weight's and the
result's together sqrt(2/3) EPS8), EPS8 in the norm.
"""
import torch

EPS8 = 2.0 ** -8
ACC = 1e-5


def make(M, N, K, R, L, seed, mix="each", free=0.2, bias=False, dy_std=2.0 ** -6):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)                      # noqa: E731
    x = rn(M, K)
    x[:, torch.randperm(K, generator=g)[: max(1, K // 512)]] *= 20.0
    W = rn(N, K) * 0.02
    s_w = torch.where(W.abs().amax(1) > 0, W.abs().amax(1) / 127.0, torch.ones(N))
    if mix == "each":
        ids = torch.randint(0, L, (M,), generator=g)
        ids[torch.rand(M, generator=g) < free] = -1
    elif mix == "runs":
        ids = torch.sort(torch.randint(0, L, (M,), generator=g)).values
        ids[M - int(free * M):] = -1
    elif mix == "none":
        ids = torch.full((M,), -1)
    else:                                           # ids that name no adapter, of every kind
        wild = torch.tensor([-1, L, L + 7, 2 ** 31 - 1, -2 ** 31, 0])
        ids = wild[torch.randint(0, 6, (M,), generator=g)]
    d = dict(x=x.bfloat16(), q=torch.round(W / s_w[:, None]).clamp(-127, 127).to(torch.int8),
             s_w=s_w, a=(rn(L, R, K) * K ** -0.5).bfloat16(), b=(rn(L, N, R) * 0.02).bfloat16(),
             scale=1.0 + torch.rand(L, generator=g), ids=ids.to(torch.int32),
             bias=rn(N) if bias else None, dy=(rn(M, N) * dy_std).bfloat16())
    return {k: None if v is None else v.cuda() for k, v in d.items()}


def _rows(d):
    for i in range(d["a"].shape[0]):
        rows = torch.nonzero(d["ids"] == i).flatten()
        if rows.numel():
            yield i, rows


def forward(d):
    """(y, h) and the bounds of (fp32 y, h)."""
    x, w = d["x"].double(), d["s_w"].double()[:, None] * d["q"].double()
    y, by = x @ w.t(), ACC * (x.abs() @ w.abs().t())
    if d["bias"] is not None:
        y += d["bias"].double()
        by += ACC * d["bias"].double().abs()
    h = torch.zeros(x.shape[0], d["a"].shape[1], dtype=torch.float64, device=x.device)
    bh = torch.zeros_like(h)
    for i, rows in _rows(d):
        a, b, c = d["a"][i].double(), d["b"][i].double(), d["scale"][i].double()
        h[rows] = x[rows] @ a.t()
        habs = x[rows].abs() @ a.abs().t()
        bh[rows] = ACC * habs
        y[rows] += c * (h[rows] @ b.t())
        by[rows] += 3 * ACC * c.abs() * (habs @ b.abs().t())
    return y, h, by + 1e-30, bh + 1e-30


def backward(d, h, xs):
    """(dx, da, db) and the bounds of each (dx's without its own rounding)."""
    dy, w = d["dy"].double(), d["s_w"].double()[:, None] * d["q"].double()
    dx, bx = dy @ w, (EPS8 + ACC) * (dy.abs() @ w.abs())
    da, db = torch.zeros(*d["a"].shape, dtype=torch.float64, device=dy.device), torch.zeros(
        *d["b"].shape, dtype=torch.float64, device=dy.device)
    ba, bb = torch.zeros_like(da), torch.zeros_like(db)
    for i, rows in _rows(d):
        a, b, c = d["a"][i].double(), d["b"][i].double(), d["scale"][i].double()
        g, gabs = c * (dy[rows] @ b), c.abs() * (dy[rows].abs() @ b.abs())
        dx[rows] += g @ a
        bx[rows] += 3 * ACC * (gabs @ a.abs())
        da[i] = g.t() @ xs[rows]
        ba[i] = 3 * ACC * (gabs.t() @ xs[rows].abs())
        db[i] = c * (dy[rows].t() @ h[rows].double())
        bb[i] = 3 * ACC * c.abs() * (dy[rows].abs().t() @ h[rows].double().abs())
    return dx, da, db, bx + 1e-30, ba + 1e-30, bb + 1e-30


def checkpoint(x, G):
    """(codes, exponent bytes) of the definition, in 64 bits."""
    M, K = x.shape
    v = x.double().view(M, K // G, G)
    top = v.abs().amax(2)
    e = torch.full_like(top, 121.0)
    for cand in range(120, -127, -1):               # the smallest exponent that still counts
        e = torch.where(top <= 127.0 * 2.0 ** cand, torch.full_like(e, float(cand)), e)
    step = torch.tensor([2.0 ** k for k in range(-126, 122)], dtype=torch.float64,
                        device=x.device)[(e + 126).long()].unsqueeze(2)
    c = torch.round(v / step).clamp(-127, 127).view(M, K)
    return c.to(torch.int8), (e + 127).to(torch.uint8)


def restore(codes, exps):
    M, K = codes.shape
    G = K // exps.shape[1]
    table = torch.tensor([2.0 ** (k - 127) for k in range(256)], dtype=torch.float64,
                         device=codes.device)
    return (codes.double().view(M, -1, G) * table[exps.long()].unsqueeze(2)).view(M, K)


def near(got, want, bound, what):
    err = (got.double() - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds; first at "
                             f"{at}: got {float(got[at])!r}, want {float(want[at])!r}, bound "
                             f"{float(bound[at])!r}")
