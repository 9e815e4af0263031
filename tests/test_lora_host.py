"""Refusals of the adapter and checkpoint entry points: every documented status code comes
from the arguments alone, before any device work (no GPU needed)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import int8_quantized_linear_q8_b200 as q8
from int8_quantized_linear_q8_b200 import build as q8build

GOOD, ODD, ODD4 = 0x10000, 0x10001, 0x10002      # addresses that are never dereferenced
FWD, BWD = q8.Q8_OP_LINEAR_W8A16_LORA, q8.Q8_OP_LINEAR_W8A16_LORA_BACKWARD


@pytest.fixture(scope="module")
def L():
    q8build.build()
    return q8.lib()


def _ad(a=GOOD, b=GOOD, scale=GOOD, count=2, rank=16):
    return ctypes.byref(q8.q8_adapters(a, b, scale, count, rank))


def _saved(x=GOOD, exps=GOOD, group=32):
    return ctypes.byref(q8.q8_saved_input(x, exps, group))


def _fwd(L, **k):
    c = dict(x=GOOD, q=GOOD, s=GOOD, bias=None, ad=_ad(), ids=GOOD, y=GOOD, yt=q8.Q8_BF16, h=GOOD,
             M=4, N=32, K=64, ws=GOOD, wsb=1 << 40)
    c.update(k)
    return L.q8_linear_w8a16_lora(c["x"], c["q"], c["s"], c["bias"], c["ad"], c["ids"], c["y"],
                                  c["yt"], c["h"], c["M"], c["N"], c["K"], c["ws"], c["wsb"], None)


def _bwd(L, **k):
    c = dict(dy=GOOD, q=GOOD, s=GOOD, ad=_ad(), ids=GOOD, h=GOOD, inp=_saved(), dx=GOOD, da=GOOD,
             db=GOOD, acc=0, M=4, N=32, K=64, ws=GOOD, wsb=1 << 40)
    c.update(k)
    return L.q8_linear_w8a16_lora_backward(c["dy"], c["q"], c["s"], c["ad"], c["ids"], c["h"],
                                           c["inp"], c["dx"], c["da"], c["db"], c["acc"], c["M"],
                                           c["N"], c["K"], c["ws"], c["wsb"], None)


def test_forward_refusals(L):
    assert _fwd(L, yt=7) == q8.Q8_ERR_ARG
    for bad in (dict(M=-1), dict(M=1 << 31), dict(M=(1 << 31) - 1), dict(N=1 << 30), dict(N=0), dict(K=40), dict(K=8), dict(K=65536)):
        assert _fwd(L, **bad) == q8.Q8_ERR_SHAPE, bad
    for ad in (_ad(count=0), _ad(count=1025), _ad(rank=0), _ad(rank=4), _ad(rank=20),
               _ad(rank=264)):
        assert _fwd(L, ad=ad) == q8.Q8_ERR_ARG
    assert _fwd(L, ad=None) == q8.Q8_ERR_NULL
    for name in ("x", "q", "s", "y", "h", "ids"):
        assert _fwd(L, **{name: None}) == q8.Q8_ERR_NULL, name
    for ad in (_ad(a=None), _ad(b=None), _ad(scale=None)):
        assert _fwd(L, ad=ad) == q8.Q8_ERR_NULL
    for name in ("x", "q", "y", "h"):
        assert _fwd(L, **{name: ODD}) == q8.Q8_ERR_ALIGN, name
    for name in ("s", "bias", "ids"):
        assert _fwd(L, **{name: ODD4}) == q8.Q8_ERR_ALIGN, name
    for ad in (_ad(a=ODD), _ad(b=ODD), _ad(scale=ODD4)):
        assert _fwd(L, ad=ad) == q8.Q8_ERR_ALIGN
    need = q8.q8_workspace_bytes(FWD, 40, 32, 64, 16)
    assert need > 0
    assert _fwd(L, M=40, wsb=need - 1) == q8.Q8_ERR_WORKSPACE
    assert _fwd(L, M=40, ws=None) == q8.Q8_ERR_WORKSPACE
    assert _fwd(L, M=40, ws=ODD) == q8.Q8_ERR_ALIGN
    assert _fwd(L, M=0, x=None, y=None, h=None, ids=None) == q8.Q8_OK


def test_backward_refusals(L):
    for bad in (dict(M=-1), dict(N=0), dict(N=12), dict(K=40)):
        assert _bwd(L, **bad) == q8.Q8_ERR_SHAPE, bad
    assert _bwd(L, ad=None) == q8.Q8_ERR_NULL
    assert _bwd(L, ad=_ad(rank=12)) == q8.Q8_ERR_ARG
    assert _bwd(L, inp=None) == q8.Q8_ERR_NULL
    assert _bwd(L, inp=_saved(group=48)) == q8.Q8_ERR_ARG
    assert _bwd(L, inp=_saved(group=128)) == q8.Q8_ERR_SHAPE           # K = 64
    assert _bwd(L, inp=_saved(x=None)) == q8.Q8_ERR_NULL
    assert _bwd(L, inp=_saved(exps=None)) == q8.Q8_ERR_NULL
    assert _bwd(L, inp=_saved(x=ODD)) == q8.Q8_ERR_ALIGN
    for name in ("dy", "q", "s", "h", "ids"):
        assert _bwd(L, **{name: None}) == q8.Q8_ERR_NULL, name
    for name in ("dy", "q", "dx", "da", "db", "h"):
        assert _bwd(L, **{name: ODD}) == q8.Q8_ERR_ALIGN, name
    need = q8.q8_workspace_bytes(BWD, 4, 32, 64, 16)
    assert need > 0
    assert _bwd(L, wsb=need - 1) == q8.Q8_ERR_WORKSPACE
    assert _bwd(L, ws=None) == q8.Q8_ERR_WORKSPACE
    assert _bwd(L, ws=ODD) == q8.Q8_ERR_ALIGN
    assert _bwd(L, dx=None, da=None, db=None) == q8.Q8_OK
    assert _bwd(L, M=0, acc=1) == q8.Q8_OK


def test_workspace_sizes(L):
    for op in (FWD, BWD):
        assert q8.q8_workspace_bytes(op, 0, 32, 64, 16) >= 0
        assert q8.q8_workspace_bytes(op, 4, 32, 64, 12) == 0             # invalid rank
        assert q8.q8_workspace_bytes(op, 4, 32, 63, 16) == 0             # invalid K


def test_checkpoint_refusals(L):
    save = lambda **k: (lambda c: L.q8_checkpoint_save(                          # noqa: E731
        c["x"], c["xt"], c["M"], c["K"], c["G"], c["c"], c["e"], None))(
            dict(dict(x=GOOD, xt=q8.Q8_BF16, M=4, K=64, G=32, c=GOOD, e=GOOD), **k))
    load = lambda **k: (lambda c: L.q8_checkpoint_load(                          # noqa: E731
        c["c"], c["e"], c["G"], c["y"], c["yt"], c["M"], c["K"], None))(
            dict(dict(y=GOOD, yt=q8.Q8_BF16, M=4, K=64, G=32, c=GOOD, e=GOOD), **k))
    for f, t, p in ((save, "xt", "x"), (load, "yt", "y")):
        assert f(**{t: 5}) == q8.Q8_ERR_ARG
        assert f(G=16) == q8.Q8_ERR_ARG
        assert f(G=128) == q8.Q8_ERR_SHAPE
        assert f(M=-1) == q8.Q8_ERR_SHAPE
        assert f(K=65536) == q8.Q8_ERR_SHAPE
        for name in (p, "c", "e"):
            assert f(**{name: None}) == q8.Q8_ERR_NULL
        for name in (p, "c"):
            assert f(**{name: ODD}) == q8.Q8_ERR_ALIGN
        assert f(M=0, **{p: None}) == q8.Q8_OK
    wg = lambda **k: (lambda c: L.q8_checkpoint_wgrad(                           # noqa: E731
        c["dy"], c["c"], c["e"], c["G"], c["dw"], c["acc"], c["M"], c["N"], c["K"], c["ws"],
        c["wsb"], None))(
            dict(dict(dy=GOOD, c=GOOD, e=GOOD, G=32, dw=GOOD, acc=0, M=4, N=32, K=64, ws=None,
                      wsb=0), **k))
    assert wg(G=8) == q8.Q8_ERR_ARG
    for bad in (dict(N=12), dict(N=0), dict(M=-1), dict(K=48), dict(G=256)):
        assert wg(**bad) == q8.Q8_ERR_SHAPE, bad
    for name in ("dy", "c", "e", "dw"):
        assert wg(**{name: None}) == q8.Q8_ERR_NULL
    for name in ("dy", "c", "dw"):
        assert wg(**{name: ODD}) == q8.Q8_ERR_ALIGN
    assert wg(M=0, acc=1, dy=None) == q8.Q8_OK
    need = q8.q8_workspace_bytes(q8.Q8_OP_CHECKPOINT_WGRAD, 4096, 65536, 64)
    assert need > 0
    assert wg(M=4096, N=65536) == q8.Q8_ERR_WORKSPACE
    assert wg(M=4096, N=65536, ws=GOOD, wsb=need - 1) == q8.Q8_ERR_WORKSPACE
    assert wg(M=4096, N=65536, ws=ODD, wsb=need) == q8.Q8_ERR_ALIGN


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_c99_caller(tmp_path, L):
    here = os.path.dirname(os.path.abspath(__file__))
    libdir, exe = os.path.dirname(q8.LIB_PATH), str(tmp_path / "c_abi_lora_check")
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic",
                           "-I", os.path.join(os.path.dirname(here), "include"),
                           os.path.join(here, "c_abi_lora_check.c"), "-L", libdir, "-lq8",
                           "-Wl,-rpath," + libdir, "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and "failures: 0" in out.stdout, out.stdout + out.stderr


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q8.q8_checkpoint_save(x, 32)
    with pytest.raises(ValueError):
        q8.q8_checkpoint_load(torch.zeros(2, 64, dtype=torch.int8),
                              torch.zeros(2, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        q8.q8_linear_w8a16_lora(x, torch.zeros(16, 64, dtype=torch.int8), torch.ones(16),
                                torch.zeros(1, 8, 64, dtype=torch.bfloat16),
                                torch.zeros(1, 16, 8, dtype=torch.bfloat16), torch.ones(1),
                                torch.zeros(2, dtype=torch.int32))
