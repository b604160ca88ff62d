"""Refusals and host-only parts of the operators around the linear layer, and
pins of their plain forms (CPU; nothing reaches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_lora_02_b200 as Q
from oracle import step_oracle as SO

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def L():
    from bit_quantized_lora_02_b200 import build
    build.build()
    return Q.lib()


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def test_norm_refusals_of_the_binding():
    X, w = torch.zeros(4, 64, dtype=BF16), torch.ones(64)
    s = torch.zeros(4)
    for kw, match in ((dict(weight=torch.ones(63)), "weight: shape"), (dict(bias=torch.ones(64, dtype=BF16)), "bias: dtype"),
                      (dict(residual=torch.zeros(4, 64)), "residual: dtype"), (dict(S=X), "S goes with residual"),
                      (dict(Y=torch.zeros(4, 64)), "Y: dtype"), (dict(mean=torch.zeros(3)), "mean: shape"),
                      (dict(mean=s, rms=True), "mean is not used"), (dict(weight=torch.ones(64, dtype=torch.float16)), "weight: dtype"),
                      ({}, "must be on a CUDA device")):
        args = dict(weight=w)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            Q.qlora_layer_norm_fwd(X, **args)
    with pytest.raises(ValueError, match="contiguous"):
        Q.qlora_layer_norm_fwd(torch.zeros(64, 4, dtype=BF16).t(), w)
    with pytest.raises(ValueError, match="expected \\(rows, values\\)"):
        Q.qlora_layer_norm_fwd(torch.zeros(64, dtype=BF16), w)
    with pytest.raises(ValueError, match="X: dtype"):
        Q.qlora_layer_norm_fwd(torch.zeros(4, 64, dtype=torch.float16), w)
    for kw, match in ((dict(mean=None), "mean is required"), (dict(dY=torch.zeros(4, 64)), "dY: dtype"),
                      (dict(dS=torch.zeros(3, 64, dtype=BF16)), "dS: shape"), (dict(dbias=torch.zeros(64, dtype=BF16)), "dbias: dtype"),
                      ({}, "must be on a CUDA device")):
        args = dict(dY=X, S=X, weight=w, mean=s, rstd=s)
        args.update(kw)
        with pytest.raises(ValueError, match=match):
            Q.qlora_layer_norm_bwd(**args)


def test_norm_refusals_of_the_library(L):
    def n(M=4, D=64, dt=0, wdt=1, rms=0, eps=1e-5):
        return ctypes.byref(Q.QloraNorm(M, D, dt, wdt, rms, eps))

    def fwd(d, X=0x1000, R=None, w=0x2000, b=None, S=None, Y=0x3000, mean=0x4000, rstd=0x5000):
        return L.qlora_layer_norm_fwd(d, X, R, w, b, S, Y, mean, rstd, None)
    assert fwd(None) == -1
    assert fwd(n(M=-1)) == -1 and fwd(n(D=0)) == -1
    assert fwd(n(D=16385)) == -2 and b"D=16385" in L.qlora_last_error()
    assert fwd(n(dt=2)) == -1 and fwd(n(wdt=-1)) == -1 and fwd(n(eps=float("nan"))) == -1 and fwd(n(eps=-1.0)) == -1
    assert fwd(n(), X=None) == -1 and fwd(n(), w=None) == -1 and fwd(n(), Y=None) == -1
    assert fwd(n(), X=0x1008) == -3 and fwd(n(), Y=0x3002) == -3 and fwd(n(), mean=0x4002) == -3
    assert fwd(n(), R=0x6000) == -1 and fwd(n(), S=0x6000) == -1          # S goes with R
    assert fwd(n(M=0), X=None, Y=None) == 0                                # nothing to do
    size = ctypes.c_size_t()
    assert L.qlora_layer_norm_workspace_size(n(), 0, None) == -1
    assert L.qlora_layer_norm_workspace_size(n(D=16385), 0, ctypes.byref(size)) == -2
    assert L.qlora_layer_norm_workspace_size(n(M=0), 1, ctypes.byref(size)) == 0 and size.value == 0
    assert L.qlora_layer_norm_workspace_size(n(M=1, D=100), 0, ctypes.byref(size)) == 0 and size.value == 512
    assert L.qlora_layer_norm_workspace_size(n(M=1, D=100), 1, ctypes.byref(size)) == 0 and size.value == 1024

    def bwd(d, dY=0x1000, S=0x2000, w=0x3000, mean=0x4000, rstd=0x5000, dS=None, dX=0x6000, dw=0x7000, db=None):
        return L.qlora_layer_norm_bwd(d, dY, S, w, mean, rstd, dS, dX, dw, db, None, 0, None)
    assert bwd(n(), dY=None) == -1 and bwd(n(), mean=None) == -1 and bwd(n(), dw=None) == -1 and bwd(n(), rstd=None) == -1
    assert bwd(n(), dS=0x9000, dX=None) == -1
    assert bwd(n(), dX=0x6004) == -3 and bwd(n(), db=0x8004) == -3


def test_norm_oracle_gradient():
    """The plain backward against central differences of the plain forward: step
    1e-5 in 64 bits leaves 1e-10 of truncation and 1e-16 / 1e-5 of rounding."""
    rng = np.random.default_rng(0)
    x, w, b, dy, ds = rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=11), rng.normal(size=(3, 11)), rng.normal(size=(3, 11))
    for rms in (False, True):
        def f(x_, w_, b_):
            return (SO.norm_forward(x_, w_, b_, 1e-3, rms)[0] * dy).sum() + (x_ * ds).sum()
        _, mean, rstd = SO.norm_forward(x, w, b, 1e-3, rms)
        dx, dw, db = SO.norm_backward(dy, x, w, mean, rstd, ds, rms)
        for at in ((0, 0), (2, 10), (1, 5)):
            for k, (t, g) in enumerate(((x, dx[at]), (w, dw[at[1]]), (b, db[at[1]]))):
                i = at if k == 0 else at[1]
                lo, hi = t.copy(), t.copy()
                lo[i] -= 1e-5
                hi[i] += 1e-5
                args = [x, w, b]
                num = (f(*(hi if j == k else a for j, a in enumerate(args))) - f(*(lo if j == k else a for j, a in enumerate(args)))) / 2e-5
                assert abs(num - g) < 1e-7
