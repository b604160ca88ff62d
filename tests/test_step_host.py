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
    assert fwd(n(), R=0x6000, S=0x3000) == -1                             # S and Y in one place
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


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
def test_adamw_refusals_of_the_binding():
    p, g = [torch.zeros(4, 8), torch.zeros(3)], [torch.zeros(4, 8), torch.zeros(3)]
    for args, kw, match in (((p, g), {}, "must be on a CUDA device"), ((p, g[:1]), {}, "1 tensors for 2"),
                            ((p, [g[0], torch.zeros(4)]), {}, "grads\\[1\\]: shape"),
                            ((p, [g[0], torch.zeros(3, dtype=BF16)]), {}, "grads\\[1\\]: dtype"),
                            (([], []), {}, "no parameters"), ((p, g), dict(state_bits=16), "state_bits"),
                            ((p, g), dict(copies=p), "copies are bf16"),
                            (([p[0], p[0]], [g[0], g[0]]), {}, "overlap"),
                            (([torch.zeros(8, 4).t()], [torch.zeros(4, 8)]), {}, "contiguous"),
                            (([torch.zeros(3, dtype=torch.float16)], [torch.zeros(3)]), {}, "params: dtype")):
        with pytest.raises(ValueError, match=match):
            Q.qlora_adamw_alloc(*args, **kw)
    flat = torch.zeros(64)
    with pytest.raises(ValueError, match="overlap"):
        Q.qlora_adamw_alloc([flat[:40], flat[32:]], [torch.zeros(40), torch.zeros(32)])


def test_adamw_refusals_of_the_library(L):
    def opt(pd=1, gd=1, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, step=1, scale=None, clock=None):
        return ctypes.byref(Q.QloraAdamW(pd, gd, bits, lr, b1, b2, eps, wd, step, scale, clock))

    def one(param=0x1000, copy=None, grad=0x2000, n=100, m=0x3000, v=0x4000, ms=None, vs=None):
        return (Q.QloraAdamWTensor * 1)(Q.QloraAdamWTensor(param, copy, grad, n, m, v, ms, vs))
    step = L.qlora_adamw_step
    assert step(None, one(), 1, None) == -1
    assert step(opt(), None, 1, None) == -1 and step(opt(), one(), -1, None) == -1
    assert step(opt(), None, 0, None) == 0 and step(opt(), one(n=0), 1, None) == 0     # nothing to do
    assert step(opt(pd=2), one(), 1, None) == -1 and step(opt(gd=-1), one(), 1, None) == -1
    assert step(opt(bits=16), one(), 1, None) == -2
    for kw in (dict(b1=1.0), dict(b1=-0.1), dict(b2=float("nan")), dict(eps=-1.0), dict(wd=-1.0), dict(lr=float("nan")),
               dict(lr=-1.0), dict(step=0)):
        assert step(opt(**kw), one(), 1, None) == -1, kw
    assert step(opt(clock=0x1004), one(), 1, None) == -3 and step(opt(scale=0x1002), one(), 1, None) == -3
    for kw in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1)):
        assert step(opt(), one(**kw), 1, None) == -1, kw
    assert step(opt(bits=8), one(), 1, None) == -1                                     # no scales
    assert step(opt(pd=0), one(copy=0x5000), 1, None) == -1                            # a copy beside bf16
    for kw in (dict(param=0x1008), dict(grad=0x2004), dict(m=0x3008), dict(copy=0x5008)):
        assert step(opt(), one(**kw), 1, None) == -3, kw
    two = (Q.QloraAdamWTensor * 2)(one()[0], one(copy=0x5000)[0])
    assert step(opt(), two, 2, None) == -1                                             # copies for all or none
    vals = L.qlora_adamw_state_values
    assert vals(0, None, None, None, None, None, None, None) == 0 and vals(-1, None, None, None, None, None, None, None) == -1
    assert vals(10, None, 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, None) == -1
    assert vals(10, 0x1004, 0x1000, 0x1000, 0x1000, 0x1000, 0x1000, None) == -3
    assert vals(10, 0x1000, 0x1000, 0x1000, 0x1000, 0x1008, 0x1000, None) == -3


def test_adamw_oracle_codes():
    """E4M3 codes against torch's conversion for every code, every midpoint and
    random values; coded states against their own error bounds (half a step: 2^-4
    of m above the subnormals, half a code of the fourth root)."""
    vals = SO.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(vals), np.isnan(t)) and np.array_equal(vals[~np.isnan(vals)], t[~np.isnan(t)])
    pos = np.sort(vals[:127])
    y = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, np.random.default_rng(0).uniform(-448, 448, 1000)]).astype(np.float32)
    y = np.concatenate([y, -y])
    assert np.array_equal(SO.e4m3_code(y), torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    rng = np.random.default_rng(1)
    m, v = rng.normal(size=1000).astype(np.float32), (rng.normal(size=1000) ** 2).astype(np.float32)
    mc, ms, vc, vs = SO.adamw_encode(m, v)
    dm, dv = SO.adamw_decode(mc, ms, vc, vs)
    j = np.arange(1000) // 256
    assert ms.shape == (4,) and np.all(np.abs(dm - m) <= np.maximum(2.0 ** -4 * np.abs(m), ms[j] / 448 * 2.0 ** -10) * 1.0001)
    root, got = v.astype(np.float64) ** 0.25, dv.astype(np.float64) ** 0.25
    assert np.all(np.abs(got - root) <= vs[j] / 255 * 0.5001 + 1e-6)
    assert np.all(vc[v > 0] >= 1)


def test_adamw_oracle_step():
    """The plain step against a hand-worked value: p = 1, g = 0.5, first step: m' =
    0.05, v' = 0.00025, both corrected to 0.5 and 0.25, so the update is lr."""
    p, m, v = SO.adamw_param(np.array([1.0]), np.zeros(1), np.zeros(1), np.array([0.5]), 1, 0.1, 0.9, 0.999, 0.0, 0.2)
    assert np.allclose(p, 1.0 * (1 - 0.02) - 0.1) and np.allclose(m, 0.05) and np.allclose(v, 0.00025)


# ---------------------------------------------------------------------------
# log probabilities of given tokens
# ---------------------------------------------------------------------------
def test_logprobs_refusals_of_the_binding():
    z, t = torch.zeros(4, 64, dtype=BF16), torch.zeros(4, dtype=torch.int64)
    s = torch.zeros(4)
    for args, kw, match in (((z, t), {}, "must be on a CUDA device"), ((z, t.int()), {}, "targets: dtype"),
                            ((z, t[:3]), {}, "targets: shape"), ((z[0], t), {}, "expected \\(tokens, vocabulary\\)"),
                            ((z, t), dict(vocab=65), "vocab=65"), ((z, t), dict(vocab=0), "vocab=0"),
                            ((torch.zeros(64, 4, dtype=BF16).t(), t), {}, "strides"),
                            ((torch.zeros(1, 64).expand(4, 64), t), {}, "strides"),
                            ((z.half(), t), {}, "logits: dtype"),
                            ((z, t), dict(out=Q.TokenLogprobs(s, s), entropy=True), "other results"),
                            ((z, t), dict(out=Q.TokenLogprobs(s[:3], s)), "out.logp: shape")):
        with pytest.raises(ValueError, match=match):
            Q.qlora_token_logprobs_fwd(*args, **kw)
    for args, kw, match in (((z, t, s, s), {}, "must be on a CUDA device"), ((z, t, s, None), {}, "dlogp is required"),
                            ((z, t, s, s), dict(dentropy=s), "dentropy needs entropy"),
                            ((z, t, s[:2], s), {}, "lse: shape"), ((z, t, s, s.double()), {}, "dlogp: dtype"),
                            ((z, t, s, s), dict(dlogits=torch.zeros(4, 64)), "dlogits must have")):
        with pytest.raises(ValueError, match=match):
            Q.qlora_token_logprobs_bwd(*args, **kw)


def test_logprobs_refusals_of_the_library(L):
    def d(N=4, V=100, ld=100, dt=0, top=0):
        return ctypes.byref(Q.QloraLogits(N, V, ld, dt, top))

    def fwd(l, z=0x1000, t=0x2000, logp=0x3000, lse=0x4000, ent=None, ids=None, tl=None):
        return L.qlora_token_logprobs_fwd(l, z, t, logp, lse, ent, ids, tl, None)
    assert fwd(None) == -1 and fwd(d(N=-1)) == -1 and fwd(d(V=0)) == -1 and fwd(d(ld=99)) == -1 and fwd(d(dt=2)) == -1
    assert fwd(d(V=(1 << 30) + 1, ld=1 << 31)) == -2 and fwd(d(N=1 << 31, ld=1 << 40)) == -1
    assert fwd(d(top=33), ids=0x5000, tl=0x6000) == -2 and fwd(d(V=3, ld=3, top=4), ids=0x5000, tl=0x6000) == -1
    assert fwd(d(top=1)) == -1 and fwd(d(), ids=0x5000) == -1 and fwd(d(top=1), ids=0x5000) == -1
    assert fwd(d(), z=None) == -1 and fwd(d(), t=None) == -1 and fwd(d(), logp=None) == -1 and fwd(d(), lse=None) == -1
    assert fwd(d(), z=0x1001) == -3 and fwd(d(dt=1), z=0x1002) == -3 and fwd(d(), t=0x2004) == -3 and fwd(d(), ent=0x7002) == -3
    assert fwd(d(N=0), z=None, t=None, logp=None, lse=None) == 0

    def bwd(l, z=0x1000, t=0x2000, lse=0x3000, dl=0x4000, ent=None, dh=None, out=0x5000, cols=100, ldd=100):
        return L.qlora_token_logprobs_bwd(l, z, t, lse, dl, ent, dh, out, cols, ldd, None)
    assert bwd(d(), cols=99) == -1 and bwd(d(), ldd=99) == -1 and bwd(d(), dh=0x6000) == -1
    assert bwd(d(), t=None) == -1 and bwd(d(), dl=None) == -1 and bwd(d(), out=None) == -1 and bwd(d(), out=0x5001) == -3
    assert bwd(d(), out=0x1000, ldd=104) == -1                            # in place with other strides
    assert bwd(d(N=0), z=None, t=None, lse=None, dl=None, out=None) == 0


def test_logprobs_oracle():
    """The plain forward against torch's log_softmax in 64 bits, and the plain
    backward against its autograd."""
    z = torch.randn(5, 37, dtype=torch.float64, requires_grad=True)
    t = torch.tensor([3, 36, -100, 0, 37])
    ref = SO.token_logprobs(z.detach().numpy(), t.numpy(), top=4)
    q = torch.log_softmax(z, 1)
    counts = (t >= 0) & (t < 37)
    logp = torch.where(counts, q.gather(1, t.clamp(0, 36)[:, None])[:, 0], 0.0)
    ent = -(q.exp() * q).sum(1)
    assert np.allclose(ref["logp"], logp.detach().numpy(), atol=1e-12) and np.allclose(ref["entropy"], ent.detach().numpy(), atol=1e-12)
    assert np.array_equal(ref["top_ids"], torch.topk(z, 4, 1).indices.numpy())
    a, b = torch.randn(5, dtype=torch.float64), torch.randn(5, dtype=torch.float64)
    ((logp * a).sum() + (ent * b).sum()).backward()
    got = SO.token_logprobs_backward(z.detach().numpy(), t.numpy(), ref["lse"], a.numpy(), ref["entropy"], b.numpy())
    assert np.allclose(got, z.grad.numpy(), atol=1e-12)


@pytest.mark.parametrize("top", [-1, 33, (1 << 32) + 2])
def test_number_of_alternatives_outside_its_range(top):
    """Refused before anything is allocated for them or their number is cut to 32 bits."""
    with pytest.raises(ValueError, match="expected 0 to 32"):
        Q.qlora_token_logprobs_fwd(torch.zeros(4, 64, dtype=BF16), torch.zeros(4, dtype=torch.int64), top=top)


def test_norm_backward_without_its_input():
    """What a forward pass in place returns for S when it had no residual."""
    X, w, s = torch.zeros(4, 64, dtype=BF16), torch.ones(64), torch.zeros(4)
    with pytest.raises(ValueError, match="S is required"):
        Q.qlora_layer_norm_bwd(X, None, w, s, s)
