"""Plain 64-bit forms of the operators around the linear layer in a fine-tuning
step (numpy only; test infrastructure, shares no code with the kernels)."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def norm_forward(S, w, b, eps, rms):
    """(Y, mean, rstd) of the rows of S (already X + R)."""
    S = np.asarray(S, np.float64)
    mean = np.zeros(S.shape[0]) if rms else S.mean(axis=1)
    d = S - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    Y = d * rstd[:, None] * np.asarray(w, np.float64)
    if b is not None:
        Y = Y + np.asarray(b, np.float64)
    return Y, mean, rstd


def norm_backward(dY, S, w, mean, rstd, dS, rms):
    """(dX, dw, db); mean and rstd are the forward's."""
    dY, S, w = (np.asarray(x, np.float64) for x in (dY, S, w))
    rstd = np.asarray(rstd, np.float64)[:, None]
    xh = (S - (0.0 if rms else np.asarray(mean, np.float64)[:, None])) * rstd
    g = dY * w
    dX = g - xh * (g * xh).mean(axis=1, keepdims=True)
    if not rms:
        dX = dX - g.mean(axis=1, keepdims=True)
    dX = dX * rstd
    if dS is not None:
        dX = dX + np.asarray(dS, np.float64)
    return dX, (dY * xh).sum(axis=0), dY.sum(axis=0)


# ---------------------------------------------------------------------------
# log probabilities of given tokens
# ---------------------------------------------------------------------------
def token_logprobs(z, targets, top=0):
    """dict of logp, lse, entropy, top_ids, top_logp for logits z (N x V).  A
    target outside [0, V) gives logp 0.  A row of -inf only: lse and logp -inf,
    entropy 0."""
    z = np.asarray(z, np.float64)
    N, V = z.shape
    out = {"logp": np.zeros(N), "lse": np.zeros(N), "entropy": np.zeros(N)}
    for i in range(N):
        m = z[i].max()
        if m == -np.inf:
            out["lse"][i] = -np.inf
        else:
            e = np.exp(z[i] - m)
            s = e.sum()
            out["lse"][i] = m + np.log(s)
            live = e > 0
            out["entropy"][i] = np.log(s) + (e[live] * (m - z[i][live])).sum() / s
        t = int(targets[i])
        if 0 <= t < V:
            # from the maximum, not from lse: beside logits of 1e38 log s would vanish in it
            out["logp"][i] = -np.inf if m == -np.inf else (z[i, t] - m) - np.log(s)
    if top:
        ids = np.argsort(-(z + 0.0), axis=1, kind="stable")[:, :top]
        out["top_ids"] = ids.astype(np.int32)
        best = np.take_along_axis(z, ids, 1)
        m = z.max(axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            ls = np.log(np.exp(z - m).sum(axis=1, keepdims=True))
            out["top_logp"] = np.where(best == -np.inf, -np.inf, (best - m) - ls)
    return out


def token_logprobs_backward(z, targets, lse, dlogp, entropy=None, dentropy=None):
    z = np.asarray(z, np.float64)
    N, V = z.shape
    dz = np.zeros((N, V))
    for i in range(N):
        if lse[i] == -np.inf:
            continue
        q = z[i] - float(lse[i])
        p = np.exp(q)
        t = int(targets[i])
        if 0 <= t < V:
            dz[i] -= float(dlogp[i]) * p
            dz[i, t] += float(dlogp[i])
        if dentropy is not None:
            live = p > 0
            dz[i][live] -= float(dentropy[i]) * p[live] * (q[live] + float(entropy[i]))
    return dz


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
BLOCK = 256
_f = np.float32


def e4m3_values():
    """The 256 E4M3 values by code (NaN at 0x7F and 0xFF)."""
    out = np.zeros(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 127) == 127 else (-v if c & 128 else v)
    return out


_E4M3 = e4m3_values()
_E4M3_POS = _E4M3[:127]


def e4m3_code(y):
    """Nearest E4M3 code of fp32 values |y| <= 448 (1 + 2^-22), ties to the even code."""
    a = np.abs(np.asarray(y, np.float64))
    hi = np.clip(np.searchsorted(_E4M3_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _E4M3_POS[lo], _E4M3_POS[hi] - a
    c = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (c + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def adamw_encode(m, v):
    """8-bit states of fp32 moments of one tensor: per block of 256 (the last may
    be short) m as E4M3 codes of m * 448 / s_m with s_m the largest |m| (blocks
    below 2^-100 store zeros), v as round(u * 255 / s_u) of its fourth root u,
    at least 1 where v > 0.  All arithmetic in fp32, each step rounded."""
    n = m.size
    nb = -(-n // BLOCK)
    mc, vc = np.zeros(n, np.uint8), np.zeros(n, np.uint8)
    ms, vs = np.zeros(nb, _f), np.zeros(nb, _f)
    for j in range(nb):
        sl = slice(j * BLOCK, min(n, (j + 1) * BLOCK))
        x = m[sl].astype(_f)
        s = np.abs(x).max()
        s = _f(0) if s < _f(2.0 ** -100) else s
        inv = _f(448) / s if s > 0 else _f(0)
        mc[sl], ms[j] = e4m3_code(x * inv), s
        u = np.sqrt(np.sqrt(v[sl].astype(_f)))
        s = u.max()
        inv = _f(255) / s if s > 0 else _f(0)
        c = np.rint(u * inv)
        vc[sl], vs[j] = np.where((v[sl] > 0) & (c == 0), 1, c).astype(np.uint8), s
    return mc, ms, vc, vs


def adamw_decode(mc, ms, vc, vs):
    j = np.arange(mc.size) // BLOCK
    m = _E4M3[mc].astype(_f) * (ms * (_f(1) / _f(448)))[j]
    t = vc.astype(_f) * (vs * (_f(1) / _f(255)))[j]
    t = t * t
    return m, t * t


LIMIT = 2.0 ** 60       # of a gradient's magnitude: its square stays finite in fp32


def adamw_hold(g, limit=LIMIT):
    """g held to +-limit; NaN where it is not finite."""
    with np.errstate(invalid="ignore"):
        return (g if limit is None else np.clip(g, -limit, limit)) + g * g.dtype.type(0)


def adamw_moments(m, v, g, beta1, beta2, scale=None):
    """fp32 moments after one step, every product and sum rounded (the values an
    8-bit state encodes)."""
    g = g.astype(_f)
    if scale is not None:
        g = g * _f(scale)
    g = adamw_hold(g)
    return (m * _f(beta1) + g * _f(1.0 - beta1)), (v * _f(beta2) + (g * g) * _f(1.0 - beta2))


def adamw_param(p, m, v, g, step, lr, beta1, beta2, eps, wd, scale=None, limit=LIMIT):
    """The parameter after one step in 64 bits from the old moments m, v (limit
    None: from the gradient as it is)."""
    p, m, v, g = (np.asarray(x, np.float64) for x in (p, m, v, g))
    if scale is not None:
        g = (g.astype(_f) * _f(scale)).astype(np.float64)
    g = adamw_hold(g, limit)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p * (1 - lr * wd) - lr * mh / (np.sqrt(vh) + eps), m, v
