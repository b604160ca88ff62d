"""Workloads of the fine-tuning step's operators around the QLoRA linear layer.

Three families: layer norm (forward and backward), the log probabilities of
given tokens (forward with entropy and top alternatives, and backward) and one
AdamW step over all adapter tensors.  A case is a dict of plain values;
``prepare`` makes its inputs from a seed, ``run`` computes one pass in plain
torch operations (``own`` false) or with the library's entry points (``own``
true), ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
BLOCK = 256                      # elements that share one scale of an 8-bit state
BETA1, BETA2, EPS, LR, DECAY = 0.9, 0.999, 1e-8, 2e-4, 0.01
NORM_EPS = 1e-5
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # residual add and rms norm in front of the projections, 65B-style block, one training batch
        {"name": "norm_fwd_block", "op": "norm_fwd", "rows": 8192, "dim": 8192, "type": "bf16", "weight": "f32",
         "rms": True, "bias": False, "residual": True},
        # its backward pass, with the gradient that arrives along the residual stream
        {"name": "norm_bwd_block", "op": "norm_bwd", "rows": 8192, "dim": 8192, "type": "bf16", "weight": "f32",
         "rms": True, "bias": False, "residual": True},
        # one token while decoding: latency
        {"name": "norm_fwd_token", "op": "norm_fwd", "rows": 1, "dim": 8192, "type": "bf16", "weight": "bf16",
         "rms": False, "bias": True, "residual": True},
        # layer norm with bias in fp32, odd sizes
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "rows": 2047, "dim": 4099, "type": "f32", "weight": "f32",
         "rms": False, "bias": True, "residual": False},
        # loss of a training batch: 4 sequences of 1024 tokens, with the entropy
        {"name": "logp_fwd_train", "op": "logp_fwd", "rows": 4096, "vocab": 32000, "pad": 0, "type": "bf16",
         "top": 0, "entropy": True, "masked": False},
        # the gradient of that loss
        {"name": "logp_bwd_train", "op": "logp_bwd", "rows": 4096, "vocab": 32000, "pad": 0, "type": "bf16",
         "top": 0, "entropy": False, "masked": False},
        # one sampled token with its alternatives, large vocabulary: latency
        {"name": "logp_fwd_token_top", "op": "logp_fwd", "rows": 1, "vocab": 131072, "pad": 0, "type": "bf16",
         "top": 8, "entropy": True, "masked": False},
        # a scoring batch with alternatives, odd vocabulary in padded rows, part of it masked out
        {"name": "logp_fwd_odd_top", "op": "logp_fwd", "rows": 333, "vocab": 50001, "pad": 7, "type": "f32",
         "top": 20, "entropy": True, "masked": True},
        # the adapters of one small layer (rank 8): latency
        {"name": "adamw32_small", "op": "adamw", "layers": 1, "hidden": 4096, "ffn": 11008, "rank": 8, "bits": 32,
         "param": "bf16", "grad": "f32", "clip": False},
        # the adapters of a 32-layer model of the 7B-style projection set (448 tensors), fp32 masters with bf16 copies
        {"name": "adamw32_model", "op": "adamw", "layers": 32, "hidden": 4096, "ffn": 11008, "rank": 16, "bits": 32,
         "param": "master", "grad": "f32", "clip": True},
        # 8-bit states: twelve 65B-style blocks at rank 64, fp32 gradients as the linear layer writes them
        {"name": "adamw8_blocks", "op": "adamw", "layers": 12, "hidden": 8192, "ffn": 28672, "rank": 64, "bits": 8,
         "param": "bf16", "grad": "f32", "clip": True},
        # odd tensors, none of them a whole number of blocks, bf16 gradients
        {"name": "adamw8_odd", "op": "adamw", "layers": 6, "hidden": 1001, "ffn": 2711, "rank": 13, "bits": 8,
         "param": "master", "grad": "bf16", "clip": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "logp_fwd", "logp_bwd", "adamw"])
    if op.startswith("norm"):
        dim = _log(rng, 64, 16384)
        if rng.random() < 0.6:
            dim = -(-dim // 8) * 8
        rows = min(_log(rng, 1, 8192), 8192 * 8192 // dim)
        kind = rng.choice(["bf16", "bf16", "f32"])
        if kind == "f32":
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "dim": dim, "type": kind,
                "weight": rng.choice(["bf16", "f32"]) if kind == "bf16" else "f32", "rms": rng.random() < 0.5,
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}
    if op.startswith("logp"):
        vocab = _log(rng, 1000, 131072)
        if rng.random() < 0.5:
            vocab = -(-vocab // 8) * 8
        rows = min(_log(rng, 1, 4096), 4096 * 32000 // (vocab + 8))
        kind = rng.choice(["bf16", "bf16", "f32"])
        if kind == "f32":
            rows = max(1, rows // 2)
        return {"op": op, "rows": rows, "vocab": vocab, "pad": rng.choice([0, 0, -vocab % 8, 5]), "type": kind,
                "top": rng.choice([0, 1, 5, 8, 20, 32]) if op == "logp_fwd" else 0, "entropy": rng.random() < 0.6,
                "masked": rng.random() < 0.3}
    hidden, ffn, rank = _log(rng, 64, 8192), _log(rng, 128, 28672), _log(rng, 1, 64)
    most = 12 * 64 * (11 * 8192 + 3 * 28672)
    layers = max(1, min(_log(rng, 1, 64), most // (rank * (11 * hidden + 3 * ffn))))
    return {"op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "rank": rank, "bits": rng.choice([8, 8, 32]),
            "param": rng.choice(["bf16", "f32", "master"]), "grad": rng.choice(["f32", "f32", "bf16"]),
            "clip": rng.random() < 0.5}


def _adapter_shapes(case):
    """The A and B of every adapted projection: q, k, v, o, gate, up, down."""
    h, f, r = case["hidden"], case["ffn"], case["rank"]
    one = []
    for d, k in [(h, h)] * 4 + [(f, h)] * 2 + [(h, f)]:
        one += [(r, k), (d, r)]
    return one * case["layers"]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)

    s = {"case": case, "op": case["op"]}
    if own:
        import bit_quantized_lora_02_b200 as Q
        s["Q"] = Q
    if case["op"].startswith("norm"):
        t, wt = DTYPE[case["type"]], DTYPE[case["weight"]]
        M, D = case["rows"], case["dim"]
        scale = 1.0 + 4.0 * (torch.rand(D, generator=g, device=DEV) < 0.01)      # a few loud channels
        s["X"] = (normal(M, D) * scale + 0.3).to(t)
        s["weight"] = (1.0 + 0.1 * normal(D)).to(wt)
        s["bias"] = (0.1 * normal(D)).to(wt) if case["bias"] else None
        extra = normal(M, D).to(t) if case["residual"] else None
        if case["op"] == "norm_fwd":
            s["residual"] = extra
        else:
            s["dS"] = extra
            s["dY"] = normal(M, D).to(t)
            x = s["X"].float()
            mean = torch.zeros(M, device=DEV) if case["rms"] else x.mean(1)
            s["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + NORM_EPS)
            s["mean"] = None if case["rms"] else mean
    elif case["op"].startswith("logp"):
        t = DTYPE[case["type"]]
        N, V, ld = case["rows"], case["vocab"], case["vocab"] + case["pad"]
        z = 3.0 * normal(N, ld)
        targets = torch.randint(0, V, (N,), generator=g, device=DEV)
        z[torch.arange(N, device=DEV), targets] += 6.0 * torch.rand(N, generator=g, device=DEV)
        if case["masked"]:                                                       # tokens that a grammar rules out
            out = torch.rand(ld, generator=g, device=DEV) < 0.5
            z.masked_fill_(out[None, :], -math.inf)
        skip = torch.rand(N, generator=g, device=DEV) < 0.05                     # prompt positions: no loss
        s["logits"] = z.to(t)
        s["targets"] = torch.where(skip, torch.full_like(targets, -100), targets)
        if case["op"] == "logp_bwd":
            x = s["logits"][:, :V].float()
            m = x.amax(1, keepdim=True)
            e = torch.exp(x - m)
            total = e.sum(1)
            s["lse"] = m[:, 0] + torch.log(total)
            gap = torch.where(e > 0, m - x, 0.0)
            s["ent"] = torch.log(total) + (e * gap).sum(1) / total
            s["dlogp"] = -torch.rand(N, generator=g, device=DEV) / N
            s["dent"] = 0.01 * normal(N) / N if case["entropy"] else None
    else:
        shapes = _adapter_shapes(case)
        sizes = [a * b for a, b in shapes]
        starts, at = [], 0
        for n in sizes:
            starts.append(at)
            at += -(-n // BLOCK) * BLOCK
        s["grad"] = torch.zeros(at, device=DEV, dtype=DTYPE[case["grad"]])
        noise = 1e-3 * normal(at) * torch.exp(0.7 * normal(at))                  # gradients of unlike sizes
        old_m, old_v = 0.2 * normal(at) * noise.abs(), (noise * (0.3 + torch.rand(at, generator=g, device=DEV))).square()
        value = 0.02 * normal(at)
        real = torch.zeros(at, dtype=torch.bool)
        for o, n in zip(starts, sizes):
            real[o:o + n] = True
        real = real.to(DEV)
        for x in (noise, old_m, old_v, value):
            x *= real
        s["grad"].copy_(noise)
        s["param"] = value.to(torch.bfloat16) if case["param"] == "bf16" else value
        s["copy"] = value.to(torch.bfloat16) if case["param"] == "master" else None
        s["scale"] = torch.full((1,), 0.37, device=DEV) if case["clip"] else None
        s["step"] = 20
        if case["bits"] == 32:
            s["state"] = [old_m, old_v]
        else:
            s["state"] = list(_encode_m(old_m) + _encode_v(old_v))
        if own:
            def views(x):
                return None if x is None else [x[o:o + n].view(sh) for o, n, sh in zip(starts, sizes, shapes)]
            opt = s["Q"].qlora_adamw_alloc(views(s["param"]), views(s["grad"]), state_bits=case["bits"],
                                           copies=views(s["copy"]))
            if case["bits"] == 32:
                opt.m.copy_(s["state"][0])
                opt.v.copy_(s["state"][1])
            else:
                for to, x in zip((opt.m, opt.m_scale, opt.v, opt.v_scale), s["state"]):
                    to.copy_(x)
            s["opt"], s["state"] = opt, None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _norm_fwd(s):
    c = s["case"]
    x = s["X"].float()
    if s["residual"] is not None:
        x = (x + s["residual"].float()).to(s["X"].dtype).float()
    mean = None if c["rms"] else x.mean(1)
    d = x if c["rms"] else x - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + NORM_EPS)
    y = d * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    S = x.to(s["X"].dtype) if s["residual"] is not None else None
    return {"Y": y.to(s["X"].dtype), "S": S, "mean": mean, "rstd": rstd}


def _norm_bwd(s):
    c = s["case"]
    x, dy, w = s["X"].float(), s["dY"].float(), s["weight"].float()
    rstd = s["rstd"][:, None]
    xh = (x if c["rms"] else x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if not c["rms"]:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if s["dS"] is not None:
        dx = dx + s["dS"].float()
    return {"dX": dx.to(s["X"].dtype), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0) if c["bias"] else None}


def _logp_fwd(s):
    c = s["case"]
    x = s["logits"][:, :c["vocab"]].float()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1)
    lse = m[:, 0] + torch.log(total)
    t = s["targets"]
    counts = (t >= 0) & (t < c["vocab"])
    z = x.gather(1, torch.where(counts, t, 0)[:, None])[:, 0]
    out = {"logp": torch.where(counts, z - lse, 0.0), "lse": lse, "entropy": None, "top_ids": None, "top_logp": None}
    if c["entropy"]:
        gap = torch.where(e > 0, m - x, 0.0)
        out["entropy"] = torch.log(total) + (e * gap).sum(1) / total
    if c["top"]:
        val, idx = torch.sort(x + 0.0, dim=1, descending=True, stable=True)      # -0 + 0 = 0: equal values, lowest index first
        out["top_ids"] = idx[:, :c["top"]].to(torch.int32)
        out["top_logp"] = val[:, :c["top"]] - lse[:, None]
    return out


def _logp_bwd(s):
    c = s["case"]
    V = c["vocab"]
    logits = s["logits"]
    q = logits[:, :V].float() - s["lse"][:, None]
    p = torch.exp(q)
    t = s["targets"]
    counts = (t >= 0) & (t < V)
    dl = torch.where(counts, s["dlogp"], 0.0)[:, None]
    dz = -dl * p
    if s["dent"] is not None:
        dz = dz - s["dent"][:, None] * p * torch.where(p > 0, q + s["ent"][:, None], 0.0)
    dz.scatter_add_(1, torch.where(counts, t, 0)[:, None], dl)
    out = torch.zeros_like(logits)
    out[:, :V] = dz.to(logits.dtype)
    return {"dlogits": out}


def _encode_m(m):
    """E4M3 codes of each block of 256 against the block's largest magnitude."""
    b = m.view(-1, BLOCK)
    scale = b.abs().amax(1)
    scale = torch.where(scale < 2.0 ** -100, 0.0, scale)
    inv = torch.where(scale > 0, torch.full_like(scale, 448.0) / scale, 0.0)
    return (b * inv[:, None]).to(torch.float8_e4m3fn).view(-1), scale


def _encode_v(v):
    """8-bit codes of the fourth root of each block of 256, linear up to the block's largest."""
    b = v.view(-1, BLOCK)
    u = torch.sqrt(torch.sqrt(b))
    scale = u.amax(1)
    inv = torch.where(scale > 0, torch.full_like(scale, 255.0) / scale, 0.0)
    code = torch.round(u * inv[:, None])
    code = torch.where((b > 0) & (code == 0), 1.0, code)
    return code.to(torch.uint8).view(-1), scale


def _decode_m(code, scale):
    d = scale * torch.full_like(scale, 1.0 / 448.0)
    return (code.float().view(-1, BLOCK) * d[:, None]).view(-1)


def _decode_v(code, scale):
    d = scale * torch.full_like(scale, 1.0 / 255.0)
    u = code.float().view(-1, BLOCK) * d[:, None]
    u = u * u
    return (u * u).view(-1)


def _adamw(s):
    c = s["case"]
    s["step"] += 1
    bc1, bc2 = 1.0 - BETA1 ** s["step"], 1.0 - BETA2 ** s["step"]
    g = s["grad"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    state = s["state"]
    m, v = state if c["bits"] == 32 else (_decode_m(state[0], state[1]), _decode_v(state[2], state[3]))
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    p = s["param"].float()
    p = p * (1.0 - LR * DECAY) - (m * (LR / bc1)) / (torch.sqrt(v) * (1.0 / math.sqrt(bc2)) + EPS)
    s["param"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if c["bits"] == 32:
        s["state"] = [m, v]
    else:
        s["state"] = list(_encode_m(m) + _encode_v(v))
        m, v = _decode_m(*s["state"][:2]), _decode_v(*s["state"][2:])
    return {"param": s["param"], "copy": s["copy"], "m": m, "v": v}


def run(s):
    c = s["case"]
    if not own:
        return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "logp_fwd": _logp_fwd, "logp_bwd": _logp_bwd,
                "adamw": _adamw}[s["op"]](s)
    Q = s["Q"]
    if s["op"] == "norm_fwd":
        Y, S, mean, rstd = Q.qlora_layer_norm_fwd(s["X"], s["weight"], bias=s["bias"], residual=s["residual"],
                                                  eps=NORM_EPS, rms=c["rms"])
        return {"Y": Y, "S": S if s["residual"] is not None else None, "mean": mean, "rstd": rstd}
    if s["op"] == "norm_bwd":
        dX, dw, db = Q.qlora_layer_norm_bwd(s["dY"], s["X"], s["weight"], s["mean"], s["rstd"], dS=s["dS"],
                                            rms=c["rms"], need_dbias=c["bias"])
        return {"dX": dX, "dweight": dw, "dbias": db}
    if s["op"] == "logp_fwd":
        f = Q.qlora_token_logprobs_fwd(s["logits"], s["targets"], vocab=c["vocab"], top=c["top"],
                                       entropy=c["entropy"])
        return {"logp": f.logp, "lse": f.lse, "entropy": f.entropy, "top_ids": f.top_ids, "top_logp": f.top_logp}
    if s["op"] == "logp_bwd":
        d = Q.qlora_token_logprobs_bwd(s["logits"], s["targets"], s["lse"], s["dlogp"], entropy=s["ent"],
                                       dentropy=s["dent"], vocab=c["vocab"])
        return {"dlogits": d}
    s["step"] += 1
    Q.qlora_adamw_step(s["opt"], step=s["step"], lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY,
                       grad_scale=s["scale"])
    m, v = (s["opt"].m, s["opt"].v) if c["bits"] == 32 else Q.qlora_adamw_state(s["opt"])
    return {"param": s["param"], "copy": s["copy"], "m": m, "v": v}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"].startswith("norm"):
        M, D, e = case["rows"], case["dim"], SIZE[case["type"]]
        w = D * SIZE[case["weight"]]
        stats = 4 * M * (1 if case["rms"] else 2)
        if case["op"] == "norm_fwd":
            return {"bytes": M * D * e * (4 if case["residual"] else 2) + w * (2 if case["bias"] else 1) + stats,
                    "flops": 8 * M * D}
        return {"bytes": M * D * e * (4 if case["residual"] else 3) + w + 4 * D * (2 if case["bias"] else 1) + stats,
                "flops": 14 * M * D}
    if case["op"].startswith("logp"):
        N, V, e = case["rows"], case["vocab"], SIZE[case["type"]]
        if case["op"] == "logp_fwd":
            return {"bytes": N * V * e + N * (16 + (4 if case["entropy"] else 0)) + 8 * N * case["top"],
                    "flops": 6 * N * V}
        return {"bytes": N * V * e + N * (V + case["pad"]) * e + N * (16 + (8 if case["entropy"] else 0)),
                "flops": 5 * N * V}
    n = sum(a * b for a, b in _adapter_shapes(case))
    each = {"bf16": 4, "f32": 8, "master": 10}[case["param"]] + SIZE[case["grad"]]
    # 8-bit states: codes read and written, and the values they stand for written out
    each += 16 if case["bits"] == 32 else 4 + 16 / BLOCK + 8
    return {"bytes": n * each, "flops": 18 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _r32(x):
    """A value of the definition that is kept in 32 bits."""
    return x.to(torch.float32).to(torch.float64)


def _e4m3(y):
    """The E4M3 value next to y (ties to even, largest 448)."""
    a = y.abs()
    _, e = torch.frexp(torch.where(a > 0, a, 1.0))
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), y)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x = s["X"].double()
        if s["residual"] is not None:
            S = (x + s["residual"].double()).to(s["X"].dtype)
            x = S.double()
        D = case["dim"]
        mean = x.sum(1) / D if not case["rms"] else torch.zeros(case["rows"], dtype=torch.float64, device=DEV)
        x = x - mean[:, None]
        rstd = (x.pow(2).sum(1) / D + NORM_EPS).pow(-0.5)
        y = torch.einsum("md,m,d->md", x, rstd, s["weight"].double())
        if s["bias"] is not None:
            y += s["bias"].double()
        return {"Y": y, "S": S.double() if s["residual"] is not None else None,
                "mean": None if case["rms"] else mean, "rstd": rstd}
    if op == "norm_bwd":
        D = case["dim"]
        xh = s["X"].double()
        if not case["rms"]:
            xh = xh - s["mean"].double()[:, None]
        xh = xh * s["rstd"].double()[:, None]
        dy = s["dY"].double()
        dw = torch.einsum("md,md->d", dy, xh)
        db = dy.sum(0) if case["bias"] else None
        g = dy * s["weight"].double()
        along = torch.einsum("md,md->m", g, xh) / D
        g -= xh * along[:, None]
        if not case["rms"]:
            g -= (dy @ s["weight"].double() / D)[:, None]
        g *= s["rstd"].double()[:, None]
        if s["dS"] is not None:
            g += s["dS"].double()
        return {"dX": g, "dweight": dw, "dbias": db}
    if op.startswith("logp"):
        V = case["vocab"]
        x = s["logits"][:, :V].double()
        t = s["targets"]
        hot = t[:, None] == torch.arange(V, device=DEV)[None, :]
        counts = hot.any(1)
        if op == "logp_fwd":
            lse = torch.logsumexp(x, 1)
            logq = x - lse[:, None]
            logp = torch.where(hot, logq, 0.0).sum(1)
            ent = -torch.special.xlogy(logq.exp(), logq.exp()).sum(1) if case["entropy"] else None
            ids = best = None
            if case["top"]:
                # the k largest values, whichever of equal ones: only their values are needed here
                best = torch.topk(logq, case["top"], dim=1).values
            return {"logp": logp, "lse": lse, "entropy": ent, "top_ids": ids, "top_logp": best}
        logq = x - s["lse"].double()[:, None]
        p = logq.exp()
        dz = torch.where(counts, s["dlogp"].double(), 0.0)[:, None] * (hot.double() - p)
        if s["dent"] is not None:
            dz -= s["dent"].double()[:, None] * (torch.special.xlogy(p, p) + p * s["ent"].double()[:, None])
        return {"dlogits": torch.nn.functional.pad(dz, (0, case["pad"]))}
    step = s["step"] + 1
    g = s["grad"].double()
    if s["scale"] is not None:
        g = _r32(g * s["scale"].double())
    if case["bits"] == 32:
        m, v = (x.double() for x in s["state"])
    else:
        code, scale, vcode, vscale = s["state"]
        unit = _r32(scale.double() * float(torch.tensor(1.0 / 448.0)))
        m = _r32(code.float().double().view(-1, BLOCK) * unit[:, None]).view(-1)
        unit = _r32(vscale.double() * float(torch.tensor(1.0 / 255.0)))
        root = _r32(vcode.double().view(-1, BLOCK) * unit[:, None])
        v = _r32(_r32(root ** 2) ** 2).view(-1)
    p = s["param"].double()
    new_m, new_v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g * g
    p = (1 - LR * DECAY) * p - LR * (new_m / (1 - BETA1 ** step)) / ((new_v / (1 - BETA2 ** step)).sqrt() + EPS)
    if case["bits"] == 8:
        # the stored states are defined by 32-bit steps: each product and sum rounded on its own
        def f(x):
            return float(torch.tensor(x, dtype=torch.float32))
        m = _r32(_r32(m * f(BETA1)) + _r32(g * f(1 - BETA1))).view(-1, BLOCK)
        v = _r32(_r32(v * f(BETA2)) + _r32(_r32(g * g) * f(1 - BETA2))).view(-1, BLOCK)
        top = m.abs().amax(1)
        top = torch.where(top < 2.0 ** -100, 0.0, top)
        per = torch.where(top > 0, _r32(448.0 / top.clamp(min=2.0 ** -100)), 0.0)
        new_m = _r32(_e4m3(_r32(m * per[:, None])) * _r32(top * f(1.0 / 448.0))[:, None]).view(-1)
        root = _r32(_r32(v.sqrt()).sqrt())
        top = root.amax(1)
        per = torch.where(top > 0, _r32(255.0 / top.clamp(min=1e-30)), 0.0)
        code = torch.round(_r32(root * per[:, None]))
        code = torch.where(v > 0, code.clamp(min=1.0), code)
        root = _r32(code * _r32(top * f(1.0 / 255.0))[:, None])
        new_v = _r32(_r32(root ** 2) ** 2).view(-1)
    return {"param": p, "copy": p if s["copy"] is not None else None, "m": new_m, "v": new_v}
