"""Log probabilities of given tokens, entropies, top alternatives and the
gradient of the logits against a plain 64-bit form.

Tolerances, u = 2^-24 (half a step of fp32).  Every exponential has the relative
error of its argument's rounding, u |z - m| <= 104 u (beyond that it is 0), of
its product with log2 e (the same again) and of the hardware's function, 2^-22;
S adds at most (number of additions on one path) < 600 u: 1024 u = 2^-14 of S
is far above all of it, but the terms that make up S have |z - m| of a few, so
64 u is what is asked for where |z - m| <= 30, as in these inputs.  lse then is
off by 64 u plus its own rounding (2 u of its size), logp by 64 u + 2 u (|z_t| +
|lse|), the entropy by 64 u (1 + H) each for S and G.  A gradient takes p with
its relative error (64 u, and lse's 2 u |lse| as a factor) and, in bf16, half a
step: 2^-8."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as SO

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_quantized_lora_02_b200 as Q

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def make(N, V, dtype, seed, pad=0, std=3.0):
    g = torch.Generator().manual_seed(seed)
    z = std * torch.randn(N, V + pad, generator=g)
    t = torch.randint(0, V, (N,), generator=g)
    if N > 2:
        t[N // 2] = -100
        t[1] = V                       # just outside
    return z.to(dtype).cuda(), t.cuda()


def check_forward(z, t, V, f, top=0, entropy=True):
    zz = z[:, :V].double().cpu().numpy()
    ref = SO.token_logprobs(zz, t.cpu().numpy(), top)
    size = np.abs(np.where(np.isfinite(ref["lse"]), ref["lse"], 0))

    def near(got, want, tol):
        got, want = got.double().cpu().numpy(), np.asarray(want)
        fin = np.isfinite(want)
        assert np.array_equal(got[~fin], want[~fin])
        assert np.all(np.abs(got[fin] - want[fin]) <= (tol[fin] if isinstance(tol, np.ndarray) else tol))
    near(f.lse, ref["lse"], 64 * U + 2 * U * size)
    near(f.logp, ref["logp"], 64 * U + 2 * U * (2 * size + np.abs(np.where(np.isfinite(ref["logp"]), ref["logp"], 0))))
    if entropy:
        near(f.entropy, ref["entropy"], 64 * U * (2 + ref["entropy"]))
    if top:
        assert np.array_equal(f.top_ids.cpu().numpy(), ref["top_ids"])
        w = ref["top_logp"]
        near(f.top_logp, w, 64 * U + 4 * U * (size[:, None] + np.abs(np.where(np.isfinite(w), w, 0))))
    return ref


def check_backward(z, t, V, f, dlogp, dent, dz):
    zz = z[:, :V].double().cpu().numpy()
    lse, ent = f.lse.cpu().numpy(), None if f.entropy is None else f.entropy.cpu().numpy()
    dl, dh = dlogp.cpu().numpy(), None if dent is None else dent.cpu().numpy()
    tt = t.cpu().numpy()
    ref = SO.token_logprobs_backward(zz, tt, lse, dl, ent, dh)
    got = dz.double().cpu().numpy()
    assert not got[:, V:].any()
    with np.errstate(invalid="ignore"):
        q = np.where(np.isfinite(lse)[:, None], zz - lse[:, None].astype(np.float64), -INF)
    p = np.exp(q)
    weight = np.where((tt >= 0) & (tt < V), np.abs(dl), 0)[:, None] * np.ones_like(p)
    if dh is not None:
        weight = weight + np.abs(dh)[:, None] * (np.abs(np.where(p > 0, q, 0)) + ent[:, None])
    rel = 64 * U + 4 * U * np.abs(np.where(np.isfinite(lse), lse, 0))[:, None] + 4 * U * np.abs(np.where(p > 0, q, 0))
    tol = rel * p * weight + 4 * U * np.abs(ref) + 1e-38
    if dz.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(ref) * 1.01
    assert np.all(np.abs(got[:, :V] - ref) <= tol)


SIZES = [(1, 1, 0), (3, 2, 0), (5, 7, 1), (4, 33, 0), (9, 255, 0), (300, 1000, 0), (7, 2048, 8), (5, 2049, 3), (65, 4097, 0),
         (3, 16384, 0), (2, 16391, 5), (200, 32000, 0), (1, 50001, 7), (33, 50001, 7), (1, 65536, 0), (1, 131072, 0),
         (9, 131071, 2), (40, 20000, 0), (400, 17000, 1), (1300, 1003, 2), (1500, 8100, 0)]


@pytest.mark.parametrize("N,V,pad", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F32] if torch.cuda.is_available() else [])
def test_forward_and_backward(N, V, pad, dtype):
    z, t = make(N, V, dtype, N + V, pad)
    top = min(V, 20)
    f = Q.qlora_token_logprobs_fwd(z, t, vocab=V, top=top, entropy=True)
    check_forward(z, t, V, f, top)
    plain = Q.qlora_token_logprobs_fwd(z, t, vocab=V)
    check_forward(z, t, V, plain, entropy=False)
    assert plain.entropy is None and plain.top_ids is None
    g = torch.Generator().manual_seed(1)
    dlogp, dent = torch.randn(N, generator=g).cuda(), torch.randn(N, generator=g).cuda()
    check_backward(z, t, V, f, dlogp, dent, Q.qlora_token_logprobs_bwd(z, t, f.lse, dlogp, entropy=f.entropy,
                                                                       dentropy=dent, vocab=V))
    check_backward(z, t, V, plain, dlogp, None, Q.qlora_token_logprobs_bwd(z, t, plain.lse, dlogp, vocab=V))


@pytest.mark.parametrize("top", [1, 2, 31, 32])
@pytest.mark.parametrize("V", [32, 33, 1000, 40000, 131072])
def test_top_with_many_equal_logits(top, V):
    """Few distinct values: equal logits come by ascending index, through the list
    that overflows and the bound that is raised."""
    g = torch.Generator().manual_seed(top + V)
    rows = [torch.zeros(V), torch.randint(0, 3, (V,), generator=g).float(), torch.randint(0, 60, (V,), generator=g) / 8.0,
            torch.arange(V).float() / 64, -torch.arange(V).float() / 64, torch.full((V,), -INF), torch.full((V,), -3.38e38),
            torch.where(torch.rand(V, generator=g) < 0.5, 0.0, -0.0)]
    few = torch.full((V,), -INF)
    few[[V - 1, V // 2, 3]] = torch.tensor([1.0, 2.0, 2.0])
    low = torch.full((V,), torch.finfo(BF16).min)
    low[[V - 1, V // 3]] = 5.0
    late = torch.zeros(V)
    late[V - 20:] = torch.arange(20).float()
    z = torch.stack(rows + [few, low, late])
    for dtype in (BF16, F32):
        x = z.to(dtype).cuda()
        t = torch.full((x.shape[0],), V - 1).cuda()
        for part in (x, x[:1], x[5:6], x[8:9], x[10:11]):         # few rows are split over clusters
            f = Q.qlora_token_logprobs_fwd(part, t[:part.shape[0]], top=top, entropy=True)
            # ids against a stable sort of the same logits in fp32
            want = torch.sort(part.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
            assert torch.equal(f.top_ids.long(), want)


@pytest.mark.parametrize("low", [-INF, -1e9, "min"])
@pytest.mark.parametrize("N,V", [(1, 131072), (3, 50001), (300, 9000), (1300, 4096), (700, 1100), (40, 200)])
def test_top_under_a_mask(N, V, low):
    """Rows with 0, 1, 5 or half of their logits outside a mask, some rows without
    one: the top logits, then masked ones by index."""
    g = torch.Generator().manual_seed(V)
    for dtype in (BF16, F32):
        z = (3 * torch.randn(N, V, generator=g)).to(dtype)
        fill = torch.finfo(dtype).min if low == "min" else low
        for r in range(N):
            left = (5, 1, V // 2, 0, V)[r % 5]
            if r % 10 == 7:
                z[r, V // 2:] = fill
            elif left < V:
                keep = torch.randperm(V, generator=g)[:left]
                row = torch.full((V,), fill, dtype=dtype)
                row[keep] = z[r, keep]
                z[r] = row
        x = z.cuda()
        f = Q.qlora_token_logprobs_fwd(x, top=20, entropy=True)
        want = torch.sort(x.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :20]
        assert torch.equal(f.top_ids.long(), want)


def test_rows_that_a_mask_leaves_empty_and_single_survivors():
    V = 5000
    z = torch.full((4, V), -INF)
    z[1, 77] = 3.0
    z[2] = torch.finfo(F32).min
    z[3, 4999] = -1e4
    t = torch.tensor([5, 77, 1, 10])
    for dtype in (F32, BF16):
        x = z.to(dtype).cuda()
        if dtype == BF16:
            x[2] = torch.finfo(BF16).min
        f = Q.qlora_token_logprobs_fwd(x, t.cuda(), top=2, entropy=True)
        assert f.lse[0] == -INF and f.logp[0] == -INF and f.entropy[0] == 0
        assert f.logp[1] == 0 and f.entropy[1] == 0 and f.top_ids[1, 0] == 77 and f.top_logp[1].tolist() == [0.0, -INF]
        assert abs(f.logp[2].item() + np.log(V)) <= 64 * U + 2 * U * 10 and abs(f.entropy[2].item() - np.log(V)) <= 64 * U * 11
        assert f.logp[3] == -INF and f.entropy[3] == 0 and f.top_ids[:, 0].tolist() == [0, 77, 0, 4999]
        d = Q.qlora_token_logprobs_bwd(x, t.cuda(), f.lse, torch.ones(4).cuda(), entropy=f.entropy,
                                       dentropy=torch.ones(4).cuda())
        assert d.isfinite().all() and not d[0].any() and not d[1].any()
        assert d[3, 10] == 1 and d[3, 4999] == -1


@pytest.mark.parametrize("dtype", [BF16, F32] if torch.cuda.is_available() else [])
@pytest.mark.parametrize("V", [700, 9001, 70000])
def test_logits_of_any_size(dtype, V):
    """Rows around 1e38 and the type's largest and lowest values, beside ordinary
    ones, with and without the entropy."""
    g = torch.Generator().manual_seed(V)
    z = torch.randn(10, V, generator=g)
    big = torch.finfo(dtype).max
    z[0] *= 1e38
    z[1] = -1e38
    z[2] = -9.9e37
    z[3] = -2.5e38
    z[3, 5] = -2.4e38
    z[4, 7] = big
    z[5] = -big
    z[6] = big
    z[7, :] = -INF
    z[7, V - 1] = -big
    z[8] = -big
    z[8, 3] = -1.0
    z[9] = z[9] * 100 - 1e9
    x = z.to(dtype).cuda()
    t = torch.tensor([0, 1, 2, 5, 7, 9, V - 1, V - 1, 3, 4]).cuda()
    for part in (x, x[5:6], x[6:7], x[2:3]) + ((x.repeat(130, 1),) if V == 700 else ()):   # 1300 rows: a warp to each
        tt = t[:part.shape[0]] if part.shape[0] <= 10 else t.repeat(130)
        for ent in (False, True):
            f = Q.qlora_token_logprobs_fwd(part, tt, top=3, entropy=ent)
            # a draw beyond 3.4 times 1e38 is infinite: its row is NaN throughout
            odd = (part == INF).any(1)
            keep = (~odd).cpu().numpy()
            assert f.lse[odd].isnan().all() and f.logp[odd].isnan().all()
            zz = part.double().cpu().numpy()[keep]
            ref = SO.token_logprobs(zz, tt.cpu().numpy()[keep], 3)
            assert np.array_equal(f.top_ids.cpu().numpy()[keep], ref["top_ids"])
            lse = f.lse.double().cpu().numpy()[keep]
            assert np.all(np.abs(lse - ref["lse"]) <= 4 * U * np.abs(ref["lse"]) + 64 * U)
            got = f.logp.double().cpu().numpy()[keep]
            # two logits 3.6e38 apart: their difference is -infinity in fp32
            want = np.where(ref["logp"] < -3.4028235e38, -INF, ref["logp"])
            assert np.array_equal(np.isinf(got), np.isinf(want))
            got, want = (np.where(np.isinf(x), 0, x) for x in (got, want))
            assert np.all(np.abs(got - want) <= 64 * U + 4 * U * (np.abs(want) + 20))
            if ent:
                assert np.all(np.abs(f.entropy.double().cpu().numpy()[keep] - ref["entropy"]) <= 64 * U * (2 + ref["entropy"]))
            dl = torch.ones(part.shape[0]).cuda()
            for place in (None, part.clone()):
                src = part if place is None else place
                d = Q.qlora_token_logprobs_bwd(src, tt, f.lse, dl, entropy=f.entropy, dentropy=dl if ent else None,
                                               dlogits=place)[~odd]
                assert d.isfinite().all()
                # every row's gradient sums to 0 but for the roundings of its entries
                assert np.all(np.abs(d.double().sum(1).cpu().numpy()) <= 2 * (half(dtype) + 64 * U) * (3 + np.log(V)))


def half(dtype):
    return torch.finfo(dtype).eps / 2


@pytest.mark.parametrize("V", [1000, 40000])
def test_non_finite_logits_stay_in_their_row(V):
    z, t = make(6, V, F32, 3)
    clean = Q.qlora_token_logprobs_fwd(z, t, top=4, entropy=True)
    z[2, V // 2] = float("nan")
    z[4, 1] = INF
    f = Q.qlora_token_logprobs_fwd(z, t, top=4, entropy=True)
    for name in ("logp", "lse", "entropy", "top_ids", "top_logp"):
        a, b = getattr(f, name), getattr(clean, name)
        for i in (0, 1, 3, 5):
            assert torch.equal(a[i], b[i])
    t[2] = t[4] = 0
    f = Q.qlora_token_logprobs_fwd(z, t, top=4, entropy=True)
    assert f.logp[[2, 4]].isnan().all() and f.lse[[2, 4]].isnan().all() and f.entropy[[2, 4]].isnan().all()
    assert ((f.top_ids >= 0) & (f.top_ids < V)).all()


@pytest.mark.parametrize("dtype", [BF16, F32] if torch.cuda.is_available() else [])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_strided_rows_any_alignment_and_nothing_outside(dtype, shift):
    N, V, ld = 6, 4001, 4100
    g = torch.Generator().manual_seed(7)
    buf = (3 * torch.randn(N * ld + 64, generator=g)).to(dtype).cuda()
    z = buf[shift:shift + N * ld].view(N, ld)[:, 5:5 + V + 3]
    t = torch.randint(0, V, (N,), generator=g).cuda()
    f = Q.qlora_token_logprobs_fwd(z, t, vocab=V, top=5, entropy=True)
    check_forward(z, t, V, f, 5)
    dl = torch.randn(N, generator=g).cuda()
    want = Q.qlora_token_logprobs_bwd(z, t, f.lse, dl, vocab=V)
    check_backward(z, t, V, f, dl, None, want)
    out = torch.full((N * 4500 + 64,), 9.0, dtype=dtype, device="cuda")
    dz = out[2:2 + N * 4500].view(N, 4500)[:, 3:3 + V + 3]
    Q.qlora_token_logprobs_bwd(z, t, f.lse, dl, vocab=V, dlogits=dz)
    assert torch.equal(dz, want)
    dz.fill_(9.0)
    assert (out == 9).all()
    # in place: only the rows' own columns change
    before = buf.clone()
    got = Q.qlora_token_logprobs_bwd(z, t, f.lse, dl, vocab=V, dlogits=z)
    assert got is z and torch.equal(z, want)
    z.copy_(before[shift:shift + N * ld].view(N, ld)[:, 5:5 + V + 3])
    assert torch.equal(buf, before)


def test_no_rows_and_no_targets():
    z = torch.empty(0, 100, dtype=BF16, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    f = Q.qlora_token_logprobs_fwd(z, t, top=3, entropy=True)
    assert f.logp.shape == (0,) and f.top_ids.shape == (0, 3)
    assert Q.qlora_token_logprobs_bwd(z, t, f.lse, f.logp).shape == (0, 100)
    z, t = make(4, 3001, BF16, 5)
    f, g = Q.qlora_token_logprobs_fwd(z, t, top=3), Q.qlora_token_logprobs_fwd(z, top=3)
    assert g.logp is None and torch.equal(f.lse, g.lse) and torch.equal(f.top_ids, g.top_ids)


def test_gradient_against_differences():
    """Central differences of a weighted sum of logp and entropy: with h = 2^-5 the
    truncation is h^2 / 6 of third derivatives below 2, 4e-4, and the rounding 64 u
    (2 + H) |weights| / h < 2e-3."""
    V, h = 12, 2.0 ** -5
    z, t = make(3, V, F32, 2, std=1.0)
    t = torch.tensor([3, 0, 11]).cuda()
    wl, wh = torch.tensor([1.0, -0.5, 2.0]).cuda(), torch.tensor([0.3, 1.0, -1.0]).cuda()
    f = Q.qlora_token_logprobs_fwd(z, t, entropy=True)
    d = Q.qlora_token_logprobs_bwd(z, t, f.lse, wl, entropy=f.entropy, dentropy=wh)

    def total(x):
        r = Q.qlora_token_logprobs_fwd(x, t, entropy=True)
        return ((r.logp.double() * wl) + (r.entropy.double() * wh)).sum().item()
    for i in range(3):
        for j in (0, 3, 7, 11):
            up, down = z.clone(), z.clone()
            up[i, j] += h
            down[i, j] -= h
            assert abs((total(up) - total(down)) / (2 * h) - d[i, j].item()) <= 3e-3


def test_captured_reused_outputs_and_a_side_stream():
    for N, V in ((1, 131072), (64, 32000)):
        z, t = make(N, V, BF16, 4)
        want = Q.qlora_token_logprobs_fwd(z, t, top=8, entropy=True)
        dl = torch.ones(N).cuda()
        grad = Q.qlora_token_logprobs_bwd(z, t, want.lse, dl)
        buf = torch.zeros_like(z)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f = Q.qlora_token_logprobs_fwd(buf, t, top=8, entropy=True)
            d = Q.qlora_token_logprobs_bwd(buf, t, f.lse, dl)
        graph.replay()
        buf.copy_(z)
        graph.replay()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        g = Q.qlora_token_logprobs_fwd(z, t, top=8, entropy=True, stream=side)
        h = Q.qlora_token_logprobs_fwd(z, t, top=8, entropy=True, out=g, stream=side)
        e = Q.qlora_token_logprobs_bwd(z, t, g.lse, dl, stream=side)
        torch.cuda.synchronize()
        assert h is g
        for r in (f, g):
            for name in ("logp", "lse", "entropy", "top_ids", "top_logp"):
                assert torch.equal(getattr(r, name), getattr(want, name))
        assert torch.equal(d, grad) and torch.equal(e, grad)


def device_reference(z, t, top):
    """The same definitions in 64 bits as the oracle's, on the device, for shapes
    that would take the host minutes (finite logits only)."""
    x = z.double()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1)
    lse = m[:, 0] + torch.log(s)
    counts = (t >= 0) & (t < z.shape[1])
    zt = x.gather(1, torch.where(counts, t, 0)[:, None])[:, 0]
    ent = torch.log(s) + (e * (m - x)).sum(1) / s
    ids = torch.sort(z.float() + 0.0, dim=1, descending=True, stable=True).indices[:, :top]
    return torch.where(counts, zt - lse, 0.0), lse, ent, ids, x.gather(1, ids) - lse[:, None]


# Rows enough that every CTA (or warp) of each variant of the forward walks over
# three at least, and that its ring of two batches wraps within them, at 148 SMs:
# 256, 512 and 128 threads and one warp to a row.
@pytest.mark.parametrize("N,V,pad", [(4000, 9001, 0), (4000, 32000, 0), (1700, 17001, 2), (4000, 5001, 3), (8000, 1000, 0),
                                     (8000, 509, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32] if torch.cuda.is_available() else [])
@pytest.mark.parametrize("top,entropy", [(20, True), (0, True), (0, False), (5, False)])
def test_many_rows_for_every_variant(N, V, pad, dtype, top, entropy):
    g = torch.Generator(device="cuda").manual_seed(N + V)
    z = (3 * torch.randn(N, V + pad, generator=g, device="cuda")).to(dtype)
    t = torch.randint(0, V, (N,), generator=g, device="cuda")
    t[1], t[N // 2] = V, -100
    dl, dh = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    f = Q.qlora_token_logprobs_fwd(z, t, vocab=V, top=top, entropy=entropy)
    d = Q.qlora_token_logprobs_bwd(z, t, f.lse, dl, entropy=f.entropy, dentropy=dh if entropy else None, vocab=V)
    assert not d[:, V:].any()
    for r in range(0, N, 500):
        b = slice(r, min(N, r + 500))
        logp, lse, ent, ids, best = device_reference(z[b, :V], t[b], top)
        size = lse.abs()
        assert ((f.lse[b] - lse).abs() <= 64 * U + 2 * U * size).all()
        assert ((f.logp[b] - logp).abs() <= 64 * U + 2 * U * (2 * size + logp.abs())).all()
        if entropy:
            assert ((f.entropy[b] - ent).abs() <= 64 * U * (2 + ent)).all()
        if top:
            assert torch.equal(f.top_ids[b].long(), ids)
            assert ((f.top_logp[b] - best).abs() <= 64 * U + 4 * U * (size[:, None] + best.abs())).all()
        q = z[b, :V].double() - f.lse[b, None].double()
        p, counts = torch.exp(q), (t[b] >= 0) & (t[b] < V)
        w = torch.where(counts, dl[b].double(), 0.0)[:, None]
        want, weight = -w * p, w.abs().expand_as(p)
        if entropy:
            want = want - dh[b, None].double() * p * (q + f.entropy[b, None].double())
            weight = weight + dh[b, None].double().abs() * (q.abs() + f.entropy[b, None].double())
        want.scatter_add_(1, torch.where(counts, t[b], 0)[:, None], w)
        rel = 64 * U + 4 * U * size[:, None] + 4 * U * q.abs()
        tol = rel * p * weight + 4 * U * want.abs() + 1e-38
        if dtype == BF16:
            tol = tol + 2.0 ** -8 * want.abs() * 1.01
        assert ((d[b, :V].double() - want).abs() <= tol).all()
