"""Layer norm (forward with the residual add, backward with the weight's
gradient) against a plain 64-bit form.

Tolerances.  u = 2^-24 is half a step of fp32.  A row's sums take fewer than 64
additions on any path from a value to the total (at most 32 values per thread,
5 shuffles, 17 warps), so a sum is off by at most 64 u times the sum of
magnitudes; the few products behind it and the square root add less than that
again: 128 u times the magnitudes that enter.  The weight's gradient adds M
rows: (M + 16) u.  An output in bf16 adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as SO

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_quantized_lora_02_b200 as Q

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def half(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(M, D, dtype, wdtype, seed, bias, residual):
    g = torch.Generator().manual_seed(seed)
    X = (torch.randn(M, D, generator=g) * 2 + 0.5).to(dtype).cuda()
    R = torch.randn(M, D, generator=g).to(dtype).cuda() if residual else None
    w = (1 + 0.2 * torch.randn(D, generator=g)).to(wdtype).cuda()
    b = torch.randn(D, generator=g).to(wdtype).cuda() if bias else None
    dY = torch.randn(M, D, generator=g).to(dtype).cuda()
    dS = torch.randn(M, D, generator=g).to(dtype).cuda() if residual else None
    return X, R, w, b, dY, dS


def check_forward(X, R, w, b, eps, rms, Y, S, mean, rstd):
    ref_S = X if R is None else (X.float() + R.float()).to(X.dtype)
    assert torch.equal(S, ref_S)
    x = f64(S)
    Yr, mr, rr = SO.norm_forward(x, f64(w), f64(b), eps, rms)
    size = np.abs(x).mean(axis=1)
    if not rms:
        assert np.all(np.abs(f64(mean) - mr) <= 128 * U * size + 1e-40)
    # the variance is off by 128 u of itself and by what the mean's error adds
    assert np.all(np.abs(f64(rstd) / rr - 1) <= 128 * U * (1 + (0 if rms else 1) * size * rr))
    term = np.abs(f64(w)) * rr[:, None] * (np.abs(x) + size[:, None]) * (1 + size * rr)[:, None]
    tol = 128 * U * (term + (0 if b is None else np.abs(f64(b)))) + half(X.dtype) * np.abs(Yr) * 1.01 + 1e-40
    assert np.all(np.abs(f64(Y) - Yr) <= tol)


def check_backward(dY, S, w, mean, rstd, dS, rms, dX, dw, db):
    r = SO.norm_backward(f64(dY), f64(S), f64(w), f64(mean), f64(rstd), f64(dS), rms)
    M = S.shape[0]
    g = np.abs(f64(dY) * f64(w))
    xs = f64(S)
    centre = 0.0 if rms else f64(mean)[:, None]
    rs = f64(rstd)[:, None]
    xh = (np.abs(xs) + np.abs(centre)) * rs           # bounds |xh| and its rounding
    term = rs * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    tol = 128 * U * (term + (0 if dS is None else np.abs(f64(dS)))) + half(S.dtype) * np.abs(r[0]) * 1.01 + 1e-40
    assert np.all(np.abs(f64(dX) - r[0]) <= tol)
    rows = (M + 16) * U
    assert np.all(np.abs(f64(dw) - r[1]) <= rows * (np.abs(f64(dY)) * xh).sum(0) + 1e-40)
    if db is not None:
        assert np.all(np.abs(f64(db) - r[2]) <= rows * np.abs(f64(dY)).sum(0) + 1e-40)


CASES = [(M, D) for M, D in ((1, 1), (2, 7), (5, 64), (3, 255), (9, 256), (700, 257), (4, 512), (33, 1000), (5, 1024),
                             (700, 1025), (2, 2047), (150, 2048), (303, 2049), (7, 4096), (310, 4099), (151, 5003),
                             (1, 8192), (160, 8192), (300, 8191), (160, 8193), (1, 16384), (150, 16384), (301, 16381),
                             (2000, 300), (1300, 511))]


@pytest.mark.parametrize("M,D", CASES)
@pytest.mark.parametrize("dtype,wdtype,rms,bias,residual", [
    (BF16, F32, True, False, True), (BF16, BF16, False, True, False), (F32, F32, False, True, True),
    (F32, BF16, True, True, False), (BF16, F32, False, False, True)] if torch.cuda.is_available() else [])
def test_forward_and_backward(M, D, dtype, wdtype, rms, bias, residual):
    X, R, w, b, dY, dS = inputs(M, D, dtype, wdtype, M + D, bias, residual)
    Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R, eps=1e-5, rms=rms)
    assert (S is X) == (R is None) and (mean is None) == rms
    check_forward(X, R, w, b, 1e-5, rms, Y, S, mean, rstd)
    dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, rms=rms, need_dbias=bias)
    assert (db is None) == (not bias)
    check_backward(dY, S, w, mean, rstd, dS, rms, dX, dw, db)
    again = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, rms=rms, need_dbias=bias)
    for p, q in zip((dX, dw, db), again):
        assert p is None or torch.equal(p, q)                      # deterministic


def test_every_width_class_with_one_row_and_many():
    """Each width around the limits of the kernels' variants, with rows that start
    at every offset from a 16-byte boundary."""
    for D in (8, 9, 249, 250, 505, 506, 1017, 1018, 2041, 2042, 4089, 4090, 8185, 8186, 16377, 16378):
        for M in (1, 17):
            X, R, w, b, dY, dS = inputs(M, D, BF16, F32, D, True, True)
            Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R)
            check_forward(X, R, w, b, 1e-5, False, Y, S, mean, rstd)
            dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, need_dbias=True)
            check_backward(dY, S, w, mean, rstd, dS, False, dX, dw, db)


def test_no_rows():
    X = torch.empty(0, 96, dtype=BF16, device="cuda")
    w = torch.ones(96, device="cuda")
    Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w)
    assert Y.shape == (0, 96) and rstd.shape == (0,)
    dX, dw, db = Q.qlora_layer_norm_bwd(X, X, w, mean, rstd, need_dbias=True,
                                        dweight=torch.full((96,), 7.0, device="cuda"))
    assert dX.shape == (0, 96) and not dw.any() and not db.any()


@pytest.mark.parametrize("D", [1000, 1001, 8192, 8193])
def test_nothing_is_written_outside_the_rows(D):
    """Outputs are slices of larger buffers: the values around them stay."""
    M = 5
    X, R, w, b, dY, dS = inputs(M, D, BF16, F32, 3, True, True)

    def framed():
        buf = torch.full((M * D + 128,), 5.0, dtype=BF16, device="cuda")
        return buf, buf[64:64 + M * D].view(M, D)
    (by, Y), (bs, S), (bx, dX) = framed(), framed(), framed()
    _, _, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R, Y=Y, S=S)
    Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, dX=dX)
    for buf in (by, bs, bx):
        assert (buf[:64] == 5).all() and (buf[64 + M * D:] == 5).all()


@pytest.mark.parametrize("D", [4096, 4097])
def test_in_place(D):
    M = 200
    X, R, w, b, dY, dS = inputs(M, D, BF16, F32, 11, True, True)
    Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R)
    x, r = X.clone(), R.clone()
    Y2, S2, m2, r2 = Q.qlora_layer_norm_fwd(x, w, bias=b, residual=r, Y=x, S=r)
    assert torch.equal(Y, Y2) and torch.equal(S, S2) and torch.equal(mean, m2) and torch.equal(rstd, r2)
    dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, need_dbias=True)
    for name in ("dY", "dS"):
        a, c = dY.clone(), dS.clone()
        got = Q.qlora_layer_norm_bwd(a, S, w, mean, rstd, dS=c, need_dbias=True, dX=a if name == "dY" else c)
        assert torch.equal(got[0], dX) and torch.equal(got[1], dw) and torch.equal(got[2], db)


def test_large_mean_and_tiny_variance():
    """The variance is summed around the mean, so a common offset costs nothing
    but the offset's own rounding; a constant row is divided by sqrt(eps)."""
    D = 4096
    g = torch.Generator().manual_seed(0)
    X = (torch.randn(64, D, generator=g) + 1000.0).cuda()
    X[3] = 2.5
    w = torch.ones(D, device="cuda")
    Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, eps=1e-5)
    check_forward(X, None, w, None, 1e-5, False, Y, S, mean, rstd)
    assert not Y[3].any()
    Y, _, _, rstd = Q.qlora_layer_norm_fwd(torch.zeros(2, D, device="cuda"), w, eps=1e-5, rms=True)
    assert not Y.any() and torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_non_finite_value_stays_in_its_row(value):
    X, _, w, b, _, _ = inputs(300, 1001, BF16, F32, 5, True, False)
    clean, _, _, _ = Q.qlora_layer_norm_fwd(X, w, bias=b)
    X[17, 400] = value
    Y, _, _, _ = Q.qlora_layer_norm_fwd(X, w, bias=b)
    keep = torch.arange(300, device="cuda") != 17
    assert Y[17].isnan().all() and torch.equal(Y[keep], clean[keep])


def test_gradient_against_differences():
    """Central differences of a weighted sum of the forward's outputs, in fp32:
    step h = 2^-4, so the difference is off by at most 2 * 128 u |f| / (2 h) for
    rounding and by h^2 / 6 of the third derivative, which for values of order
    one over D = 40 entries stays below 0.02 here."""
    D, h = 40, 2.0 ** -4
    X, R, w, b, dY, dS = inputs(3, D, F32, F32, 1, True, True)

    def f(X_, w_, b_):
        Y, S, _, _ = Q.qlora_layer_norm_fwd(X_, w_, bias=b_, residual=R)
        return ((Y.double() * dY.double()).sum() + (S.double() * dS.double()).sum()).item()
    _, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R)
    dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, need_dbias=True)
    for i, j in ((0, 0), (1, 17), (2, 39)):
        for t, grad in ((X, dX[i, j]), (w, dw[j]), (b, db[j])):
            at = (i, j) if t is X else (j,)
            up, down = t.clone(), t.clone()
            up[at] += h
            down[at] -= h
            args = [(up if t is x else x, down if t is x else x) for x in (X, w, b)]
            num = (f(*(p for p, _ in args)) - f(*(q for _, q in args))) / (2 * h)
            assert abs(num - grad.item()) <= 0.02


def test_captured_and_replayed_on_a_side_stream():
    M, D = 300, 4099
    X, R, w, b, dY, dS = inputs(M, D, BF16, F32, 2, True, True)
    want_f = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R)
    want_b = Q.qlora_layer_norm_bwd(dY, want_f[1], w, want_f[2], want_f[3], dS=dS, need_dbias=True)
    other = X.clone() * 2
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    buf = other.clone()
    with torch.cuda.graph(graph):
        f = Q.qlora_layer_norm_fwd(buf, w, bias=b, residual=R)
        g = Q.qlora_layer_norm_bwd(dY, f[1], w, f[2], f[3], dS=dS, need_dbias=True)
    graph.replay()
    buf.copy_(X)
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(want_f + want_b, f + g):
        assert torch.equal(p, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R, stream=side)
    g = Q.qlora_layer_norm_bwd(dY, f[1], w, f[2], f[3], dS=dS, need_dbias=True, stream=side)
    side.synchronize()
    for p, q in zip(want_f + want_b, f + g):
        assert torch.equal(p, q)


# The longest path of additions in a row's sum is 40 values of a thread (rows of
# 16377 to 16383 values), 5 shuffles and 16 warps: 61; the 1024-thread forward has
# 16 + 5 + 32.  Both are fewer than the 64 that the tolerances above count.
@pytest.mark.parametrize("M,D", [(40, 300), (700, 1001), (3, 2049), (40, 8192), (300, 8192), (150, 16381)])
@pytest.mark.parametrize("dtype,rms,scale", [(BF16, True, 1e20), (F32, True, 1e36), (F32, False, 1e20), (BF16, False, 1e30),
                                             (BF16, True, 1e36)] if torch.cuda.is_available() else [])
def test_rows_whose_squares_pass_the_range(M, D, dtype, rms, scale):
    """Finite rows whose sum of squares is infinite in fp32, beside ordinary ones:
    the same formula, forward and backward.  rstd is a normal number here (above
    1e-37), so the tolerances are those of ordinary rows."""
    X, R, w, b, dY, dS = inputs(M, D, dtype, F32, M + D, True, True)
    X[::2] = (X[::2].double() * scale).to(dtype)
    for res in (R, None):
        Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=res, rms=rms)
        check_forward(X, res, w, b, 1e-5, rms, Y, S, mean, rstd)
        dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, rms=rms, need_dbias=True)
        check_backward(dY, S, w, mean, rstd, dS, rms, dX, dw, db)


@pytest.mark.parametrize("D", [64, 1001, 8192])
def test_the_largest_values(D):
    """+-3e38: rstd is 1 / 3e38, a subnormal number whose half step is 2^-150 /
    2^-128 = 2^-22 of it; then the product and its rounding to the output."""
    sign = torch.where(torch.arange(D) % 3 == 1, -1.0, 1.0).cuda()
    w = torch.ones(D, device="cuda")
    for dtype in (F32, BF16):
        X = (3e38 * sign).to(dtype).repeat(5, 1)
        Y, _, _, rstd = Q.qlora_layer_norm_fwd(X, w, rms=True)
        want = 1.0 / X[0, 0].double()
        assert ((rstd.double() - want).abs() <= (2.0 ** -22 + 128 * U) * want).all()
        assert ((Y.double() - sign).abs() <= 2.0 ** -22 + 128 * U + half(dtype)).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rms", [True, False])
@pytest.mark.parametrize("M,D", [(300, 1001), (2500, 300), (40, 4096), (300, 8192), (300, 9001)])
def test_a_row_with_a_non_finite_value_is_nan_throughout(value, rms, M, D):
    for dtype in (BF16, F32):
        X, R, w, b, _, _ = inputs(M, D, dtype, F32, 5, True, True)
        keep = torch.arange(M, device="cuda") != 17
        for res in (None, R):
            clean = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=res, rms=rms)[0]
            bad = X.clone()
            bad[17, D // 2] = value
            Y, _, _, rstd = Q.qlora_layer_norm_fwd(bad, w, bias=b, residual=res, rms=rms)
            assert Y[17].isnan().all() and rstd[17].isnan() and torch.equal(Y[keep], clean[keep])


def test_a_row_whose_sum_passes_the_range_is_nan_throughout():
    """Only with a mean: its sum is fp32."""
    X = torch.full((3, 1000), 1e30, device="cuda")
    X[1] = 1e37
    w = torch.ones(1000, device="cuda")
    Y = Q.qlora_layer_norm_fwd(X, w, bias=w)[0]
    assert Y[1].isnan().all() and Y[0].isfinite().all() and Y[2].isfinite().all()
    assert Q.qlora_layer_norm_fwd(X, w, bias=w, rms=True)[0].isfinite().all()


def test_in_place_without_a_residual_leaves_no_input_for_the_backward():
    X, _, w, b, _, _ = inputs(20, 300, BF16, F32, 3, True, False)
    want, S, _, _ = Q.qlora_layer_norm_fwd(X, w, bias=b)
    assert S is X
    x = X.clone()
    Y, S, mean, rstd = Q.qlora_layer_norm_fwd(x, w, bias=b, Y=x)
    assert Y is x and torch.equal(Y, want) and S is None
    with pytest.raises(ValueError, match="S is required"):
        Q.qlora_layer_norm_bwd(x, S, w, mean, rstd)
    empty = X[:0]
    assert Q.qlora_layer_norm_fwd(empty, w, bias=b)[1] is empty


@pytest.mark.parametrize("D", [1, 4, 64, 100, 128])
@pytest.mark.parametrize("dtype", [BF16, F32] if torch.cuda.is_available() else [])
def test_constant_rows_of_huge_values(D, dtype):
    """xh is 0 throughout a constant row and rstd is 1 / sqrt(eps) = 316, so that
    mean rstd is infinite; dX is rstd (g - mean g), and nothing of the windows next
    to the row enters it.  (-1)^r 2^(120 + r) 2^7 stays below 2^128, so mean is exact
    where D is a power of two; elsewhere the row's own rounding counts as usual."""
    X = torch.stack([torch.full((D,), (-1.0) ** r * 2.0 ** (118 + r)) for r in range(3)]).to(dtype).cuda()
    _, _, w, _, dY, _ = inputs(3, D, dtype, F32, 4, False, False)
    for bias in (False, True):
        Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, eps=1e-5)
        dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, need_dbias=bias)
        assert dX.isfinite().all() and dw.isfinite().all()
        if D & (D - 1) == 0:
            assert torch.equal(mean, X[:, 0].float()) and not Y.any() and not dw.any()
            check_backward(dY, S - mean[:, None].to(dtype), w, mean * 0, rstd, None, False, dX, dw, db)


# Rows enough that every CTA (or warp) of each variant walks over at least six, two
# more than the most rows that its loads run ahead, at 148 SMs: a warp to a row
# with 8, 16 and 32 values to a thread; 32 to 512 threads; 16, 32 and 40 values.
@pytest.mark.parametrize("M,D", [(13900, 200), (13900, 300), (13900, 511), (13900, 1000), (6900, 2048), (2590, 2049),
                                 (2590, 4099), (1740, 8192), (870, 8191), (870, 12000), (870, 16381)])
@pytest.mark.parametrize("dtype,wdtype,rms,bias,residual", [
    (BF16, F32, True, False, True), (F32, F32, False, True, True), (BF16, BF16, False, True, False),
    (F32, F32, True, False, False)] if torch.cuda.is_available() else [])
def test_many_rows_for_every_variant(M, D, dtype, wdtype, rms, bias, residual):
    X, R, w, b, dY, dS = inputs(M, D, dtype, wdtype, M + D, bias, residual)
    Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=R, rms=rms)
    check_forward(X, R, w, b, 1e-5, rms, Y, S, mean, rstd)
    dX, dw, db = Q.qlora_layer_norm_bwd(dY, S, w, mean, rstd, dS=dS, rms=rms, need_dbias=bias)
    check_backward(dY, S, w, mean, rstd, dS, rms, dX, dw, db)


@pytest.mark.parametrize("D", [300, 1001, 8192, 16381])
@pytest.mark.parametrize("rms", [True, False])
def test_rows_beyond_the_range_in_place(D, rms):
    """Such rows are read again after their sums: in place they give what they give
    elsewhere, for the first, the last and neighbouring rows of a CTA."""
    M = 900
    X, R, w, b, _, _ = inputs(M, D, BF16, F32, 12, True, True)
    for r in (0, 1, 5, 148, 296, 444, 592, 898, 899):
        X[r] = X[r].double().mul(1e25).to(BF16)
    X[7, 3] = float("inf")
    for res in (None, R):
        Y, S, mean, rstd = Q.qlora_layer_norm_fwd(X, w, bias=b, residual=res, rms=rms)
        keep = torch.arange(M, device="cuda") != 7
        assert Y[keep].isfinite().all() and Y[7].isnan().all()
        for y_in_residual in (False, True):
            x, r = X.clone(), None if res is None else R.clone()
            if res is None and y_in_residual:
                continue
            y, s = (r, x) if y_in_residual else (x, r)
            Y2, S2, m2, r2 = Q.qlora_layer_norm_fwd(x, w, bias=b, residual=r, rms=rms, Y=y, S=s)
            for p, q in ((Y, Y2), (S, S2), (mean, m2), (rstd, r2)):
                assert p is None or q is None or torch.equal(p[keep], q[keep])
            assert Y2[7].isnan().all() and r2[7].isnan()
