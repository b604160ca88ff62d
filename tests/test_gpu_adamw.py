"""AdamW over many tensors, with moments in 32 and in 8 bits.

The 8-bit states are defined down to the bit (every step one fp32 operation), so
they are compared for equality.  Tolerances elsewhere, with u = 2^-24, half a
step of fp32: a 32-bit moment takes three rounded operations on each term
(4 u of the terms' magnitudes); the update is a product, a quotient of two
units in the last place, a square root and three more operations on m' and v'
whose own errors are 3 u: 16 u of the update covers it (2^-22 for the fast
division is 4 u), and the subtraction adds u of the parameter.  A bf16
parameter adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as SO

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_quantized_lora_02_b200 as Q

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
SHAPES = [(3, 5), (16, 64), (64, 16), (1,), (255,), (256,), (257,), (0, 7), (13, 1001), (4099,), (512, 100), (2048,), (8, 4096)]


def make(shapes, seed, param=F32, grad=F32, copies=False):
    g = torch.Generator().manual_seed(seed)
    P = [(0.05 * torch.randn(*s, generator=g)).to(param).cuda() for s in shapes]
    G = [(1e-3 * torch.randn(*s, generator=g) * torch.exp(torch.randn(*s, generator=g))).to(grad).cuda() for s in shapes]
    C = [torch.zeros(s, dtype=BF16, device="cuda") for s in shapes] if copies else None
    return P, G, C


def host(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def codes(st, i):
    n, o = st.params[i].numel(), st.starts[i]
    b = slice(o // 256, o // 256 + -(-n // 256))
    return (st.m.view(torch.uint8)[o:o + n].cpu().numpy(), st.m_scale[b].cpu().numpy(),
            st.v[o:o + n].cpu().numpy(), st.v_scale[b].cpu().numpy())


def check_step(st, before, hyper, t, scale=None):
    """One step's results against the oracle's, from the tensors before it."""
    lr, b1, b2, eps, wd = hyper
    m_all, v_all = Q.qlora_adamw_state(st)
    for i, (p0, g0, m0, v0) in enumerate(before):
        n, o = p0.size, st.starts[i]
        if n == 0:
            continue
        p1, m1, v1 = SO.adamw_param(p0, m0, v0, g0, t, lr, b1, b2, eps, wd, scale)
        got = host(st.params[i]).astype(np.float64)
        upd = np.abs(p1 - p0 * (1 - lr * wd))
        # where m' cancels, its rounding counts against the terms, not against the sum
        gs = np.abs(g0 if scale is None else g0 * scale)
        den = np.sqrt(v1 / (1 - b2 ** t)) + eps
        slack = 8 * U * lr * (b1 * np.abs(m0) + (1 - b1) * gs) / (1 - b1 ** t) / den
        tol = 16 * U * upd + slack + 4 * U * np.abs(p0) + 1e-40
        if st.params[i].dtype == BF16:
            tol = tol + 2.0 ** -8 * np.abs(p1) * 1.01
        assert np.all(np.abs(got - p1) <= tol), i
        if st.copies is not None:
            assert torch.equal(st.copies[i], st.params[i].to(BF16))
        if st.state_bits == 32:
            gm, gv = host(m_all[o:o + n]), host(v_all[o:o + n])
            assert np.all(np.abs(gm - m1) <= 4 * U * (b1 * np.abs(m0) + (1 - b1) * gs) + 1e-44)
            assert np.all(np.abs(gv - v1) <= 4 * U * (np.abs(v1)) + 1e-44)
        else:
            m32, v32 = SO.adamw_moments(m0.astype(np.float32), v0.astype(np.float32), g0, b1, b2, scale)
            want = SO.adamw_encode(m32, v32)
            for a, b in zip(codes(st, i), want):
                assert np.array_equal(a, b), i
            dm, dv = SO.adamw_decode(*want)
            assert np.array_equal(host(m_all[o:o + n]), dm) and np.array_equal(host(v_all[o:o + n]), dv)


def snapshot(st):
    m, v = Q.qlora_adamw_state(st)
    out = []
    for i, p in enumerate(st.params):
        n, o = p.numel(), st.starts[i]
        out.append((host(p), host(st.grads[i]), host(m[o:o + n]).copy(), host(v[o:o + n]).copy()))
    return out


HYPER = (1e-3, 0.9, 0.999, 1e-8, 0.01)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,copies", [(BF16, F32, False), (F32, F32, False), (F32, F32, True), (BF16, BF16, False),
                                               (F32, BF16, True)])
def test_steps(bits, param, grad, copies):
    P, G, C = make(SHAPES, 1, param, grad, copies)
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits, copies=C)
    scale = torch.tensor([0.37], device="cuda")
    for t in (1, 2, 3, 4):
        g = torch.Generator().manual_seed(100 + t)
        for x in G:
            x.mul_((0.5 + torch.rand(x.shape, generator=g)).to(x.dtype).cuda())
        before = snapshot(st)
        s = scale if t > 2 else None
        Q.qlora_adamw_step(st, step=t, lr=HYPER[0], betas=HYPER[1:3], eps=HYPER[3], weight_decay=HYPER[4], grad_scale=s)
        check_step(st, before, HYPER, t, None if s is None else np.float32(0.37))


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_in_several_launches(bits):
    """More tensors than one launch takes, their sizes around block ends."""
    rng = np.random.default_rng(5)
    shapes = [(int(n),) for n in rng.integers(1, 600, size=901)] + [(20000,), (1,)]
    P, G, _ = make(shapes, 3)
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits)
    before = snapshot(st)
    Q.qlora_adamw_step(st, step=1, lr=1e-3, weight_decay=0.01)
    check_step(st, before, HYPER, 1)


def test_large_tensors_take_several_blocks_per_warp():
    P, G, _ = make([(3000, 4096), (777, 1001)], 4, BF16, F32)
    st = Q.qlora_adamw_alloc(P, G, state_bits=8)
    for t in (1, 2):
        before = snapshot(st)
        Q.qlora_adamw_step(st, step=t, lr=1e-3, weight_decay=0.01)
    check_step(st, before, HYPER, 2)


@pytest.mark.parametrize("bits", [32, 8])
def test_values_at_the_edges(bits):
    """Blocks of zeros, of tiny and of huge gradients, and gradients that vanish:
    nothing turns non-finite and the states are still the oracle's."""
    n = 256 * 8 + 17
    g = torch.zeros(n)
    g[256:512] = 1e-30
    g[512:768] = 1e-20
    g[768:1024] = 1e15
    g[1024] = 1.0
    g[1025:1280] = 1e-9
    g[1280:] = torch.linspace(-1, 1, n - 1280)
    P, G = [torch.full((n,), 0.5, device="cuda")], [g.cuda()]
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits)
    for t in (1, 2, 3):
        before = snapshot(st)
        Q.qlora_adamw_step(st, step=t, lr=1e-3, weight_decay=0.01)
        assert P[0].isfinite().all()
        if bits == 8:
            m32, v32 = SO.adamw_moments(before[0][2], before[0][3], before[0][1], 0.9, 0.999)
            for a, b in zip(codes(st, 0), SO.adamw_encode(m32, v32)):
                assert np.array_equal(a, b)
            assert (codes(st, 0)[2][v32 > 0] >= 1).all()      # a positive second moment never becomes zero
            assert t > 1 or (v32[512:1280] > 0).all()
        if t == 2:
            G[0].zero_()


def test_a_non_finite_gradient_spoils_its_block_only():
    n = 1024
    P, G, _ = make([(n,)], 6)
    st = Q.qlora_adamw_alloc(P, G, state_bits=8)
    clean = [t.clone() for t in P]
    st2 = Q.qlora_adamw_alloc(clean, [G[0].clone()], state_bits=8)
    G[0][300] = float("nan")
    Q.qlora_adamw_step(st, step=1, lr=1e-3)
    Q.qlora_adamw_step(st2, step=1, lr=1e-3)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[300] = False
    assert P[0][300].isnan() and torch.equal(P[0][keep], clean[0][keep])
    keep[256:512] = False
    assert torch.equal(st.m.view(torch.uint8)[keep], st2.m.view(torch.uint8)[keep]) and torch.equal(st.v[keep], st2.v[keep])


@pytest.mark.parametrize("bits", [32, 8])
def test_nothing_outside_the_tensors_changes(bits):
    """Parameters, copies and gradients are slices of larger buffers; the states'
    padding up to whole blocks stays zero."""
    shapes = [(1001,), (77,), (4096,)]
    _, G, _ = make(shapes, 8)
    buf = torch.full((8000,), 3.0, device="cuda")
    cbuf = torch.full((8000,), 3.0, dtype=BF16, device="cuda")
    at, P, C = 16, [], []
    for (n,) in shapes:
        P.append(buf[at:at + n])
        C.append(cbuf[at:at + n])
        at += -(-n // 16) * 16 + 16
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits, copies=C)
    inside = torch.zeros(8000, dtype=torch.bool, device="cuda")
    for p in P:
        o = (p.data_ptr() - buf.data_ptr()) // 4
        inside[o:o + p.numel()] = True
    Q.qlora_adamw_step(st, step=1, lr=1e-2)
    assert (buf[~inside] == 3).all() and (cbuf[~inside] == 3).all() and (buf[inside] != 3).any()
    for i, (n,) in enumerate(shapes):
        o = st.starts[i]
        end = st.starts[i + 1] if i + 1 < len(shapes) else st.m.numel()
        assert not st.m.view(torch.uint8 if bits == 8 else F32)[o + n:end].any() and not st.v[o + n:end].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_advance_with_the_clock(bits):
    P, G, _ = make([(64, 100), (5, 7)], 9)
    P2 = [p.clone() for p in P]
    st, ref = Q.qlora_adamw_alloc(P, G, state_bits=bits), Q.qlora_adamw_alloc(P2, G, state_bits=bits)
    clock = Q.qlora_adamw_clock(1e-3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Q.qlora_adamw_step(st, clock=clock, weight_decay=0.01)
    for t in (1, 2, 3):
        if t == 3:
            clock[0] = 5e-4
        graph.replay()
        Q.qlora_adamw_step(ref, step=t, lr=1e-3 if t < 3 else 5e-4, weight_decay=0.01)
    torch.cuda.synchronize()
    assert clock[1].item() == 3
    for a, b in zip(P + [st.m.view(torch.uint8), st.v], P2 + [ref.m.view(torch.uint8), ref.v]):
        assert torch.equal(a, b)


def test_other_gradients_and_a_side_stream():
    P, G, _ = make([(100, 33), (8,)], 10)
    P2 = [p.clone() for p in P]
    other = [g * 2 for g in G]
    st, ref = Q.qlora_adamw_alloc(P, G, state_bits=8), Q.qlora_adamw_alloc(P2, other, state_bits=8)
    st.set_grads(other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Q.qlora_adamw_step(st, step=1, lr=1e-3, stream=side)
    m, v = Q.qlora_adamw_state(st, stream=side)
    side.synchronize()
    Q.qlora_adamw_step(ref, step=1, lr=1e-3)
    m2, v2 = Q.qlora_adamw_state(ref)
    for a, b in zip(P + [m, v], P2 + [m2, v2]):
        assert torch.equal(a, b)


def test_eight_bit_states_train_like_thirty_two():
    """A quadratic with curvatures over four decades: 300 steps with 8-bit states
    end as low as with 32-bit ones to within a factor of 2, from a start 10^4
    times higher."""
    n = 4096
    curve = torch.logspace(-2, 2, n).cuda()
    ends = {}
    for bits in (32, 8):
        p = torch.ones(n, device="cuda")
        g = torch.empty_like(p)
        st = Q.qlora_adamw_alloc([p], [g], state_bits=bits)
        for t in range(1, 301):
            torch.mul(curve, p, out=g)
            Q.qlora_adamw_step(st, step=t, lr=2e-2 * 0.98 ** t + 1e-5)
        ends[bits] = (curve * p * p).sum().item()
    assert ends[8] <= 2 * ends[32] + 1e-4 * curve.sum().item()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scaled", [False, True])
def test_gradients_whose_squares_pass_the_range(bits, scaled):
    """Finite gradients up to the largest: the step is the formula's (AdamW's steps
    do not depend on the gradients' scale, so holding them to 2^60 changes none),
    the states stay finite, and the neighbours move on in the next steps."""
    n = 1024 + 100
    g0 = 1e-3 * torch.randn(n, generator=torch.Generator().manual_seed(1))
    big = {10: 1e19, 300: 1e20, 301: -3e38, 700: -2.0 ** 64, 1100: 3e38}
    P, G = [torch.full((n,), 0.5, device="cuda")], [g0.clone().cuda()]
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits)
    scale = torch.tensor([0.5], device="cuda") if scaled else None
    for t in (1, 2, 3, 4):
        if t == 2:
            for i, x in big.items():
                G[0][i] = x
        if t == 3:
            G[0].copy_(g0)
        before = snapshot(st)
        Q.qlora_adamw_step(st, step=t, lr=1e-3, weight_decay=0.01, grad_scale=scale)
        check_step(st, before, HYPER, t, None if scale is None else np.float32(0.5))
        assert all(x.isfinite().all() for x in P + list(Q.qlora_adamw_state(st)))
        p0, gr, m0, v0 = before[0]
        if t == 2 and bits == 32:
            # the formula itself, in 64 bits, without a limit on the gradient: where
            # |g| > 2^60 the old moments are below 2^-60 of the new ones
            want, _, _ = SO.adamw_param(p0, m0, v0, gr, t, *HYPER, limit=None)
            if scale is not None:
                want, _, _ = SO.adamw_param(p0, m0, v0, gr * 0.5, t, *HYPER, limit=None)
            assert np.all(np.abs(host(P[0]) - want) <= 32 * U * (np.abs(want - p0) + np.abs(p0)))
        if t > 2:
            near = np.arange(256, 512)
            near = near[(near != 300) & (near != 301)]
            assert bits == 8 or (host(P[0])[near] != p0[near]).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_non_finite_gradient_shows(bits, value):
    P, G, _ = make([(1024,)], 6)
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits)
    G[0][300] = value
    Q.qlora_adamw_step(st, step=1, lr=1e-3)
    m, v = Q.qlora_adamw_state(st)
    assert P[0][300].isnan() and P[0].isnan().sum() == 1 and m[300].isnan() and v[300].isnan()


@pytest.mark.parametrize("bits,param,grad,copies", [(32, F32, F32, True), (32, BF16, BF16, False), (8, BF16, F32, False),
                                                    (8, F32, BF16, True)])
def test_more_blocks_per_warp_than_its_loads_run_ahead(bits, param, grad, copies):
    """Four blocks to a warp with 32-bit states (loads one ahead), five with 8-bit
    ones (three ahead), at 148 SMs; a second tensor starts in a later chunk."""
    P, G, C = make([(6200 if bits == 32 else 7400, 4096), (777, 1001)], 4, param, grad, copies)
    st = Q.qlora_adamw_alloc(P, G, state_bits=bits, copies=C)
    Q.qlora_adamw_step(st, step=1, lr=1e-3, weight_decay=0.01)
    before = snapshot(st)
    Q.qlora_adamw_step(st, step=2, lr=1e-3, weight_decay=0.01)
    check_step(st, before, HYPER, 2)
