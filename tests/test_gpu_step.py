"""One fine-tuning step through the library's operators as they are used together:
residual add and rms norm -> NF4 linear layer with its adapter -> log
probabilities of the next tokens -> their gradient -> the layer's backward ->
the norm's backward -> AdamW over the adapter and the norm's weight.  Run
eagerly, and captured into a graph that advances a clock; compared with the same
step in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as SO

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import bit_quantized_lora_02_b200 as Q

BF16 = torch.bfloat16
M, K, V, PADDED, R, ALPHA = 200, 256, 1003, 1008, 8, 16.0


class Step:
    """Everything a training program keeps: inputs, the quantised head, masters
    with bf16 copies, gradient buffers and the optimiser's state."""

    def __init__(self, bits, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.x = torch.randn(M, K, generator=g).to(BF16).cuda()
        self.res = torch.randn(M, K, generator=g).to(BF16).cuda()
        self.t = torch.randint(0, V, (M,), generator=g).cuda()
        self.t[::17] = -100
        self.head = (0.05 * torch.randn(PADDED, K, generator=g)).to(BF16).cuda()
        self.q = Q.nf4_quantize(self.head)
        masters = [1 + 0.1 * torch.randn(K, generator=g), torch.randn(R, K, generator=g) / 8,
                   0.01 * torch.randn(PADDED, R, generator=g)]
        self.p = [m.cuda() for m in masters]
        self.c = [m.to(BF16) for m in self.p]
        self.g = [torch.zeros_like(m) for m in self.p]
        self.opt = Q.qlora_adamw_alloc(self.p, self.g, state_bits=bits, copies=self.c)
        self.dl = torch.full((M,), -1.0 / M, device="cuda")          # loss = -mean logp

    def forward_backward(self):
        w, A, B = self.c
        y, s, _, rstd = Q.qlora_layer_norm_fwd(self.x, w, residual=self.res, rms=True)
        z, T = Q.qlora_linear_fwd(y, self.q, A, B, ALPHA)
        f = Q.qlora_token_logprobs_fwd(z, self.t, vocab=V, entropy=True)
        dz = Q.qlora_token_logprobs_bwd(z, self.t, f.lse, self.dl, vocab=V, dlogits=z)      # in place
        dy, _, _ = Q.qlora_linear_bwd(dz, y, self.q, A, B, ALPHA, T_save=T, dA=self.g[1], dB=self.g[2])
        dx, _, _ = Q.qlora_layer_norm_bwd(dy, s, w, None, rstd, rms=True, dweight=self.g[0])
        return f, dx


def reference(st):
    """Loss and gradients in 64 bits from the same bf16 weights."""
    W = Q.nf4_dequantize(st.q).double().cpu().numpy()
    w, A, B = (c.double().cpu().numpy() for c in st.c)
    s = (st.x.float() + st.res.float()).to(BF16).double().cpu().numpy()
    y, _, rstd = SO.norm_forward(s, w, None, 1e-5, True)
    sc = ALPHA / R
    z = y @ W.T + sc * (y @ A.T) @ B.T
    t = st.t.cpu().numpy()
    r = SO.token_logprobs(z[:, :V], t)
    dz = np.zeros_like(z)
    dz[:, :V] = SO.token_logprobs_backward(z[:, :V], t, r["lse"], st.dl.cpu().numpy())
    dy = dz @ W + sc * (dz @ B) @ A
    dA, dB = sc * (dz @ B).T @ y, sc * dz.T @ (y @ A.T)
    dx, dw, _ = SO.norm_backward(dy, s, w, None, rstd, None, True)
    return r, dx, [dw, dA, dB]


@pytest.mark.parametrize("bits", [32, 8])
def test_step_against_64_bits(bits):
    """Each value passes a handful of roundings to bf16 (2^-8 each: S, Y, the
    logits, their gradient, dY, dX) and products of K = 256 or V = 1003 terms
    whose errors are independent: 3% of a gradient's norm bounds six of them
    (6 x 2^-8 = 2.3%); a log probability is off by the logit's own rounding and
    the input's, 2^-8 (|z| + |lse|) + 2^-7 |y| |w| sqrt(K) of its terms."""
    st = Step(bits)
    ref, dx_ref, grads = reference(st)
    before = [p.clone() for p in st.p]
    f, dx = st.forward_backward()
    size = np.abs(ref["lse"]) + 8
    assert np.all(np.abs(f.logp.double().cpu().numpy() - ref["logp"]) <= 2.0 ** -6 * size)
    assert np.all(f.logp.cpu().numpy()[::17] == 0)
    for got, want in zip([dx] + st.g, [dx_ref] + grads):
        got = got.double().cpu().numpy()
        assert np.linalg.norm(got - want) <= 0.03 * np.linalg.norm(want)
    Q.qlora_adamw_step(st.opt, step=1, lr=1e-3, weight_decay=0.01)
    for p, old, g, c in zip(st.p, before, st.g, st.c):
        # the first step moves every weight by lr g / (|g| + eps) beside the decay
        want = old.double() * (1 - 1e-5) - 1e-3 * g.double() / (g.double().abs() + 1e-8)
        assert ((p.double() - want).abs() <= 1e-3 * 2.0 ** -18 + 2.0 ** -22 * want.abs()).all()
        assert torch.equal(c, p.to(BF16))
    assert Q.qlora_device_status() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_steps_equal_eager_ones(bits):
    """The whole step in a graph, replayed: bit for bit the eager steps (every
    kernel sums in a fixed order)."""
    eager, cap = Step(bits), Step(bits)
    clock = Q.qlora_adamw_clock(1e-3)
    warm = Step(bits)
    warm.forward_backward()                      # kernels loaded before the capture
    Q.qlora_adamw_step(warm.opt, step=1, lr=1e-3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f, dx = cap.forward_backward()
        Q.qlora_adamw_step(cap.opt, clock=clock, weight_decay=0.01)
    for t in (1, 2, 3):
        graph.replay()
        fe, dxe = eager.forward_backward()
        Q.qlora_adamw_step(eager.opt, step=t, lr=1e-3, weight_decay=0.01)
        torch.cuda.synchronize()
        assert torch.equal(f.logp, fe.logp) and torch.equal(dx, dxe)
        for a, b in zip(cap.p + cap.c + cap.g, eager.p + eager.c + eager.g):
            assert torch.equal(a, b)
    assert clock[1].item() == 3


def test_two_streams_at_once():
    """Two steps on two streams, each with its own tensors, give what each gives
    alone."""
    alone = [Step(8, seed) for seed in (1, 2)]
    want = [s.forward_backward()[1] for s in alone]
    both = [Step(8, seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in both]
    got = []
    for s, stream in zip(both, streams):
        with torch.cuda.stream(stream):
            got.append(s.forward_backward()[1])
            Q.qlora_adamw_step(s.opt, step=1, lr=1e-3)
    for s in alone:
        Q.qlora_adamw_step(s.opt, step=1, lr=1e-3)
    torch.cuda.synchronize()
    for a, b, s, r in zip(got, want, both, alone):
        assert torch.equal(a, b)
        assert all(torch.equal(x, y) for x, y in zip(s.p, r.p))


def test_two_threads_at_once():
    """Calls of two host threads, each on its own stream, do not disturb each other."""
    import threading
    g = torch.Generator().manual_seed(5)
    x, w = torch.randn(33, 1001, generator=g).to(BF16).cuda(), torch.randn(1001, generator=g).cuda()
    t = torch.arange(33).cuda()
    want = Q.qlora_layer_norm_fwd(x, w), Q.qlora_token_logprobs_fwd(x, t, top=5, entropy=True)
    dw = Q.qlora_layer_norm_bwd(x, x, w, want[0][2], want[0][3])[1]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            for _ in range(100):
                y, _, mean, rstd = Q.qlora_layer_norm_fwd(x, w, stream=stream)
                d = Q.qlora_layer_norm_bwd(x, x, w, mean, rstd, stream=stream)[1]
                f = Q.qlora_token_logprobs_fwd(x, t, top=5 * k, entropy=True, stream=stream)
            stream.synchronize()
            assert torch.equal(y, want[0][0]) and torch.equal(d, dw) and torch.equal(f.lse, want[1].lse)
            assert not k or torch.equal(f.top_ids, want[1].top_ids)
        except Exception as e:          # a failed assertion included: it belongs to the main thread
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong


def test_more_than_2_to_the_31_values():
    """The last rows (blocks) of tensors whose offsets pass 31 bits are those of the
    same rows alone; as many rows as take the same variant of the kernel."""
    n, part = 68000, 5000
    z = torch.randn(n, 32000, device="cuda", dtype=BF16)
    assert z.numel() > 1 << 31
    t = torch.randint(0, 32000, (n,), device="cuda")
    dl = torch.randn(n, device="cuda")
    all_, one = (Q.qlora_token_logprobs_fwd(a, b, top=3, entropy=True) for a, b in ((z, t), (z[-part:], t[-part:])))
    for a, b in zip(vars(all_).values(), vars(one).values()):
        assert torch.equal(a[-part:], b)
    d = Q.qlora_token_logprobs_bwd(z[-part:], t[-part:], one.lse, dl[-part:])
    Q.qlora_token_logprobs_bwd(z, t, all_.lse, dl, dlogits=z)
    assert torch.equal(z[-part:], d)
    del z, d

    n = 263000
    x = torch.randn(n, 8192, device="cuda", dtype=BF16)
    assert x.numel() > 1 << 31
    w = torch.randn(8192, device="cuda")
    y, s, mean, rstd = Q.qlora_layer_norm_fwd(x, w, w, residual=x)
    tail = Q.qlora_layer_norm_fwd(x[-part:], w, w, residual=x[-part:])
    for a, b in zip((y, s, mean, rstd), tail):
        assert torch.equal(a[-part:], b)
    want = Q.qlora_layer_norm_bwd(y[-part:], s[-part:], w, mean[-part:], rstd[-part:])[0]
    Q.qlora_layer_norm_bwd(y, s, w, mean, rstd, dX=y)
    assert torch.equal(y[-part:], want)
    del x, y, s, want, tail

    n, part = (1 << 31) + 300, 256 * 9 + 44
    p, g = (torch.randn(n, device="cuda", dtype=BF16) for _ in range(2))
    small = [p[-part:].clone()], [g[-part:].clone()]
    big, little = Q.qlora_adamw_alloc([p], [g], 8), Q.qlora_adamw_alloc(*small, 8)
    for step in (1, 2):
        for state in (big, little):
            Q.qlora_adamw_step(state, step=step, lr=1e-2)
    assert torch.equal(p[-part:], small[0][0])
    blocks = -(-part // 256)
    for a, b in ((big.m.view(torch.uint8), little.m.view(torch.uint8)), (big.v, little.v)):
        assert torch.equal(a[-256 * blocks:], b)
    assert torch.equal(big.m_scale[-blocks:], little.m_scale) and torch.equal(big.v_scale[-blocks:], little.v_scale)
    m, v = (a[-256 * blocks:] for a in Q.qlora_adamw_state(big))
    for a, b in zip((m, v), Q.qlora_adamw_state(little)):
        assert torch.equal(a, b)


def test_weight_gradient_of_more_than_2_to_the_31_values():
    """The sums over all rows, in 64 bits by blocks of rows.  At 148 SMs each of 296
    CTAs adds 889 rows, the reduction 10 of their sums per thread and 5 more: fewer
    than 1024 roundings, on terms with 4 of their own."""
    n, D = 263000, 8192
    g = torch.Generator(device="cuda").manual_seed(3)
    s, dy = (torch.randn(n, D, generator=g, device="cuda", dtype=BF16) for _ in range(2))
    w = torch.ones(D, device="cuda")
    mean, rstd = 0.1 * torch.randn(n, generator=g, device="cuda"), 0.5 + torch.rand(n, generator=g, device="cuda")
    _, dw, db = Q.qlora_layer_norm_bwd(dy, s, w, mean, rstd, need_dbias=True, dX=None)
    want = torch.zeros(4, D, dtype=torch.float64, device="cuda")
    for at in range(0, n, 10000):
        b = slice(at, at + 10000)
        d = dy[b].double()
        xh = (s[b].double() - mean[b, None].double()) * rstd[b, None].double()
        size = (s[b].double().abs() + mean[b, None].double().abs()) * rstd[b, None].double()
        want += torch.stack([(d * xh).sum(0), d.sum(0), (d.abs() * size).sum(0), d.abs().sum(0)])
    assert ((dw.double() - want[0]).abs() <= 1024 * 2.0 ** -24 * want[2]).all()
    assert ((db.double() - want[1]).abs() <= 1024 * 2.0 ** -24 * want[3]).all()
