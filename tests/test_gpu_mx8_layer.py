"""The 8-bit operators as a training step and a decode step use them: a residual
stream's norm into 8-bit rows, a projection from them, the loss of the output
layer, and the gradients back through the same rows.  Every step is held against
64 bits on the inputs that it had, with its own operator's bounds; the whole step
gives the same bits again and from a replayed graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests import test_gpu_mx8_grad as grads  # noqa: E402
from tests import test_gpu_mx8_products as products  # noqa: E402
from tests import test_gpu_norm as norms  # noqa: E402

EPS = 1e-5


class Layer:
    """h = x + r, y = norm(h) W^T in 8 bits, loss of softmax(y head^T)."""

    def __init__(self, T, D, N, V, bits, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        b16 = torch.bfloat16
        self.x, self.r = rand(T, D).to(b16), (3 * rand(T, D)).to(b16)
        self.G = (1 + 0.2 * rand(D)).to(b16)
        self.W = (rand(N, D) / D ** 0.5).to(b16)
        self.head = (rand(V, N) / N ** 0.5).to(b16)
        self.labels = torch.randint(0, V, (T,), generator=g, device="cuda")
        self.labels[T // 2] = -100  # a padded row
        self.dloss = torch.where(self.labels == -100, 0.0, 1 / max(T - 1, 1))
        self.dH = (0.01 * rand(T, D)).to(b16)
        e = lambda *s, dtype=b16: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
        self.H, self.Y, self.dY = e(T, D), e(T, N), e(T, N)
        self.q, self.rstd = sg.Mx8.empty(T, D), e(T, dtype=torch.float32)
        self.loss, self.lse = e(T, dtype=torch.float32), e(T, dtype=torch.float32)
        self.dW, self.dN32 = e(N, D, dtype=torch.float32), e(T, D, dtype=torch.float32)
        self.dN, self.dX, self.dG, self.dhead = e(T, D), e(T, D), e(D), e(V, N)
        self.bits = bits

    def forward(self, h):
        h.rmsnorm_mx8(self.x, self.G, residual=self.r, H=self.H, rstd=self.rstd, eps=EPS, out=self.q)
        h.gemm_mx8(self.q, self.W8, self.Y)
        h.ce_forward(self.Y, self.head, self.labels, self.loss, self.lse)

    def backward(self, h):
        h.ce_backward(self.Y, self.head, self.labels, self.lse, self.dloss, self.dY, self.dhead)
        h.mx8_weight_grad(self.dY, self.q, self.dW)
        h.gemm_lowp(self.dY, self.W, self.dN32)
        self.dN.copy_(self.dN32)
        h.rmsnorm_backward(self.dN, self.H, self.G, self.rstd, self.dX, dG=self.dG, dH=self.dH)

    def results(self):
        return [t.clone() for t in (self.H, self.q.codes, self.q.scales, self.rstd, self.Y, self.loss,
                                    self.dY, self.dW, self.dX, self.dG)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("T,D,N,V", [(3, 64, 70, 50), (200, 330, 500, 300), (1030, 512, 1100, 700)])
def test_training_step(T, D, N, V, bits):
    with sg.Handle() as h:
        m = Layer(T, D, N, V, bits, seed=T)
        m.W8 = (h.mx8_quantize if bits == 8 else h.mx4_quantize)(m.W)
        h.set_workspace(max(h.ce_workspace_size(m.Y, m.head, backward=True),
                            h.rmsnorm_workspace_size(T, D), h.mx8_weight_grad_workspace_size(m.dY, m.q)))
        m.forward(h)
        m.backward(h)
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        assert torch.equal(m.H, (m.x.float() + m.r.float()).bfloat16())
        y, s = ref.norm(f(m.H), f(m.G), EPS)
        norms.check_rows(m.q, y, norms.delta(D))
        assert np.all(np.abs(f(m.rstd) - s) <= norms.delta(D) * s)
        rows = products.numbers(m.q)
        products.check(m.Y, rows, products.numbers(m.W8), 1.0, 0.0, None, "bf16")
        keep = f(m.labels) != -100
        assert np.isfinite(f(m.loss)).all() and (f(m.dY)[~keep] == 0).all()
        grads.check(m.dW, f(m.dY), rows[:, :D], 1.0, 0.0, None, "f32")
        norms.check_gradients(m.dX, m.dG, m.dN, m.H, m.G, m.rstd, m.dH, "bf16", "bf16", T, D)
        want = m.results()
        m.forward(h)
        m.backward(h)
        assert all(torch.equal(a, b) for a, b in zip(want, m.results()))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.forward(h)
            m.backward(h)
        for seed in (5, 6, 7):
            m.x.copy_(torch.randn(T, D, generator=torch.Generator(device="cuda").manual_seed(seed),
                                  device="cuda"))
            graph.replay()
            got = m.results()
            m.forward(h)
            m.backward(h)
            assert all(torch.equal(a, b) for a, b in zip(got, m.results()))


def test_gradients_against_differences():
    """Differences of the loss along dW agree with its square norm: the two losses are
    0.4 |dW| apart, their own rounding (bfloat16 rows of Y, 2^-9 of each) and the third
    derivative over a step of 0.2 are a few hundredths of that at most."""
    T, D, N, V = 256, 320, 384, 200
    with sg.Handle() as h:
        m = Layer(T, D, N, V, 8, seed=1)
        m.W8 = h.mx8_quantize(m.W)
        h.set_workspace(h.ce_workspace_size(m.Y, m.head, backward=True))
        m.forward(h)
        m.backward(h)
        total = lambda: float((m.loss.double() * m.dloss.double()).sum())  # noqa: E731
        slope = float((m.dW.double() ** 2).sum())
        step, at = 0.2 / slope ** 0.5, m.W.float()
        ends = []
        for sign in (1, -1):
            w = at + sign * step * m.dW / slope ** 0.5
            # (the projection in 32 bits: only the activations are in 8)
            m.Y.copy_(h.mx8_dequantize(m.q, torch.empty(T, D, device="cuda")) @ w.t())
            h.ce_forward(m.Y, m.head, m.labels, m.loss, m.lse)
            ends.append(total())
        assert abs((ends[0] - ends[1]) / (2 * step) / slope ** 0.5 - 1) < 0.05


def test_decode_steps_from_a_graph():
    """One token at a time through norm and projection, the stream updated in
    place, captured once and replayed."""
    D, N, steps = 512, 512, 5
    with sg.Handle() as h:
        W8 = h.mx8_quantize(torch.randn(N, D, device="cuda") / D ** 0.5)
        G = torch.ones(D, device="cuda", dtype=torch.bfloat16)
        x = torch.randn(1, D, device="cuda").bfloat16()
        stream, q = torch.zeros_like(x), sg.Mx8.empty(1, D)

        def step():
            h.rmsnorm_mx8(x, G, residual=stream, H=stream, out=q)
            h.gemm_mx8(q, W8, x)

        start = x.clone()
        step()  # (warm)
        x.copy_(start)
        stream.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        seen = []
        for _ in range(steps):
            graph.replay()
            seen.append((x.clone(), stream.clone()))
        x.copy_(start)
        stream.zero_()
        for a, b in seen:
            step()
            assert torch.equal(a, x) and torch.equal(b, stream)
