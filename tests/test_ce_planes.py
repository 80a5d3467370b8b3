"""The output layer's loss on 32-bit operands that use all 24 bits, as products
of three bfloat16 planes: what a plane product that is left out would change.

X has one nonzero a row and W one a column, so every logit and nearly every
element of a gradient is one product, which only the planes' own errors touch:
the three products left out, at most 2^-24 of it each, and a rounding of the
sum at each of six steps, 9 u with u = 2^-24.  On the CPU a model of the planes
shows that leaving out any of the six breaks that bound; on the GPU the loss
and its gradients keep it."""
import numpy as np
import pytest

from tests import ce_reference as ref

U = 2.0 ** -24
PRODUCTS = [(0, 2), (2, 0), (1, 1), (0, 1), (1, 0), (0, 0)]  # (plane of A, plane of B)


def all_bits(rng, n):
    """1 .. 2, the last bit set."""
    return 1 + (2 * rng.integers(0, 1 << 22, n) + 1) * 2.0 ** -23


def bfloat16(x):
    """float64 values that are float32 ones, rounded to the nearest bfloat16."""
    b = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7fff + ((b >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xffff0000)
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def planes(x):
    h = bfloat16(x)
    m = bfloat16(x - h)
    return h, m, bfloat16(x - h - m)


class Sparse:
    """T rows with one nonzero each, W with one a column; every other row's
    label is the word that it meets."""

    def __init__(self, T, V, D, seed=0):
        rng = np.random.default_rng([seed, T, V, D])
        self.T, self.V, self.D = T, V, D
        self.word = (V - 8) // D * np.arange(D) + 7
        self.col = np.arange(T) % D
        self.a, self.b = all_bits(rng, D), all_bits(rng, T)
        self.q = all_bits(rng, T) * np.where(rng.random(T) < 0.5, -1.0, 1.0)
        self.x, self.w = np.zeros((T, D)), np.zeros((V, D))
        self.x[np.arange(T), self.col] = self.b
        self.w[self.word, np.arange(D)] = self.a
        self.labels = self.word[np.where(np.arange(T) % 2 == 0, self.col, (self.col + 1) % D)]


SIZES = [(520, 16500, 300), (1100, 8200, 600), (4200, 2100, 2000)]


@pytest.mark.parametrize("T,V,D", SIZES)
def test_the_bound_misses_no_plane(T, V, D):
    s = Sparse(T, V, D)
    for x, y in ((s.b, s.a[s.col]), (s.q.astype(np.float32).astype(float), s.a[s.col]), (s.q, s.b)):
        px, py = planes(x), planes(y)
        assert all(np.array_equal(sum(p), v) for p, v in ((px, x), (py, y)))

        def off(left_out):
            got = sum(px[i] * py[j] for i, j in PRODUCTS if (i, j) != left_out)
            return (np.abs(got - x * y) / np.abs(x * y)).max()

        assert off(None) <= 3 * U
        for p in PRODUCTS:
            assert off(p) > 30 * U, p


@pytest.mark.gpu
@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("T,V,D", SIZES)
def test_loss_and_gradients_of_all_bits(T, V, D, small):
    """small: pieces of the vocabulary as the least workspace gives them."""
    torch = pytest.importorskip("torch")
    import fp32_gemm_major_amd as sg
    s = Sparse(T, V, D)
    X, W = (torch.from_numpy(v).float().cuda() for v in (s.x, s.w))
    Y = torch.from_numpy(s.labels).cuda()
    loss, lse, dl = (torch.empty(T, device="cuda") for _ in range(3))
    with sg.Handle(workspace=False) as h:
        # logits of 64 to 256 for one word, 0 for the others: lse is the logit,
        # off by the planes' 9 u and its own rounding
        h.set_workspace(h.ce_workspace_size(X, W, least=small))
        h.ce_forward(X, W, Y, loss, lse, alpha=64.0)
        z, _, want = ref.forward(s.x, s.w, s.labels, 64.0)
        assert np.all(np.abs(lse.double().cpu().numpy() - want) <= 11 * U * want)

        # logits of 1 to 4: p = exp(z - lse) is off by z's 9 u * 4, the
        # difference's and the argument's roundings (17 u and 25 u: |z - lse|
        # is below 17) and the exponential's (4 u); dz by that and two roundings
        z, _, want = ref.forward(s.x, s.w, s.labels)
        lse.copy_(torch.from_numpy(want))
        dl.copy_(torch.from_numpy(s.q))
        dX, dW = torch.full_like(X, 9.0), torch.full_like(W, 9.0)
        h.set_workspace(h.ce_workspace_size(X, W, backward=True, least=small))
        h.ce_backward(X, W, Y, lse, dl, dX, dW)
    e = lse.double().cpu().numpy()
    dz = ref.dlogits(z, s.labels, e, s.q)
    p = np.abs(s.q)[:, None] * np.exp(z - e[:, None])
    ez = 82 * U * p + 2 * U * np.abs(dz)
    dx, dw = ref.gradients(s.x, s.w, s.labels, dz)
    terms = -(-T // D)  # of a sum for dW
    for got, want, err, mag, n in ((dX, dx, ez @ s.w, np.abs(dz) @ s.w, 1),
                                   (dW, dw, ez.T @ s.x, np.abs(dz).T @ s.x, terms)):
        bound = err + (6 * n + 5) * U * mag
        off = np.abs(got.double().cpu().numpy() - want)
        assert np.all(off <= bound), (np.nanmax(off - bound), np.argwhere(~(off <= bound))[:3])
