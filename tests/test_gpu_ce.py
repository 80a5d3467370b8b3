"""The output layer's cross entropy and its gradients on the GPU against the
plain 64-bit implementation (ce_reference).

Most cases draw X and W from small integers times powers of two, so that the
logits are exact in any order of summation.  What is left, with u = 2^-24:

* exp: |z - lse| <= 40 here; the argument's product with log2(e) and its
  rounding move the result by at most 2*40*u relative, v_exp_f32 by 2^-22;
* the sum of V exponentials: a lane adds at most V/64 of them one after the
  other, the rest are joined in fewer than 32 steps, each step with an
  exponential's error of its own: (V/64 + 32) u + 32 * 2^-20 relative at the
  most; with those lse is off by E = (V/64 + 32) u + 2^-14, plus |lse| 4u from
  the logarithm's result and the addition of the maximum;
* dz: relative E + 2^-19 of p, then half a step of its type (up to 128 rows of
  16-bit operands keep what that leaves, rounded in turn: half a step of half a
  step);
* a gradient: that error of every dz against |W| or |X|, 4 n u of the sum of
  magnitudes of n products, and half a step of the type of the result.
  (binary16: dz and X may also lose half a step of the subnormal numbers.)"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import ce_reference as ref  # noqa: E402
from tests import mx_reference  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


class Problem:
    """Exact-logit inputs on the host (64-bit) and the device."""

    def __init__(self, T, V, D, dt, seed=0, ignored=0.2, alpha=0.5, uneven=False, pad=0):
        rng = np.random.default_rng([seed, T, V, D])
        self.T, self.V, self.D, self.dt, self.alpha = T, V, D, dt, alpha
        # |z| stays near 10 whatever D is: W has about 16 nonzeros a row
        self.x = rng.integers(-4, 5, (T, D)).astype(float) / 2
        self.w = rng.integers(-4, 5, (V, D)).astype(float) / 4 * (rng.random((V, D)) < 16 / D)
        self.labels = rng.integers(0, V, T)
        self.labels[rng.random(T) < ignored] = ref.IGNORE
        size = np.exp2(rng.integers(-18, 1, T)) if uneven else 1.0
        self.dloss = (rng.standard_normal(T) * size).astype(np.float32).astype(float)
        self.dlse = (rng.standard_normal(T) * size).astype(np.float32).astype(float)
        tt = DTYPES[dt]
        self.X, self.W = self.strided(self.x, tt, pad), self.strided(self.w, tt, pad)
        self.Y = torch.from_numpy(self.labels).cuda()
        self.loss, self.lse = (torch.full((T,), float("nan"), device="cuda") for _ in range(2))
        self.dl, self.de = (torch.from_numpy(v).float().cuda() for v in (self.dloss, self.dlse))
        self.dx_buf = torch.full((T, D + pad), 9.0, dtype=tt, device="cuda")
        self.dw_buf = torch.full((V, D + pad), 9.0, dtype=tt, device="cuda")
        self.dX, self.dW = self.dx_buf[:, :D], self.dw_buf[:, :D]

    @staticmethod
    def strided(v, tt, pad):
        buf = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=tt, device="cuda")
        buf[:, :v.shape[1]] = torch.from_numpy(v).to(tt)
        return buf[:, :v.shape[1]]

    def forward(self, h, **kw):
        h.ce_forward(self.X, self.W, self.Y, self.loss, self.lse, alpha=self.alpha, **kw)

    def backward(self, h, dlse=True, **kw):
        h.ce_backward(self.X, self.W, self.Y, self.lse, self.dl, kw.pop("dX", self.dX),
                      kw.pop("dW", self.dW), dlse=self.de if dlse else None, alpha=self.alpha, **kw)

    def sum_error(self):
        return (self.V / 64 + 32) * U + 2.0 ** -14

    def check_forward(self):
        self.z, loss, lse = ref.forward(self.x, self.w, self.labels, self.alpha)
        keep = self.labels != ref.IGNORE
        z_label = self.z[np.arange(self.T), np.where(keep, self.labels, 0)]
        got_loss, got_lse = (t.double().cpu().numpy() for t in (self.loss, self.lse))
        tol = self.sum_error() + 4 * U * np.abs(lse)
        assert np.all(np.abs(got_lse - lse) <= tol), np.abs(got_lse - lse).max()
        assert np.all(np.abs(got_loss - loss) <= tol + U * (np.abs(loss) + np.abs(z_label)))
        assert np.all(got_loss[~keep] == 0) and np.all(got_lse[~keep] == 0)

    def check_backward(self, dlse=True):
        z, _, lse = ref.forward(self.x, self.w, self.labels, self.alpha)
        de = self.dlse if dlse else None
        dz = ref.dlogits(z, self.labels, lse, self.dloss, de)
        dx, dw = ref.gradients(self.x, self.w, self.labels, dz, self.alpha)
        half = torch.finfo(DTYPES[self.dt]).eps / 2
        keep = self.labels != ref.IGNORE
        p = np.where(keep, np.abs(self.dloss + (self.dlse if dlse else 0.0)), 0.0)[:, None] * np.exp(
            np.where(keep[:, None], z - lse[:, None], -np.inf))
        rel = 2 * self.sum_error() + 2.0 ** -18
        ez = rel * p + 4 * U * np.abs(dz)
        ez += (half if self.T > 128 else half * half) * (np.abs(dz) + ez)
        ax, aw = np.abs(np.where(keep[:, None], self.x, 0.0)), np.abs(self.w)
        low_x = low_w = 0.0
        if self.dt == "f16":
            r = np.where(keep, np.maximum(np.abs(self.dloss), np.abs(self.dloss + (
                self.dlse if dlse else 0.0))), 0.0)
            ez = ez + 2.0 ** -38 * 2 * r[:, None]
            # X * 2^(k-kmax), off by 2^-25 at most, against dz' < 2^15
            low_w = keep.sum() * 2.0 ** (15 - 25 - 13) * 2 * r.max(initial=0.0)
            low_x = low_w * 0 + 2.0 ** -25  # the result's own subnormal numbers
            low_w = low_w + 2.0 ** -25
        for got, want, err, mag in (
                (self.dX, dx, ez @ aw + low_x, 4 * max(self.V, 1) * U * (np.abs(dz) @ aw)),
                (self.dW, dw, ez.T @ ax + low_w, 4 * max(self.T, 1) * U * (np.abs(dz).T @ ax))):
            bound = self.alpha * (err + mag)
            if self.dt == "f16":
                bound = bound + 2.0 ** -25
            bound = bound + half * (np.abs(want) + bound) + 4 * U * np.abs(want)
            off = np.abs(got.double().cpu().numpy() - want)
            assert np.all(off <= bound), (np.nanmax(off - bound), np.argwhere(~(off <= bound))[:3])
        assert (self.dX[torch.from_numpy(~keep).cuda()] == 0).all()
        D = self.D
        assert (self.dx_buf[:, D:] == 9).all() and (self.dw_buf[:, D:] == 9).all()


SIZES = [(1, 1, 1), (1, 5, 3), (2, 300, 7), (3, 100, 16), (16, 257, 64), (17, 1000, 33), (64, 512, 128),
         (65, 2050, 100), (130, 5000, 257), (256, 1024, 256), (300, 777, 512), (513, 4099, 130),
         # packed rows: 128- and 256-square tiles, ragged and whole in every extent
         (20, 4096, 72), (129, 2048, 320), (257, 6401, 392), (300, 33001, 264), (260, 65536, 64),
         (520, 9001, 100), (600, 700, 1030)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,V,D", SIZES)
def test_loss_and_gradients(handle, T, V, D, dt):
    p = Problem(T, V, D, dt, pad=0 if T % 2 else 3)
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


FEW = [(4, 1, 1), (1, 131, 1030), (8, 700, 260), (9, 64, 257), (16, 5000, 515), (7, 40000, 4),
       (2, 20000, 300), (13, 63, 2), (8, 65, 9), (5, 12000, 96), (15, 129, 2050)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,V,D", FEW)
def test_few_rows(handle, T, V, D, dt):
    p = Problem(T, V, D, dt, seed=10, uneven=T % 2 == 1, pad=T % 4)
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()
    both = [t.clone() for t in (p.dX, p.dW)]
    p.dX.zero_(), p.dW.zero_()
    p.backward(handle, dW=None)
    p.backward(handle, dX=None)
    assert all(torch.equal(a, b) for a, b in zip(both, (p.dX, p.dW)))


# 32-bit operands in planes: tiles enough of z, and of dW but for the last two
# (forward in planes, backward over the library's products).
WIDE = [(520, 16500, 300), (1100, 8200, 600), (4200, 2100, 2000), (513, 13057, 257), (520, 16500, 16),
        (4097, 2048, 130)]


@pytest.mark.parametrize("T,V,D", WIDE)
def test_32_bit_loss_and_gradients_in_planes(T, V, D):
    p = Problem(T, V, D, "f32", pad=0 if T % 2 else 3)
    with sg.Handle(workspace=False) as h:
        h.set_workspace(max(h.ce_workspace_size(p.X, p.W, backward=b) for b in (False, True)))
        p.forward(h)
        p.check_forward()
        p.backward(h)
        p.check_backward()


@pytest.mark.parametrize("count", [0, 1, 127, 128, 129, 256, 257, 512, 600])
def test_32_bit_rows_that_count_at_tile_edges(handle, count):
    p = Problem(600, 13200, 264, "f32", seed=6, ignored=0.0)
    p.labels[np.random.default_rng(count).permutation(600)[count:]] = ref.IGNORE
    p.Y.copy_(torch.from_numpy(p.labels))
    p.X[p.Y == ref.IGNORE] = float("nan")
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("T,V,D", [(2100, 220, 1900), (700, 900, 500), (9000, 130, 70), (9000, 130, 1)])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_many_rows_few_words(handle, T, V, D, dt):
    p = Problem(T, V, D, dt, seed=9)
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


def test_more_rows_than_a_grid_extent_holds():
    p = Problem(70000, 130, 24, "f32", seed=7)
    with sg.Handle(workspace=False) as h:
        h.set_workspace(max(h.ce_workspace_size(p.X, p.W, backward=b) for b in (False, True)))
        p.forward(h)
        p.check_forward()
        p.backward(h)
        p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,V,D", [(5, 2050, 64), (16, 9000, 70), (8, 3000, 2), (130, 3000, 96), (300, 1111, 40),
                                   (550, 14000, 300)])
def test_least_workspace_takes_small_pieces(T, V, D, dt):
    p = Problem(T, V, D, dt, seed=1)
    with sg.Handle(workspace=False) as h:
        for backward in (False, True):
            least = h.ce_workspace_size(p.X, p.W, backward=backward, least=True)
            assert least <= h.ce_workspace_size(p.X, p.W, backward=backward)
            h.set_workspace(least - 64)
            with pytest.raises(sg.SgemmError) as e:
                (p.backward if backward else p.forward)(h)
            assert e.value.status == sg.SGEMM_ERR_SCRATCH
            h.set_workspace(least)
            guard = h.workspace.clone().fill_(float("nan"))
            h.workspace.copy_(guard)  # nothing in it is taken for a result
            (p.backward if backward else p.forward)(h)
        p.check_forward()
        p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
def test_full_workspace(dt):
    p = Problem(200, 9000, 72, dt, seed=2)
    with sg.Handle(workspace=False) as h:
        h.set_workspace(h.ce_workspace_size(p.X, p.W, backward=True))
        p.forward(h)
        p.check_forward()
        p.backward(h, dlse=False)
        p.check_backward(dlse=False)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T", [4, 90])
def test_uneven_upstream_gradients(handle, T, dt):
    """Rows whose gradients differ by 2^18: none vanishes, none overflows."""
    p = Problem(T, 600, 48, dt, seed=3, uneven=True)
    p.forward(handle)
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -60, 2.0 ** -14])
def test_gradients_of_lse_beside_small_ones_of_loss(handle, size, T, dt):
    p = Problem(T, 500, 40, dt, seed=9, ignored=0.1)
    p.dloss = (p.dloss * size).astype(np.float32).astype(float)
    p.dl.copy_(torch.from_numpy(p.dloss))
    p.forward(handle)
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** -14, 2.0 ** 10])
def test_half_gradients_keep_their_range(handle, scale):
    """binary16 dz neither vanishes nor overflows, whatever dloss' size: the
    gradients scale with it.  Each of the two results carries half a step:
    2^-11 of its value, and at most 2^-25 where it is one of binary16's
    subnormal numbers; the first one's is multiplied by the scale.  Together
    2^-10 |one * scale| + 2^-25 (1 + scale) and terms of second order."""
    p = Problem(20, 900, 64, "f16", seed=4)
    p.forward(handle)
    p.backward(handle)
    one = p.dX.double().cpu().numpy().copy()
    p.dl.mul_(scale)
    p.de.mul_(scale)
    p.backward(handle)
    got = p.dX.double().cpu().numpy()
    assert np.all(np.abs(got - one * scale) <=
                  1.01 * (2.0 ** -25 * (1 + scale) + 2.0 ** -10 * np.abs(one * scale)))


@pytest.mark.parametrize("size", [2.0 ** -20, 2.0 ** -13, 1.0, 2.0 ** 10])
@pytest.mark.parametrize("T", [60, 300])
def test_half_gradients_of_w_for_small_x_and_uneven_rows(handle, T, size):
    """binary16 dW keeps the terms of rows whose dloss is far below the largest,
    whatever X's size.  Beside dz's rounding and the result's, a row's X may
    lose, scaled for the product, half a step of the subnormal numbers, 2^-25,
    where the largest |dz x| of all rows is scaled to 2^28 or more: with r the
    row's largest |dz| and M the largest r max|x|, 2^-36 M |dz| / r at the
    most."""
    V, D, alpha = 700, 48, 0.5
    p = Problem(T, V, D, "f16", seed=8, ignored=0.1)
    rng = np.random.default_rng(T)
    weight = np.exp2(-rng.integers(0, 13, T).astype(float))
    p.dloss = (np.sign(p.dloss) * (1 + rng.random(T)) * weight).astype(np.float32).astype(float)
    # (results of about 2^-4 times the rows' weights)
    p.dloss *= 2.0 ** -4 / size
    p.x *= size
    p.alpha = alpha / size if size >= 1 else alpha
    p.w *= 1.0 if size >= 1 else 2.0 ** -6
    p.X, p.W = p.strided(p.x, torch.float16, 0), p.strided(p.w, torch.float16, 0)
    p.dl.copy_(torch.from_numpy(p.dloss))
    p.forward(handle)
    p.backward(handle, dlse=False)
    z, _, lse = ref.forward(p.x, p.w, p.labels, p.alpha)
    dz = ref.dlogits(z, p.labels, lse, p.dloss)
    _, want = ref.gradients(p.x, p.w, p.labels, dz, p.alpha)
    keep = p.labels != ref.IGNORE
    r = np.where(keep, np.abs(p.dloss), 0.0)
    ax = np.abs(np.where(keep[:, None], p.x, 0.0))
    half = 2.0 ** -11
    prob = r[:, None] * np.exp(np.where(keep[:, None], z - lse[:, None], -np.inf))
    e = (2 * p.sum_error() + 2.0 ** -18) * prob + 4 * U * np.abs(dz)
    e += (half if T > 128 else half * half) * (np.abs(dz) + e) + 2.0 ** -37 * r[:, None]
    big = (r * ax.max(1)).max()
    share = (np.abs(dz) / np.where(r > 0, r, 1.0)[:, None]).sum(0)
    bound = p.alpha * (e.T @ ax + 4 * T * U * (np.abs(dz).T @ ax) + 2.0 ** -36 * big * share[:, None])
    bound = bound + half * (np.abs(want) + bound) + 2.0 ** -25
    off = np.abs(p.dW.double().cpu().numpy() - want)
    assert np.all(off <= bound), (np.nanmax(off / bound), np.argwhere(~(off <= bound))[:3])


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T", [3, 70])
def test_left_out_rows_may_hold_anything(handle, T, dt):
    p = Problem(T, 400, 40, dt, seed=5, ignored=0.4)
    p.labels[0], p.labels[1] = ref.IGNORE, 7
    p.Y.copy_(torch.from_numpy(p.labels))
    out = p.Y == ref.IGNORE
    p.X[out] = float("nan")
    p.X[0, 0] = float("inf")
    p.dl[out] = float("nan")
    p.de[out] = float("inf")
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T", [1, 40, 200])
def test_every_row_left_out(handle, T, dt):
    p = Problem(T, 300, 24, dt, ignored=2.0)
    p.forward(handle)
    p.backward(handle)
    for t in (p.loss, p.lse, p.dX, p.dW):
        assert (t == 0).all()


def test_no_rows(handle):
    for tt in DTYPES.values():
        X, W = torch.empty(0, 24, dtype=tt, device="cuda"), torch.ones(30, 24, dtype=tt, device="cuda")
        Y, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
        dW = torch.full_like(W, 3.0)
        handle.ce_forward(X, W, Y, f, f.clone())
        handle.ce_backward(X, W, Y, f, f, torch.empty_like(X), dW)
        assert (dW == 0).all()


@pytest.mark.parametrize("dt", list(DTYPES))
def test_no_rows_need_no_workspace(dt):
    tt = DTYPES[dt]
    X, W = torch.empty(0, 24, dtype=tt, device="cuda"), torch.ones(30, 24, dtype=tt, device="cuda")
    Y, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    dW = torch.full_like(W, 3.0)
    with sg.Handle(workspace=False) as h:
        h.set_workspace(h.ce_workspace_size(X, W))
        h.ce_forward(X, W, Y, f, f.clone())
        h.set_workspace(h.ce_workspace_size(X, W, backward=True))
        h.ce_backward(X, W, Y, f, f, torch.empty_like(X), dW)
    assert (dW == 0).all()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("count", [0, 1, 127, 128, 255, 256, 257, 384, 512, 600])
def test_rows_that_count_at_tile_edges(handle, count, dt):
    p = Problem(600, 1300, 72, dt, seed=6, ignored=0.0)
    p.labels[np.random.default_rng(count).permutation(600)[count:]] = ref.IGNORE
    p.Y.copy_(torch.from_numpy(p.labels))
    p.X[p.Y == ref.IGNORE] = float("nan")
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T", [6, 200])
def test_no_read_past_the_operands(handle, T, dt):
    """X and W end where their buffers do not: NaNs stand behind the last
    element of W's and X's rows and after the last row."""
    V, D = 333, 40
    p = Problem(T, V, D, dt, seed=7)
    for name, rows in (("X", T), ("W", V)):
        t = getattr(p, name)
        buf = torch.full((rows * (D + 8) + 4096,), float("nan"), dtype=t.dtype, device="cuda")
        view = buf[:rows * (D + 8)].view(rows, D + 8)[:, :D]
        view.copy_(t)
        setattr(p, name, view)
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,V,D,pad", [(4, 300, 40, 100), (70, 1300, 72, 600), (300, 777, 64, 65),
                                       (530, 1000, 41, 300), (530, 14000, 290, 300)])
def test_rows_far_apart(handle, T, V, D, pad, dt):
    p = Problem(T, V, D, dt, seed=8, pad=pad)
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    p.check_backward()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,V", [(1, 50), (1, 5000), (3, 700), (33, 2000), (128, 3000), (129, 3000),
                                 (256, 3000), (900, 6000)])
def test_gradients_lose_no_more_than_their_rounding(handle, T, V, dt):
    """Error in the 2-norm against 64 bits: that of rounding the exact
    gradients, or, past 128 rows, sqrt(2) of it and a tenth (dz's rounding is
    another of the same size)."""
    D = 96
    rng = np.random.default_rng([T, V])
    tt = DTYPES[dt]
    W = torch.from_numpy(rng.standard_normal((V, D)) * 2 / D ** 0.5).to(tt).cuda()
    labels = rng.integers(0, V, T)
    w = W.double().cpu().numpy()
    X = torch.from_numpy(rng.standard_normal((T, D)) + 2 * rng.random((T, 1)) * w[labels]).to(tt).cuda()
    Y = torch.from_numpy(labels).cuda()
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dl = torch.full((T,), (1024.0 if dt == "f16" else 1.0) / (T + 0.37), device="cuda")
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    handle.ce_forward(X, W, Y, loss, lse)
    handle.ce_backward(X, W, Y, lse, dl, dX, dW)
    x = X.double().cpu().numpy()
    z, _, e = ref.forward(x, w, labels)
    want = ref.gradients(x, w, labels, ref.dlogits(z, labels, e, dl.double().cpu().numpy()))
    for got, g in zip((dX, dW), want):
        own = np.linalg.norm(torch.from_numpy(g).to(tt).double().numpy() - g)
        off = np.linalg.norm(got.double().cpu().numpy() - g)
        assert off <= (1.02 if T <= 128 else 1.1 * 2 ** 0.5) * own, (off, own)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("bad", [-1, 50, 2 ** 40])
def test_labels_out_of_range(handle, dt, bad):
    p = Problem(9, 50, 16, dt, ignored=0.0)
    p.Y[4] = bad
    p.forward(handle)
    assert torch.isnan(p.loss).nonzero().flatten().tolist() == [4]
    assert torch.isfinite(p.lse).all()
    p.backward(handle)
    assert torch.isnan(p.dX).all(1).nonzero().flatten().tolist() == [4]
    assert torch.isnan(p.dW).any()


def test_another_ignore_index(handle):
    p = Problem(30, 60, 16, "f32", ignored=0.3)
    p.Y[p.Y == ref.IGNORE] = 2 ** 35
    p.forward(handle, ignore_index=2 ** 35)
    p.check_forward()
    p.backward(handle, ignore_index=2 ** 35)
    p.check_backward()


@pytest.mark.parametrize("dt", list(DTYPES))
def test_one_gradient_alone(handle, dt):
    p = Problem(40, 700, 56, dt)
    p.forward(handle)
    p.backward(handle)
    dx, dw = p.dX.clone(), p.dW.clone()
    p.dX.fill_(9.0)
    p.dW.fill_(9.0)
    p.backward(handle, dW=None)
    assert torch.equal(p.dX, dx) and (p.dW == 9).all()
    p.dX.fill_(9.0)
    p.backward(handle, dX=None)
    assert torch.equal(p.dW, dw) and (p.dX == 9).all()
    p.backward(handle, dX=None, dW=None)


@pytest.mark.parametrize("T,V,D", [(3, 1000, 64), (70, 5000, 128), (300, 2000, 256)])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_large_logits(handle, T, V, D, dt):
    """Logits of some hundreds: no exponential may overflow, and rows whose
    label is certain lose nothing."""
    p = Problem(T, V, D, dt, alpha=32.0, ignored=0.1)
    z, loss, lse = ref.forward(p.x, p.w, p.labels, p.alpha)
    p.labels[::2] = np.where(p.labels[::2] == ref.IGNORE, ref.IGNORE, z[::2].argmax(1))
    p.Y.copy_(torch.from_numpy(p.labels))
    z, loss, lse = ref.forward(p.x, p.w, p.labels, p.alpha)
    p.forward(handle)
    # (every logit is a multiple of 4: the sum's terms are 1, e^-4, ...)
    tol = (V / 64 + 32) * U + 2.0 ** -14 + 4 * U * np.abs(z).max()
    assert np.all(np.abs(p.lse.double().cpu().numpy() - lse) <= tol)
    assert np.all(np.abs(p.loss.double().cpu().numpy() - loss) <= 2 * tol)
    p.backward(handle)
    assert torch.isfinite(p.dX).all() and torch.isfinite(p.dW).all()


@pytest.mark.parametrize("T,V,D", [(2, 999, 130), (40, 3000, 200), (200, 4000, 320)])
@pytest.mark.parametrize("dt", list(DTYPES))
def test_random_inputs(handle, T, V, D, dt):
    """Normal values: the logits' own rounding, at most 4 D u sum|x w|, comes on
    top of the bounds."""
    rng = np.random.default_rng([T, V])
    tt = DTYPES[dt]
    X = torch.from_numpy(rng.standard_normal((T, D))).to(tt).cuda()
    W = torch.from_numpy(rng.standard_normal((V, D)) * 2 / D ** 0.5).to(tt).cuda()
    labels = rng.integers(0, V, T)
    Y = torch.from_numpy(labels).cuda()
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    handle.ce_forward(X, W, Y, loss, lse)
    x, w = X.double().cpu().numpy(), W.double().cpu().numpy()
    z, want, want_lse = ref.forward(x, w, labels)
    ez = 4 * D * U * (np.abs(x) @ np.abs(w).T).max(1) + (V / 64 + 32) * U + 2.0 ** -14
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= ez + 4 * U * np.abs(want_lse))
    assert np.all(np.abs(loss.double().cpu().numpy() - want) <= 2 * ez)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T", [1, 10, 100, 520, 65536])
def test_small_losses_keep_their_bits(T, dt):
    """Labels that are nearly certain, logits of about 25 that are exact in any
    order: the loss log(1 + s) is off by s's own errors (2^-16 relative here:
    few words, |z - m| < 50), by the rounding of the sum 1 + s -- V additions of
    at most u each, in whatever order -- by the exponential of the largest term
    (v_exp_f32: one unit in the last place, 2 u), and by the logarithm and the
    steps that join the parts (at most 6 u), not by lse's own rounding."""
    V, D = 40, 64
    rng = np.random.default_rng(T)
    w = rng.integers(-1, 2, (V, D)).astype(float)
    labels = rng.integers(0, V, T)
    x = w[labels] * rng.choice([1.0, 1.5, 2.0], (T, 1)) / 4
    tt = DTYPES[dt]
    X, W = torch.from_numpy(x).to(tt).cuda(), torch.from_numpy(w).to(tt).cuda()
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    with sg.Handle(workspace=False) as h:
        h.set_workspace(h.ce_workspace_size(X, W))
        h.ce_forward(X, W, torch.from_numpy(labels).cuda(), loss, lse)
    _, want, _ = ref.forward(x, w, labels)
    assert want.max() < 0.1
    got = loss.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= 2.0 ** -15 * want + (V + 8) * U), np.abs(got - want).max()


@pytest.mark.parametrize("T", [1, 40, 520, 65536])
@pytest.mark.parametrize("D", [1, 2, 4])
def test_32_bit_logits_keep_24_bits(T, D):
    """One word: lse is the logit itself.  Operands with all 24 bits set: a
    product of 16 bits or 21 would miss the library's 32-bit bound, 4 D u
    sum|x w|, to which the logarithm's scale and back add 4 u |z|."""
    rng = np.random.default_rng([T, D])
    x, w = (1 + (rng.integers(0, 1 << 11, s) * 4096 + 2047) * 2.0 ** -23 for s in ((T, D), (1, D)))
    X, W = (torch.from_numpy(v).float().cuda() for v in (x, w))
    assert np.array_equal(X.double().cpu().numpy(), x)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    with sg.Handle(workspace=False) as h:
        h.set_workspace(h.ce_workspace_size(X, W))
        h.ce_forward(X, W, torch.zeros(T, dtype=torch.int64, device="cuda"), loss, lse)
    z = (x @ w.T)[:, 0]
    assert np.all(np.abs(lse.double().cpu().numpy() - z) <= (4 * D + 4) * U * z)
    assert np.all(np.abs(loss.double().cpu().numpy()) <= (4 * D + 8) * U * z)


def test_gradients_by_differences(handle):
    rng = np.random.default_rng(3)
    T, V, D = 20, 500, 32
    X = torch.from_numpy(rng.standard_normal((T, D))).float().cuda()
    W = torch.from_numpy(rng.standard_normal((V, D)) * 0.3).float().cuda()
    Y = torch.from_numpy(rng.integers(0, V, T)).cuda()
    loss, lse, dl = (torch.empty(T, device="cuda") for _ in range(3))
    dl.fill_(1.0)
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    handle.ce_forward(X, W, Y, loss, lse)
    handle.ce_backward(X, W, Y, lse, dl, dX, dW)
    for t, g in ((X, dX), (W, dW)):
        d = torch.from_numpy(rng.standard_normal(t.shape)).float().cuda()
        d /= d.norm()
        total = []
        for h in (2.0 ** -5, -2.0 ** -5):
            keep = t.clone()
            t += h * d
            handle.ce_forward(X, W, Y, loss, lse)
            total.append(loss.double().sum().item())
            t.copy_(keep)
        slope = (total[0] - total[1]) / 2.0 ** -4
        # third-order term of a unit direction (|z'''| under 8 here) and the
        # rounding of 20 losses of about 6
        assert abs(slope - (g.double() * d.double()).sum().item()) < 8 * 2.0 ** -10 + 20 * 64 * U * 16


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("T,V,D", [(1, 1500, 64), (40, 1500, 64), (300, 1500, 64), (600, 13200, 264)])
def test_same_bits_every_call_and_in_graphs(dt, T, V, D):
    """Two eager calls, and a captured one replayed with eager work of other
    sizes between on the same workspace: the same bits."""
    p = Problem(T, V, D, dt)
    with sg.Handle(workspace=False) as h, sg.Handle(workspace=False) as other:
        size = h.ce_workspace_size(p.X, p.W, backward=True)
        for each in (h, other):
            each.set_workspace(size)

        def work():
            p.forward(h)
            p.backward(h)

        outs = (p.loss, p.lse, p.dX, p.dW)
        work()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            work()
            torch.cuda.synchronize()
            with torch.cuda.graph(g, stream=s):
                work()
        torch.cuda.synchronize()
        q = Problem(33, 700, 48, dt)
        for _ in range(3):
            for t in outs:
                t.fill_(5.0)
            q.forward(h)
            q.backward(h)
            with torch.cuda.stream(s):  # another handle's work beside the replay
                q.forward(other)
            s.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("T", [5, 40, 300])
def test_past_32_bit_offsets(T):
    """W and dW of 2.2e9 elements (the reference's sums in 64 bits on the GPU,
    by pieces)."""
    V, D = 540000, 4096
    W = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(std=0.03)
    X = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_()
    Y = torch.randint(0, V, (T,), device="cuda")
    Y[0], Y[1], Y[2] = V - 1, 524288, ref.IGNORE
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dl = torch.full((T,), 0.5, device="cuda")
    dX, dW = torch.empty_like(X), torch.empty_like(W)
    with sg.Handle(workspace=False) as h:
        h.set_workspace(h.ce_workspace_size(X, W, backward=True))
        h.ce_forward(X, W, Y, loss, lse)
        h.ce_backward(X, W, Y, lse, dl, dX, dW)
    x = X.double()
    z = torch.cat([x @ w.double().t() for w in W.split(60000)], 1)
    want = torch.logsumexp(z, 1)
    keep = Y != ref.IGNORE
    # 4 D u sum|x w| of about 0.03 * 4096 * 0.64, and the sum's bound
    tol = 4 * D * U * 80 + (V / 64 + 32) * U + 2.0 ** -14
    assert ((lse.double() - want).abs()[keep] < tol).all() and lse[2] == 0 and loss[2] == 0
    assert ((loss.double() - (want - z.gather(1, Y.clamp(min=0)[:, None])[:, 0])).abs()[keep] < 2 * tol).all()
    dz = torch.exp(z - want[:, None])
    dz[torch.arange(T), Y.clamp(min=0)] -= 1
    dz *= 0.5 * keep[:, None]
    half = 2.0 ** -8
    at = torch.cat([Y[keep], torch.tensor([0, 1, 524287, 524289, V - 2], device="cuda")])
    for got, w, size in ((dW[at], dz[:, at].t() @ x, dz[:, at].abs().t() @ x.abs()),
                         (dX, sum(a @ b.double() for a, b in zip(dz.split(60000, 1), W.split(60000))),
                          sum(a.abs() @ b.double().abs() for a, b in zip(dz.split(60000, 1),
                                                                         W.split(60000))))):
        bound = half * w.abs() + (half + 2 * tol) * 1.01 * size
        assert ((got.double() - w).abs() <= bound).all()


def test_refusals(handle):
    p = Problem(6, 40, 16, "bf16")
    with pytest.raises(ValueError):
        handle.ce_forward(p.X, p.W, p.Y, p.loss[:5], p.lse)
    with pytest.raises(TypeError):
        handle.ce_forward(p.X, p.W, p.Y.int(), p.loss, p.lse)
    with pytest.raises(ValueError):
        handle.ce_forward(p.X, p.W, p.Y.cpu(), p.loss, p.lse)
    with pytest.raises(ValueError):
        handle.ce_backward(p.X, p.W, p.Y, p.lse, p.dl, p.dX.float(), p.dW)
    with pytest.raises(ValueError):
        handle.ce_backward(p.X, p.W, p.Y, p.lse, p.dl, p.dX, p.dW[:39])
    with pytest.raises(sg.SgemmError) as e:
        handle.ce_backward(p.X, p.W, p.Y, p.lse, p.dl, p.X, None)
    assert e.value.status == sg.SGEMM_ERR_ALIAS
    with sg.Handle(workspace=False) as bare, pytest.raises(sg.SgemmError) as e:
        p.forward(bare)
    assert e.value.status == sg.SGEMM_ERR_SCRATCH


@pytest.mark.parametrize("T", [1, 16, 100])
def test_quantised_layer_under_the_loss(handle, T):
    """The operators together: activations through a layer with 4-bit weights,
    the result through the output layer's loss, and back to the gradient of
    the layer's result."""
    rng = np.random.default_rng(T)
    K, D, V = 200, 96, 900
    x = rng.integers(-3, 4, (T, K)).astype(float)
    wq = handle.mx4_quantize(torch.from_numpy(rng.standard_normal((K, D))).bfloat16().cuda(), trans=True)
    X = torch.from_numpy(x).bfloat16().cuda()
    hidden = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    handle.gemm_mx4(X, wq, hidden, alpha=0.25)
    a = mx_reference.dequantize(*mx_reference.quantize(x))
    b = mx_reference.dequantize(wq.codes.cpu().numpy(), wq.scales.cpu().numpy())
    want, mag = mx_reference.product(0.25, a, b)
    half = torch.finfo(torch.bfloat16).eps / 2
    got = hidden.double().cpu().numpy()
    tol = 4 * wq.K * U * mag
    assert np.all(np.abs(got - want) <= tol + half * (np.abs(want) + tol))
    p = Problem(T, V, D, "bf16", ignored=0.0)
    p.x, p.X, p.alpha = got, hidden, 0.125
    p.forward(handle)
    z, loss, lse = ref.forward(got, p.w, p.labels, p.alpha)
    # hidden's 8 bits times W's 3 over 96 columns: the logits are exact
    p.check_forward()
    p.backward(handle)
    p.check_backward()
