"""The root-mean-square norm into 8-bit rows and its gradients on the GPU against
the plain 64-bit implementation (mx8_reference).

Rounding: a lane adds the squares of its values one after another (16 at most,
of longer rows 8 * ceil(D / 8192)) and the lanes' sums follow in about 20 steps,
so a sum is off by (terms + 20) * 2^-24 of its terms' magnitudes; a quotient, a
root and a product more take half a step of 2^-23 each.  y is therefore off by
`delta(D)` of itself before it is rounded to 8 bits, and a code by half of its
own step more: 2^-4 of the value, at least 2^-10 of the scale."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests.test_gpu_mx import DTYPES, as_numpy, strided  # noqa: E402

EPS = 1e-5


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


def delta(D):
    terms = max(16, 8 * -(-D // 8192))
    return (terms + 28) * 2.0 ** -24


def rows(T, D, seed, dt):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, D)) * np.exp2(rng.integers(-3, 4, (T, 1)))
    x *= np.where(rng.random(D) < 0.02, 10.0, 1.0)
    return torch.from_numpy(x).to(DTYPES[dt])


def check_rows(q, y, d):
    """8-bit rows against the float64 values y that are known to d * |y|."""
    codes, scales = as_numpy(q)
    T, D = y.shape
    nb = scales.shape[1]
    full = np.zeros((T, 32 * nb))
    full[:, :D] = y
    bad = ~np.isfinite(full.reshape(T, nb, 32)).all(-1)
    assert np.array_equal(scales == 255, bad)
    full.reshape(T, nb, 32)[bad] = 0
    amax = np.abs(full).reshape(T, nb, 32).max(-1)
    e = scales.astype(int) - 127
    ok = bad | ((e >= ref.exponent(amax * (1 - d))) & (e <= ref.exponent(amax * (1 + d))))
    assert ok.all()
    got = ref.dequantize(codes, np.where(bad, 0, scales).astype(np.uint8))
    scale = np.repeat(np.exp2(e.astype(float)), 32, axis=1)
    half = np.maximum(np.abs(full) * (1 + d) / 16, scale * 2.0 ** -10)
    worst = np.abs(got - full) - half - d * np.abs(full)
    worst.reshape(T, nb, 32)[bad] = -1
    assert (worst <= 0).all(), np.argwhere(worst > 0)[:3]
    assert (codes[:, D:] == 0).all()
    assert (codes.reshape(T, nb, 32)[bad] == 0).all()


def half_step(dt):
    return torch.finfo(DTYPES[dt]).eps / 2


WIDTHS = [1, 7, 31, 32, 33, 64, 500, 512, 513, 1000, 1024, 1025, 2048, 2050, 4096, 4100, 8192, 8195,
          16384, 16390, 40001]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("D", WIDTHS)
def test_norm(handle, D, dt):
    for T in (1, 5, 131) if D < 5000 else (1, 3):
        x, r = rows(T, D, D + T, dt), rows(T, D, D + T + 1, dt)
        g = (1 + 0.3 * torch.from_numpy(np.random.default_rng(D).standard_normal(D))).to(DTYPES[dt])
        for residual, pad, gt in ((True, 0, dt), (True, 3, "f32"), (False, 5, dt)):
            X, _ = strided(x, pad, fill=float("nan"))
            R, _ = strided(r, pad + 1, fill=float("nan"))
            H, hbuf = strided(torch.zeros_like(x), pad, fill=7.0)
            G = g.to(DTYPES[gt]).cuda()
            nb = -(-D // 32)
            cbuf = torch.full((T, 32 * nb + 3), 0xA5, dtype=torch.uint8, device="cuda")
            sbuf = torch.full((T, nb + 1), 0xA5, dtype=torch.uint8, device="cuda")
            q = sg.Mx8(cbuf[:, :32 * nb], sbuf[:, :nb])
            rstd = torch.zeros(T, device="cuda")
            out = handle.rmsnorm_mx8(X, G, residual=R if residual else None, H=H, rstd=rstd, eps=EPS,
                                     out=q)
            assert out is q
            h = (x.float() + r.float()).to(x.dtype) if residual else x
            assert torch.equal(H.cpu(), h)
            assert (hbuf[:, D:] == 7.0).all()
            y, s = ref.norm(h.double().numpy(), G.double().cpu().numpy(), EPS)
            assert np.all(np.abs(rstd.double().cpu().numpy() - s) <= delta(D) * s)
            check_rows(q, y, delta(D))
            assert (cbuf[:, 32 * nb:] == 0xA5).all() and (sbuf[:, nb:] == 0xA5).all()


@pytest.mark.parametrize("D", [40, 700, 1500, 5000, 17000])
def test_norm_in_place_and_without_outputs(handle, D):
    T = 9
    x, r = rows(T, D, 1, "bf16").cuda(), rows(T, D, 2, "bf16").cuda()
    G = torch.ones(D, device="cuda")
    H = torch.empty_like(x)
    q = handle.rmsnorm_mx8(x, G, residual=r, H=H)
    q0 = handle.rmsnorm_mx8(x, G, residual=r)
    assert torch.equal(q.codes, q0.codes) and torch.equal(q.scales, q0.scales)
    for into in ("X", "residual"):
        a, b = x.clone(), r.clone()
        q1 = handle.rmsnorm_mx8(a, G, residual=b, H=a if into == "X" else b)
        assert torch.equal(a if into == "X" else b, H)
        assert torch.equal(q.codes, q1.codes) and torch.equal(q.scales, q1.scales)


@pytest.mark.parametrize("D", [40, 700, 1500, 5000, 17000])
def test_norm_special_rows(handle, D):
    """Rows of zeros, of infinities and NaNs, of the largest values and of
    subnormal ones, beside ordinary ones that keep their results."""
    x = rows(8, D, 3, "f32")
    x[1] = 0
    x[2, D // 2] = float("inf")
    x[3, D - 1] = float("nan")
    x[4] = 2.0 ** -140
    x[5] = 3e38  # (its square leaves 32 bits; its rstd is a subnormal of 2^-149's steps)
    X, G = x.cuda(), torch.full((D,), 0.5, device="cuda")
    rstd = torch.empty(8, device="cuda")
    q = handle.rmsnorm_mx8(X, G, rstd=rstd, eps=EPS)
    s = rstd.cpu()
    assert abs(float(s[1]) * EPS ** 0.5 - 1) < 1e-6 and float(s[2]) == 0 and torch.isnan(s[3])
    assert abs(float(s[5]) * 3e38 - 1) < 2.0 ** -21
    y = handle.mx8_dequantize(q, torch.empty(8, D, device="cuda")).cpu()
    block = slice(D // 2 // 32 * 32, min(D, D // 2 // 32 * 32 + 32))
    assert (y[1] == 0).all() and torch.isnan(y[3]).all()
    assert torch.isnan(y[2, block]).all() and torch.nan_to_num(y[2]).abs().sum() == 0
    keep = [0, 4, 6, 7]
    want, _ = ref.norm(x[keep].double().numpy(), np.full(D, 0.5), EPS)
    check_rows(sg.Mx8(q.codes[keep], q.scales[keep]), want, delta(D))
    check_rows(sg.Mx8(q.codes[5:6], q.scales[5:6]), np.full((1, D), 0.5), 2.0 ** -21)
    # bfloat16's squares are added in 32 bits, eight at a time
    q = handle.rmsnorm_mx8(torch.full((1, D), 1e19, device="cuda").bfloat16(), G, rstd=rstd[:1])
    assert float(rstd[0]) == 0 and not q.codes.any()
    # eps 0: a row of zeros is 0 * inf
    q = handle.rmsnorm_mx8(X[:2], G, eps=0.0)
    assert (q.scales[1] == 255).all() and not (q.scales[0] == 255).any()


@pytest.mark.parametrize("T,D,dt", [(600, 1501, "f32"), (400, 2000, "f16"), (300, 4096, "f32"),
                                    (30, 20000, "f32")])
def test_codes_of_the_exact_norm(handle, T, D, dt):
    """Of 32-bit and binary16 rows every code is that of the norm in 64 bits: the
    factor and what the rounding of y leaves are kept to 2^-40 at least, and of a
    million values 1e6 * 8 / log(2) * 2 * 2^-40 = 2e-5 lie that near to a border of the
    codes' rounding, eight of which there are in a binade."""
    x, r, G = rows(T, D, 11, dt).cuda(), rows(T, D, 12, dt).cuda(), rows(1, D, 13, dt)[0].cuda()
    eps = float(np.float32(EPS))
    q = handle.rmsnorm_mx8(x, G, residual=r, eps=eps)
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, _ = ref.norm(f((x.float() + r.float()).to(x.dtype)), f(G), eps)
    for got, exact in zip(as_numpy(q), ref.quantize(want)):
        assert np.array_equal(got, exact)


def check_gradients(dx, dg, dy, h, g, rstd, dh, dt, gt, T, D):
    f = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    want, wg, size, gsize = ref.norm_gradients(f(dy), f(h), f(g), f(rstd), f(dh))
    bound = (delta(D) + 8 * 2.0 ** -24) * size
    if dt != "f32":
        bound = bound + half_step(dt) * (np.abs(want) + bound) + (2.0 ** -25 if dt == "f16" else 0)
    err = np.abs(f(dx) - want)
    assert (err <= bound).all(), np.argwhere(err > bound)[:3]
    if dg is not None:
        bound = (T + 24) * 2.0 ** -24 * gsize
        if gt != "f32":
            bound = bound + half_step(gt) * (np.abs(wg) + bound) + (2.0 ** -25 if gt == "f16" else 0)
        assert (np.abs(f(dg) - wg) <= bound).all()


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("D", WIDTHS)
def test_backward(handle, D, dt):
    for T in (1, 5, 1301) if D < 1100 else (1, 3, 530) if D < 5000 else (1, 7):
        h, dy, dh = rows(T, D, D, dt), rows(T, D, D + 1, dt), rows(T, D, D + 2, dt)
        rstd = torch.from_numpy(ref.norm(h.double().numpy(), np.ones(D), EPS)[1]).float().cuda()
        for stream, pad, gt, gain in ((True, 0, dt, True), (False, 3, "f32", True), (True, 1, dt, False)):
            g = (1 + 0.3 * torch.from_numpy(np.random.default_rng(D).standard_normal(D)))
            G = g.to(DTYPES[gt]).cuda()
            H, _ = strided(h, pad, fill=float("nan"))
            dY, _ = strided(dy, pad + 2, fill=float("nan"))
            dH = strided(dh, pad, fill=float("nan"))[0] if stream else None
            dX, xbuf = strided(torch.zeros_like(h), pad, fill=7.0)
            dG = torch.full_like(G, float("nan")) if gain else None
            handle.rmsnorm_backward(dY, H, G, rstd, dX, dG=dG, dH=dH)
            check_gradients(dX, dG, dY, H, G, rstd, dH, dt, gt, T, D)
            assert (xbuf[:, D:] == 7.0).all()
            if stream and pad == 0:  # in place
                for name in ("dY", "dH"):
                    a, b = dY.clone(), dH.clone()
                    to = a if name == "dY" else b
                    handle.rmsnorm_backward(a, H, G, rstd, to, dG=dG, dH=b)
                    assert torch.equal(to, dX)


def test_backward_workspace(handle):
    """Any workspace from the least on gives dG; less is refused; without dG
    none is needed; the same workspace gives the same bits."""
    T, D = 700, 900
    h, dy = rows(T, D, 1, "f32").cuda(), rows(T, D, 2, "f32").cuda()
    G = torch.ones(D, device="cuda")
    rstd = torch.full((T,), 0.1, device="cuda")
    least, full = sg.sgemm_rmsnorm_workspace_size(handle.h, T, D)
    assert handle.rmsnorm_workspace_size(T, D, least=True) == least < full
    with sg.Handle(workspace=False) as own:
        dX, dG = torch.empty_like(h), torch.empty_like(G)
        own.rmsnorm_backward(dy, h, G, rstd, dX)
        with pytest.raises(sg.SgemmError) as e:
            own.rmsnorm_backward(dy, h, G, rstd, dX, dG=dG)
        assert e.value.status == sg.SGEMM_ERR_SCRATCH
        own.set_workspace(least - 4)
        with pytest.raises(sg.SgemmError):
            own.rmsnorm_backward(dy, h, G, rstd, dX, dG=dG)
        for size in (least, 3 * least + 8, full, 2 * full):
            own.set_workspace(size)
            runs = []
            for _ in range(2):
                dG.fill_(float("nan"))
                own.rmsnorm_backward(dy, h, G, rstd, dX, dG=dG)
                check_gradients(dX, dG, dy, h, G, rstd, None, "f32", "f32", T, D)
                runs.append(dG.clone())
            assert torch.equal(*runs)


def test_empty(handle):
    X, G = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    q = handle.rmsnorm_mx8(X, G)
    assert q.rows == 0 and q.K == 64
    dG = torch.full_like(G, 3.0)
    handle.rmsnorm_backward(X, X.clone(), G, torch.empty(0, device="cuda"), X.clone(), dG=dG)
    assert (dG == 0).all()


def test_past_32_bit_offsets(handle):
    # the last rows start past 2^32 bytes
    T, D, ld = 40000, 100, 65537
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((T, D), (ld, 1))
    X.copy_(rows(T, D, 8, "bf16"))
    small = X.contiguous()
    G = torch.ones(D, device="cuda")
    rstd, rstd2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    a, b = handle.rmsnorm_mx8(X, G, H=X, rstd=rstd), handle.rmsnorm_mx8(small, G, rstd=rstd2)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) and torch.equal(rstd, rstd2)
    dX = torch.empty_like(small)
    handle.rmsnorm_backward(small, small, G, rstd, dX)
    handle.rmsnorm_backward(X, small, G, rstd, X)
    assert torch.equal(X, dX)


def test_side_stream_and_graph(handle):
    """On another stream than the current one, and captured into a graph that is
    replayed on other inputs."""
    T, D = 300, 1500
    x, r = rows(T, D, 1, "bf16").cuda(), rows(T, D, 2, "bf16").cuda()
    dy = rows(T, D, 3, "bf16").cuda()
    G = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    H, dX, dG = torch.empty_like(x), torch.empty_like(x), torch.empty_like(G)
    rstd, q = torch.empty(T, device="cuda"), sg.Mx8.empty(T, D)

    def step(stream=None):
        handle.rmsnorm_mx8(x, G, residual=r, H=H, rstd=rstd, out=q, stream=stream)
        handle.rmsnorm_backward(dy, H, G, rstd, dX, dG=dG, dH=dy, stream=stream)

    def results():
        return [t.clone() for t in (H, dX, dG, rstd, q.codes, q.scales)]

    step()
    want = results()
    for t in (H, dX, dG, rstd, q.codes, q.scales):
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (5, 6, 7):
        x.copy_(rows(T, D, seed, "bf16"))
        dy.copy_(rows(T, D, seed + 10, "bf16"))
        graph.replay()
        got = results()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, results()))


def test_refusals_of_the_binding(handle):
    x = torch.zeros(4, 64, device="cuda")
    G, rstd = torch.ones(64, device="cuda"), torch.ones(4, device="cuda")
    with pytest.raises(ValueError):
        handle.rmsnorm_mx8(x, G, residual=x.bfloat16())
    with pytest.raises(ValueError):
        handle.rmsnorm_mx8(x, G, H=x[:3])
    with pytest.raises(TypeError):
        handle.rmsnorm_mx8(x, G.half())
    with pytest.raises(TypeError):
        handle.rmsnorm_mx8(x, G, out=sg.Mx4.empty(4, 64))
    with pytest.raises(ValueError):
        handle.rmsnorm_mx8(x, G, rstd=rstd[:3])
    with pytest.raises(ValueError):
        handle.rmsnorm_mx8(x, G.cpu())
    with pytest.raises(sg.SgemmError):
        handle.rmsnorm_mx8(x[:2], G, H=x[1:3])
    with pytest.raises(ValueError):
        handle.rmsnorm_backward(x, x, G, rstd, x[:, :32])
    with pytest.raises(TypeError):
        handle.rmsnorm_backward(x, x.clone(), G, rstd, x, dG=G.half())
    with pytest.raises(sg.SgemmError):
        handle.rmsnorm_backward(x, x, G, rstd, x)  # (dX over H)
