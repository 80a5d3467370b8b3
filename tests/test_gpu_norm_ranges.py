"""The norm's results over its types' whole ranges, against 64 bits.

The forward norm's factor is the 64-bit root of a sum of squares in 64 bits, rounded
to 32: off by half a step, 2^-24 of itself (and a hair for the 64-bit steps)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests.test_gpu_mx import DTYPES, as_numpy  # noqa: E402
from tests.test_gpu_norm import rows  # noqa: E402

EPS = float(np.float32(1e-5))
HAIR = 1 + 2.0 ** -18


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


def f64(t):
    return t.double().cpu().numpy()


def power_of_two(n):
    return ((n.long() + 1023) << 52).view(torch.float64)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("D", [1, 33, 500, 1000, 2048, 4100, 8192, 16390])
def test_rstd_is_rounded_once(handle, D, dt):
    T = 40
    x, r = rows(T, D, D, dt), rows(T, D, D + 1, dt)
    rstd = torch.empty(T, device="cuda")
    handle.rmsnorm_mx8(x.cuda(), torch.ones(D, device="cuda"), residual=r.cuda(), rstd=rstd, eps=EPS)
    h = (x.float() + r.float()).to(x.dtype).double().numpy()
    s = ref.norm(h, np.ones(D), EPS)[1]
    assert np.all(np.abs(f64(rstd) - s) <= 2.0 ** -24 * HAIR * s)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 1000, 17000])
def test_results_past_32_bits_leave_no_codes(handle, D, dt):
    """A gain that takes y past the largest 32-bit value makes an infinity of it, and
    so no number of its block: the scale is 255 and the codes are 0, as the rows'
    format has it.  The other blocks keep their results."""
    T = 6
    x = rows(T, D, D, dt)
    x[:, 40] = 4 * x.abs().amax(1)  # past its neighbours in every row: over the norm
    G = (1 + 0.3 * torch.from_numpy(np.random.default_rng(D).standard_normal(D))).float()
    for sign in (1, -1):
        G[40] = sign * 3.4e38
        q = handle.rmsnorm_mx8(x.cuda(), G.cuda(), eps=EPS)
        codes, scales = as_numpy(q)
        y, _ = ref.norm(x.double().numpy(), G.double().numpy(), EPS)
        assert (np.abs(y[:, 40]) > 2.0 ** 128 * 1.01).all()
        assert (scales[:, 1] == 255).all() and (codes[:, 32:64] == 0).all()
        y[:, 40] = np.inf
        want = ref.quantize(y)
        assert np.array_equal(scales == 255, want[1] == 255)
        if dt == "f32":
            assert np.array_equal(codes, want[0]) and np.array_equal(scales, want[1])


@pytest.mark.parametrize("dt,power", [(dt, p) for p in (-110, -100, -75, -65, -60, -40, 20, 50)
                                      for dt in ("f32", "bf16")] + [("f32", 75), ("f32", 110)])
@pytest.mark.parametrize("D", [40, 1000, 17000])
def test_scale_of_a_row_does_not_matter(handle, D, power, dt):
    """Without eps the norm of a row times a power of two is the row's norm, down to
    rows whose squares are far below 32 bits' smallest (and up to where bfloat16 rows'
    leave 32 bits, 32-bit ones' far past that)."""
    T = 5
    x = rows(T, D, 3, dt)
    x = torch.where(x.abs() < 2.0 ** -10, torch.ones_like(x), x)  # (no subnormal ones in any power)
    G = (1 + 0.3 * torch.from_numpy(np.random.default_rng(D).standard_normal(D))).float().cuda()
    one, far = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y, s = ref.norm(x.double().numpy(), f64(G), 0.0)
    scaled = (x.double() * 2.0 ** power).to(x.dtype)
    assert torch.equal(scaled.double(), x.double() * 2.0 ** power)
    a = handle.rmsnorm_mx8(x.cuda(), G, rstd=one, eps=0.0)
    b = handle.rmsnorm_mx8(scaled.cuda(), G, rstd=far, eps=0.0)
    assert np.all(np.abs(f64(far) * 2.0 ** power - s) <= 2.0 ** -24 * HAIR * s)
    low, high = (ref.dequantize(*ref.quantize(y * (1 + e))) for e in (-2.0 ** -40, 2.0 ** -40))
    for q in (a, b):
        got = ref.dequantize(*as_numpy(q))[:, :D]
        lo, hi = low[:, :D], high[:, :D]
        assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi)))


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("seed,channels", [(1, 0.0), (2, 1 / 64), (3, 1 / 64)])
def test_every_code_is_the_exact_norms(handle, seed, channels, dt):
    """Of 33 million values, with a channel in 64 ten times as large or none: y is kept to
    2^-40 of itself, and 33e6 * 8 / log(2) * 2 * 2^-40 = 7e-4 values lie that near to a
    border of the codes' rounding, eight of which there are in a binade."""
    T, D, part = 8192, 4096, 1024
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, r = (torch.randn(T, D, generator=g, device="cuda") for _ in range(2))
    r = torch.where(torch.rand(D, generator=g, device="cuda") < channels, 10 * r, r)
    x, r = (0.5 * x).to(DTYPES[dt]), r.to(DTYPES[dt])
    G = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(DTYPES[dt])
    H = torch.empty_like(x)
    q = handle.rmsnorm_mx8(x, G, residual=r, H=H, eps=EPS)
    got = handle.mx8_dequantize(q, torch.empty(T, D, device="cuda"))
    off = 0
    for t in range(0, T, part):
        v = H[t:t + part].double()
        y = (v / ((v * v).sum(1, keepdim=True) / D + EPS).sqrt() * G.double()).reshape(part, -1, 32)
        m, e = torch.frexp(y.abs().amax(-1, keepdim=True) / 448.0)
        scale = power_of_two(torch.where(m > 0.5, e, e - 1))
        a = y / scale
        unit = power_of_two(torch.frexp(a)[1].sub(1).clamp(min=-6) - 3)
        want = (torch.round(a / unit) * unit * scale).reshape(part, D)
        off += int((want != got[t:t + part].double()).sum())
    assert off == 0


@pytest.mark.parametrize("D,per", [(8, 4), (520, 2), (1032, 1)])
def test_more_rows_than_workgroups(handle, D, per):
    """2^21 workgroups of `per` rows at most: the ones behind them take a second turn
    of the same workgroups, with the results that they have by themselves."""
    T = per * 2 ** 21 + 3001
    g = torch.Generator(device="cuda").manual_seed(D)
    X = torch.empty(T, D, device="cuda", dtype=torch.bfloat16).normal_(generator=g)
    G = torch.ones(D, device="cuda")
    rstd, own = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    q = handle.rmsnorm_mx8(X, G, rstd=rstd)
    for t in range(0, T, 2 ** 20):
        p = handle.rmsnorm_mx8(X[t:t + 2 ** 20], G, rstd=own[t:t + 2 ** 20])
        assert torch.equal(q.codes[t:t + 2 ** 20], p.codes), t
        assert torch.equal(q.scales[t:t + 2 ** 20], p.scales), t
    assert torch.equal(rstd, own)
