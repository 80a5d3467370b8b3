"""The norm's results over its types' whole ranges, against 64 bits.

The forward norm's factor is the 64-bit root of a sum of squares in 64 bits, rounded
to 32: off by half a step, 2^-24 of itself.  bfloat16 rows add the squares of eight
neighbours in 32 bits first: the first is exact, the seven additions that follow are
off by 2^-24 of their sum each, so the row's sum by 7 * 2^-24 and its root by half of
that.  (A hair more for the products of these errors.)"""
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


def root_error(dt):
    return (3.5 if dt == "bf16" else 0) * 2.0 ** -24 * HAIR


def f64(t):
    return t.double().cpu().numpy()


def power_of_two(n):
    return ((n.long() + 1023) << 52).view(torch.float64)


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
    assert np.all(np.abs(f64(far) * 2.0 ** power - s) <= (root_error(dt) + 2.0 ** -24) * HAIR * s)
    d = root_error(dt) * HAIR + 2.0 ** -40
    low, high = (ref.dequantize(*ref.quantize(y * (1 + e))) for e in (-d, d))
    for q in (a, b):
        got = ref.dequantize(*as_numpy(q))[:, :D]
        lo, hi = low[:, :D], high[:, :D]
        assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi)))


def test_codes_of_bfloat16_rows(handle):
    """Of 33 million values hardly a code differs from the 64-bit norm's.  A lane's sum
    of eight squares is off by sqrt(7) / sqrt(12) * 2^-24 or so, a row's mean of 512 of them
    by 1/22 of that and the root by half of it: 1e-9.  A value's code then tips over
    with a chance of 8 / log(2) * 1e-9 (eight borders of the codes' rounding in a binade):
    0.4 of 33 million, more than four with a chance of 1e-4.  One rounding of y to 32 bits
    would be 3e-8 off, and ten codes."""
    T, D, part = 8192, 4096, 1024
    g = torch.Generator(device="cuda").manual_seed(5)
    x, r = (torch.randn(T, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    G = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16()
    q = handle.rmsnorm_mx8(x, G, residual=r, eps=EPS)
    got = handle.mx8_dequantize(q, torch.empty(T, D, device="cuda"))
    h = (x.float() + r.float()).bfloat16()
    off = 0
    for t in range(0, T, part):
        v = h[t:t + part].double()
        y = (v / ((v * v).sum(1, keepdim=True) / D + EPS).sqrt() * G.double()).reshape(part, -1, 32)
        m, e = torch.frexp(y.abs().amax(-1, keepdim=True) / 448.0)
        scale = power_of_two(torch.where(m > 0.5, e, e - 1))
        a = y / scale
        unit = power_of_two(torch.frexp(a)[1].sub(1).clamp(min=-6) - 3)
        want = (torch.round(a / unit) * unit * scale).reshape(part, D)
        off += int((want != got[t:t + part].double()).sum())
    assert off <= 4


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
