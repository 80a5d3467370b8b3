"""8-bit rows at the ends of their scales' range, in products and weight gradients,
against the plain 64-bit implementation."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests import test_gpu_mx8_products as products  # noqa: E402
from tests.test_gpu_mx import DTYPES  # noqa: E402


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


SIZES = [(2, 40, 544), (16, 70, 1024), (60, 70, 1056), (200, 300, 608), (700, 900, 352), (2900, 3050, 288)]


def small_codes(rng, q):
    """Codes of random values of at most 1 into q (E4M3 up to 0x38, E2M1 up to 2)."""
    if isinstance(q, sg.Mx8):
        c = rng.integers(0, 0x39, q.codes.shape) | 128 * rng.integers(0, 2, q.codes.shape)
    else:
        lo, hi = (rng.integers(0, 3, q.codes.shape) | 8 * rng.integers(0, 2, q.codes.shape) for _ in range(2))
        c = lo | hi << 4
    q.codes.copy_(torch.from_numpy(c.astype(np.uint8)))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("sa,sb", [(254, 0), (0, 254), (250, 10), (3, 249), (242, 127), (127, 24)])
def test_products_of_far_scales(handle, M, N, K, sa, sb, bits):
    """Scales at the ends of their range in operands whose products are inside of 32
    bits' (2^117 at most, 2^-123 at least), which alpha, a power of two, takes back to
    about 1.  Neighbouring blocks differ by a factor of two or four, so that each meets its
    own scale."""
    rng = np.random.default_rng(K)
    A, B = products.operand(M, K, 1), products.operand(N, K, 2, bits)
    for q, s in ((A, sa), (B, sb)):
        small_codes(rng, q)
        q.scales.copy_(torch.from_numpy(np.clip(s + rng.integers(-1, 2, q.scales.shape), 0, 254).astype(np.uint8)))
    back = 2.0 ** (254 - sa - sb)
    C = torch.empty(M, N, device="cuda")
    handle.gemm_mx8(A, B, C, alpha=back)
    products.check(C, products.numbers(A), products.numbers(B), back, 0.0, None, "f32", (sa, sb))


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_products_past_32_bits(handle, M, N, K, bits):
    """Sums over 2^128 are infinities, below 2^-150 (45: at most K * 2^-164) they are 0."""
    A, B = products.operand(M, K, 1), products.operand(N, K, 2, bits)
    A.codes.fill_(0x38)  # 1
    B.codes.fill_(0x38 if bits == 8 else 0x22)
    C = torch.empty(M, N, device="cuda")
    for s, want in ((254, float("inf")), (200, float("inf")), (45, 0.0), (0, 0.0)):
        A.scales.fill_(s)
        B.scales.fill_(s)
        for sign in (1, -1):
            A.codes.fill_(0x38 if sign > 0 else 0xB8)
            handle.gemm_mx8(A, B, C)
            assert (C == sign * want).all(), s


def one_token_each(T, D, codes, scales):
    """X whose token t has `codes` everywhere with scale scales[t]."""
    X = sg.Mx8.empty(T, D)
    X.codes.copy_(torch.from_numpy(np.resize(codes, (T, X.K)).astype(np.uint8)))
    X.scales.copy_(torch.from_numpy(np.repeat(np.asarray(scales, np.uint8)[:, None], X.K // 32, 1)))
    return X


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [8, 64, 100])
@pytest.mark.parametrize("N,D", [(8, 40), (130, 256), (3600, 3600)])
def test_weight_grad_takes_x_in_the_type_of_dy(handle, T, N, D, dt):
    """X's values are what dY's type makes of them, to nearest: infinities from 65520 on
    in binary16 (8-bit rows hold 61440 and 65536 next to one another) and from 2^128 on in
    bfloat16, multiples of 2^-24 below binary16's 2^-14 and of 2^-133 below bfloat16's
    2^-126."""
    codes = np.arange(256)
    codes = codes[codes % 128 != 127][:D] if D < 254 else codes[codes % 128 != 127]
    far = [127, 134, 133, 135, 111, 112, 110, 120] if dt == "f16" else [127, 254, 0, 1, 2, 246, 250, 5]
    X = one_token_each(T, D, codes, [127] * (T - 8) + far)
    x = ref.dequantize(X.codes.cpu().numpy(), X.scales.cpu().numpy())[:, :D]
    with np.errstate(over="ignore"):  # (32 bits hold what is not past them)
        x = torch.from_numpy(x.astype(np.float32)).to(DTYPES[dt]).double().numpy()
    for t in range(T - 8, T):
        # row n of dW sees one token, or none
        dy = torch.zeros(T, N)
        dy[t, 0] = 1.0
        dy[t, N - 1] = -2.0
        # (a token whose dY is 0 meets its infinities too: those columns are left out)
        others = np.isfinite(np.delete(x, t, 0)).all(0)
        assert others.sum() > D // 4
        dW = torch.empty(N, D, device="cuda")
        handle.mx8_weight_grad(dy.to(DTYPES[dt]).cuda(), X, dW)
        got = dW.double().cpu().numpy()
        assert np.array_equal(got[0][others], x[t][others])
        with np.errstate(over="ignore"):
            want = (-2 * x[t]).astype(np.float32)
        assert np.array_equal(got[N - 1][others], want[others])


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 2048, 4096), (300, 2048, 4096), (2048, 2176, 4096)])
def test_sums_of_hidden_states(handle, M, N, K, bits):
    """Unit-normal activations, a channel in 64 ten times as large: 32-bit results are off
    the 64-bit product by about 2^-15 of its norm, the matrix instruction's own sums
    (2^-14 allowed); 16-bit results by that and their rounding, which are independent of one
    another, so that their squares add up (a tenth is allowed for the sample).  The same
    call gives the same bits."""
    g = torch.Generator(device="cuda").manual_seed(K + M)
    x = torch.randn(M, K, generator=g, device="cuda")
    x = torch.where(torch.rand(K, generator=g, device="cuda") < 1 / 64, 10 * x, x)
    A = handle.mx8_quantize(x)
    w = torch.randn(N, K, generator=g, device="cuda")
    B = (handle.mx8_quantize if bits == 8 else handle.mx4_quantize)(w)
    want = torch.from_numpy(products.numbers(A)) @ torch.from_numpy(products.numbers(B)).T
    size = float(want.norm())
    C = torch.empty(M, N, device="cuda")
    handle.gemm_mx8(A, B, C)
    assert float((C.double().cpu() - want).norm()) <= 2.0 ** -14 * size
    for dt in (torch.bfloat16, torch.float16):
        rounding = float((want.to(dt).double() - want).norm())
        C = torch.empty(M, N, device="cuda", dtype=dt)
        again = torch.empty_like(C)
        handle.gemm_mx8(A, B, C)
        handle.gemm_mx8(A, B, again)
        off = float((C.double().cpu() - want).norm())
        assert off ** 2 <= 1.1 * (rounding ** 2 + (2.0 ** -14 * size) ** 2)
        assert torch.equal(C, again)
