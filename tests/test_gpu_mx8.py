"""Microscaled 8-bit rows on the GPU against the plain 64-bit implementation
(mx8_reference): codes and scales have to be equal, bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests.test_gpu_mx import DTYPES, as_numpy, strided, values  # noqa: E402


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


SIZES = [(1, 1), (1, 32), (2, 31), (3, 33), (16, 4096), (64, 256), (65, 777), (130, 2050),
         (257, 64), (1000, 100)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("R,K", SIZES)
def test_quantize(handle, R, K, trans, dt):
    x = torch.from_numpy(values(R, K, 7 * R + K)).to(DTYPES[dt])
    codes, scales = ref.quantize(x.double().numpy())
    stored = x.t().contiguous() if trans else x
    for pad in (0, 5):
        X, _ = strided(stored, pad, fill=float("nan"))
        nb = scales.shape[1]
        cbuf = torch.full((R, 32 * nb + 3), 0xA5, dtype=torch.uint8, device="cuda")
        sbuf = torch.full((R, nb + 1), 0xA5, dtype=torch.uint8, device="cuda")
        q = sg.Mx8(cbuf[:, :32 * nb], sbuf[:, :nb])
        handle.mx8_quantize(X, trans=trans, out=q)
        c, s = as_numpy(q)
        assert np.array_equal(s, scales)
        assert np.array_equal(c, codes)
        assert (cbuf[:, 32 * nb:] == 0xA5).all() and (sbuf[:, nb:] == 0xA5).all()
        Y, ybuf = strided(torch.zeros(R, K, dtype=x.dtype), 3, fill=1.5)
        handle.mx8_dequantize(q, Y)
        want = ref.dequantize(codes, scales)[:, :K]
        assert np.array_equal(Y.double().cpu().numpy(), want)
        assert (ybuf[:, K:] == 1.5).all()


@pytest.mark.parametrize("trans", [False, True])
def test_quantize_special_values(handle, trans):
    rows = []
    tiny = 2.0 ** -149
    for amax in (0.0, tiny, 5 * tiny, 2.0 ** -127, 2.0 ** -126, 2.0 ** -119, 448 * 2.0 ** -127,
                 449 * 2.0 ** -127, 1.75, np.nextafter(np.float32(1.75), np.float32(2)), 2.0 ** 126,
                 3.4e38, np.inf, -np.inf, np.nan):
        r = np.zeros(96)
        r[:32] = amax
        # ties and near ties, normal and subnormal, in the middle block
        r[32:64] = np.resize([448, 432, 416, 15.5, 16.5, 1.0625, 1.1875, -1.0625, 2.0 ** -9, 2.0 ** -10,
                              -3 * 2.0 ** -10, 2.0 ** -6 - 2.0 ** -10, 2.0 ** -11, -0.0, 447.99, -431.99,
                              1.0624999, 1.0625001, 0.9375, 0.96875, 240], 32)
        r[64:] = np.linspace(-1, 1, 32) * (amax if np.isfinite(amax) else 1.0)
        r[70] = amax
        rows.append(r)
    x = np.stack(rows).astype(np.float32)
    codes, scales = ref.quantize(x.astype(np.float64))
    X = torch.from_numpy(x.T.copy() if trans else x).cuda()
    q = handle.mx8_quantize(X, trans=trans)
    c, s = as_numpy(q)
    assert np.array_equal(s, scales)
    assert np.array_equal(c, codes)
    Y = handle.mx8_dequantize(q, torch.empty(x.shape, device="cuda"))
    # (3.4e38 is 255.8 * 2^120, nearest 256 * 2^120 = 2^128: an infinity in 32 bits)
    with np.errstate(over="ignore"):
        want = ref.dequantize(codes, scales).astype(np.float32)
    assert np.array_equal(Y.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_dequantize_every_code(handle, dt):
    codes = np.arange(256, dtype=np.uint8).reshape(8, 32)
    scales = np.full((8, 1), 130, np.uint8)
    q = sg.Mx8(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())
    Y = handle.mx8_dequantize(q, torch.empty(8, 32, dtype=DTYPES[dt], device="cuda"))
    assert np.array_equal(Y.double().cpu().numpy(), ref.dequantize(codes, scales), equal_nan=True)


def test_dequantize_fewer_columns(handle):
    q = handle.mx8_quantize(torch.from_numpy(values(5, 96, 3)).float().cuda())
    full = ref.dequantize(*as_numpy(q))
    for K in (1, 8, 31, 33, 64, 95, 96):
        Y = handle.mx8_dequantize(q, torch.empty(5, K, device="cuda"))
        assert np.array_equal(Y.cpu().numpy(), full[:, :K])


def test_quantize_past_32_bit_offsets(handle):
    # the last rows start past 2^32 bytes
    R, K, ld = 70000, 40, 32771
    buf = torch.empty(R * ld, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((R, K), (ld, 1))
    X.copy_(torch.from_numpy(values(R, K, 5)))
    q = handle.mx8_quantize(X)
    at = torch.tensor([0, 1, 32767, 32768, 65537, R - 1])
    codes, scales = ref.quantize(X[at.cuda()].double().cpu().numpy())
    c, s = as_numpy(q)
    assert np.array_equal(c[at], codes) and np.array_equal(s[at], scales)
    Y = handle.mx8_dequantize(q, X)
    assert np.array_equal(Y[at.cuda()].double().cpu().numpy(), ref.dequantize(codes, scales)[:, :K])


def test_refusals_of_the_binding(handle):
    x = torch.zeros(4, 64, device="cuda")
    q8, q4 = handle.mx8_quantize(x), handle.mx4_quantize(x)
    with pytest.raises(TypeError):
        handle.mx8_quantize(x, out=q4)
    with pytest.raises(TypeError):
        handle.mx8_dequantize(q4, x)
    with pytest.raises(TypeError):
        handle.mx4_dequantize(q8, x)
    with pytest.raises(ValueError):
        handle.mx8_quantize(x, out=sg.Mx8.empty(5, 64))
    with pytest.raises(ValueError):
        handle.mx8_quantize(x.cpu())
    with pytest.raises(sg.SgemmError):
        handle.mx8_quantize(x, out=sg.Mx8(x.view(torch.uint8)[:, :64], q8.scales))
