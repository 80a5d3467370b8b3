"""Microscaled 4-bit operators without a GPU: the plain implementation against
hand-worked values, and every refusal of the C entries and the binding."""
import ctypes

import numpy as np
import pytest

import fp32_gemm_major_amd as sg
from tests import mx_reference as ref
from tests.test_ce_host import HostHandle

A, SA, B, SB, C = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x8000000  # never touched
F32, BF16, F16 = sg.SGEMM_DTYPE_F32, sg.SGEMM_DTYPE_BF16, sg.SGEMM_DTYPE_F16


def test_reference_by_hand():
    # largest 7 -> scale 2^0: the elements are the values themselves, rounded
    x = np.zeros((1, 32))
    x[0, :16] = [7, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5.5, -2.6, -0.3, 0.2, 6, 4, -7, -0.0]
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127]]
    got = ref.dequantize(codes, scales)[0, :16]
    assert got.tolist() == [6, 4, 4, 2, 2, 1, 1, 0, -6, -3, -0.5, 0, 6, 4, -6, 0]
    assert codes[0, 0] == (6 << 4 | 7) and codes[0, 7] == (8 << 4 | 15)
    # scales: 2^(floor(log2 a) - 2), at least 2^-127
    for a, s in ((1.0, 125), (0.999, 124), (8.0, 128), (2.0 ** -125, 0), (2.0 ** -149, 0),
                 (2.0 ** 127, 252), (0.0, 0)):
        assert ref.quantize(np.full((1, 3), a))[1].tolist() == [[s]], a
    assert ref.quantize(np.array([[np.inf, 1.0]]))[1].tolist() == [[255]]


def good(**kw):
    a = dict(M=4, N=5, K=64, A=A, lda=32, SA=SA, ldsa=2, B=B, ldb=32, SB=SB, ldsb=2, dtype=F32,
             C=C, ldc=5)
    a.update(kw)
    return sg.sgemm_validate_mx(*a.values())


def test_validate_product():
    assert good() == sg.SGEMM_OK
    assert good(dtype=BF16) == sg.SGEMM_OK and good(dtype=F16) == sg.SGEMM_OK
    for bad in (-1, 3, 4, 5):
        assert good(dtype=bad) == sg.SGEMM_ERR_VALUE
    for name in ("M", "N", "K"):
        assert good(**{name: -32}) == sg.SGEMM_ERR_SIZE
    assert good(K=63) == sg.SGEMM_ERR_SIZE
    assert good(K=sg.SGEMM_MX_MAX_K + 32, lda=1 << 30, ldb=1 << 30) == sg.SGEMM_ERR_SIZE
    for name in ("M", "N"):
        assert good(**{name: sg.SGEMM_MX_MAX_ROWS + 1}, ldc=2 ** 31 - 1) == sg.SGEMM_ERR_SIZE
    for name, short in (("lda", 31), ("ldsa", 1), ("ldb", 31), ("ldsb", 1), ("ldc", 4)):
        assert good(**{name: short}) == sg.SGEMM_ERR_LD, name
    for name in ("A", "SA", "B", "SB", "C"):
        assert good(**{name: None}) == sg.SGEMM_ERR_NULL, name
    assert good(A=None, SA=None, B=None, SB=None, K=0) == sg.SGEMM_OK
    assert good(M=0, A=None, C=None) == sg.SGEMM_OK
    assert good(C=C + 2) == sg.SGEMM_ERR_VALUE and good(C=C + 1, dtype=BF16) == sg.SGEMM_ERR_VALUE
    assert good(A=A + 1, SA=SA + 1, B=B + 3, SB=SB + 1) == sg.SGEMM_OK  # any byte address
    # the last four bytes of A's and of B's codes
    assert good(C=A + 32 * 3 + 28) == sg.SGEMM_ERR_ALIAS
    assert good(C=B + 32 * 4 + 28) == sg.SGEMM_ERR_ALIAS
    assert good(C=SA + 4) == sg.SGEMM_ERR_ALIAS and good(C=SB + 8) == sg.SGEMM_ERR_ALIAS


def test_null_handle():
    lib = sg.library()
    assert lib.sgemm_mx_quantize(None, F32, 0, 1, 32, A, 32, B, 16, C, 1, None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_mx_dequantize(None, F32, 1, 32, A, 16, B, 1, C, 32, None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_run_mx(None, 1, 1, 32, 1.0, A, 16, SA, 1, B, 16, SB, 1, 0.0, F32, C, 1,
                            None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_run_mx_quant(None, F32, 1, 1, 32, 1.0, A, 32, B, 16, SB, 1, 0.0, F32, C, 1,
                                  None) == sg.SGEMM_ERR_HANDLE


def test_sizes_that_a_launch_does_not_hold():
    """A launch's threads are counted in 32 bits: 2^24 workgroups of 256, each
    with 512 units of eight values (or 64 rows of 256 where X is stored across
    K).  Refused before anything touches the device; one less gets as far as
    that (and no further without one)."""
    h = HostHandle()
    lib, at = sg.library(), ctypes.addressof(h)
    X, codes, scales = 1 << 60, 1 << 52, 1 << 56  # never touched
    K = 1 << 20
    fits = ((1 << 24) - 1) * 512 * 8 // K  # rows of whole blocks

    def quantize(R, trans=0, k=K):
        return lib.sgemm_mx_quantize(at, BF16, trans, R, k, X, R if trans else k, codes, k // 2, scales,
                                     k // 32, None)

    def dequantize(R):
        return lib.sgemm_mx_dequantize(at, BF16, R, K, codes, K // 2, scales, K // 32, X, K, None)

    def product(R):
        return lib.sgemm_run_mx_quant(at, BF16, R, 1, K, 1.0, X, K, codes, K // 2, scales, K // 32, 0.0,
                                      F32, 1 << 48, 1, None)

    for call in (quantize, dequantize, product):
        assert call(fits + 1) == sg.SGEMM_ERR_UNSUPPORTED
        assert call(fits) == sg.SGEMM_ERR_DEVICE
    assert quantize(1 << 22, 1, 1 << 16) == sg.SGEMM_ERR_UNSUPPORTED
    assert quantize((1 << 22) - 64, 1, 1 << 16) == sg.SGEMM_ERR_DEVICE


def test_mx4_container():
    torch = pytest.importorskip("torch")
    u8 = dict(dtype=torch.uint8)
    q = sg.Mx4.empty(3, 65, "cpu")
    assert (q.rows, q.K, tuple(q.codes.shape), tuple(q.scales.shape)) == (3, 96, (3, 48), (3, 3))
    sg.Mx4(torch.zeros(3, 64, **u8)[:, :32], torch.zeros(3, 2, **u8))
    with pytest.raises(ValueError):
        sg.Mx4(torch.zeros(3, 32, **u8), torch.zeros(3, 3, **u8))
    with pytest.raises(ValueError):
        sg.Mx4(torch.zeros(3, 32, **u8), torch.zeros(4, 2, **u8))
    with pytest.raises(ValueError):
        sg.Mx4(torch.zeros(32, 3, **u8).t(), torch.zeros(3, 2, **u8))
    with pytest.raises(TypeError):
        sg.Mx4(torch.zeros(3, 32), torch.zeros(3, 2, **u8))


def test_matrix_checks():
    torch = pytest.importorskip("torch")
    assert sg._matrix("X", torch.zeros(3, 5, dtype=torch.bfloat16)) == (BF16, 5)
    assert sg._matrix("X", torch.zeros(3, 8)[:, :5]) == (F32, 8)
    for t in (torch.zeros(3, 5, dtype=torch.float64), torch.zeros(5)):
        with pytest.raises(TypeError):
            sg._matrix("X", t)
    for t in (torch.zeros(3, 5).t(), torch.zeros(1, 5).expand(3, 5)):
        with pytest.raises(ValueError):
            sg._matrix("X", t)


def test_sizes_and_strides_past_32_bits():
    """The C ABI's ints: what does not fit them is refused, not cut to its low
    32 bits (a stride of 2^32 + 64 would read as 64)."""
    torch = pytest.importorskip("torch")
    far = 2 ** 32 + 64
    strided = torch.empty_strided((2, 64), (far, 1), dtype=torch.bfloat16, device="meta")
    for t in (strided, torch.empty((2 ** 32 + 5, 1), device="meta"),
              torch.empty((1, 2 ** 32 + 5), device="meta"),
              torch.empty_strided((2, 4), (2 ** 31, 1), device="meta")):
        with pytest.raises(ValueError):
            sg._matrix("X", t)
    assert sg._matrix("X", torch.empty_strided((2, 4), (2 ** 31 - 1, 1), device="meta")) == (F32, 2 ** 31 - 1)
    # (one row has no stride to speak of)
    assert sg._matrix("X", torch.empty_strided((1, 64), (far, 1), device="meta")) == (F32, 64)
    u8 = dict(dtype=torch.uint8, device="meta")
    sg.Mx4(torch.empty((2, 32), **u8), torch.empty((2, 2), **u8))
    with pytest.raises(ValueError):
        sg.Mx4(torch.empty_strided((2, 32), (far, 1), **u8), torch.empty((2, 2), **u8))
    with pytest.raises(ValueError):
        sg.Mx4(torch.empty((2, 32), **u8), torch.empty_strided((2, 2), (far, 1), **u8))
    with pytest.raises(ValueError):
        sg.Mx4.empty(2 ** 32 + 5, 32, "meta")
    with pytest.raises(ValueError):
        sg._ce_shapes(strided, torch.empty((5, 64), dtype=torch.bfloat16, device="meta"))
    # the products of 32- and 16-bit operands, sizes given or taken from tensors
    A, B, C = (torch.empty((2, 2), device="meta") for _ in range(3))
    assert sg._shapes(A, B, C, None, None, None, None, None, None, False, False) == (2,) * 6
    one = torch.empty_strided((1, 2), (far, 1), device="meta")
    assert sg._shapes(one, B, one, None, None, None, None, None, None, False, False) == (1, 2, 2, 2, 2, 2)
    for name in ("M", "N", "K", "lda", "ldb", "ldc"):
        a = dict(M=None, N=None, K=None, lda=None, ldb=None, ldc=None) | {name: 2 ** 32 + 2}
        flat = (torch.empty(2 ** 35, device="meta") for _ in range(3))
        b = dict(M=2, N=2, K=2, lda=2, ldb=2, ldc=2) | {name: 2 ** 32 + 2}
        with pytest.raises(ValueError):
            sg._shapes(A, B, C, *a.values(), False, False)
        with pytest.raises(ValueError):
            sg._shapes(*flat, *b.values(), False, False)
