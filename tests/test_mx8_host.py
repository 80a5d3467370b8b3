"""Microscaled 8-bit rows and the norm without a GPU: the plain implementation
against hand-worked values and differences, and every refusal of the C entries
and the binding."""
import ctypes

import numpy as np
import pytest

import fp32_gemm_major_amd as sg
from tests import mx8_reference as ref
from tests.test_ce_host import HostHandle

F32, BF16, F16 = sg.SGEMM_DTYPE_F32, sg.SGEMM_DTYPE_BF16, sg.SGEMM_DTYPE_F16
X, R, G, H = 0x10000000, 0x20000000, 0x30000000, 0x40000000  # never touched
CODES, SCALES, RSTD = 0x50000000, 0x60000000, 0x70000000
DY, DH, DX, DG = 0x80000000, 0x90000000, 0xA0000000, 0xB0000000


def test_reference_by_hand():
    x = np.zeros((1, 32))
    # largest 448: scale 2^0, the elements are the values themselves, rounded
    x[0, :12] = [448, 432, 416, -17, 15.5, 1.0625, 1.1875, 2 ** -9, 2 ** -10, 3 * 2 ** -10, -0.0, 240]
    codes, scales = ref.quantize(x)
    assert scales.tolist() == [[127]]
    got = ref.dequantize(codes, scales)[0, :12]
    assert got.tolist() == [448, 448, 416, -16, 16, 1, 1.25, 2 ** -9, 0, 2 ** -8, 0, 240]
    assert codes[0, 0] == 0x7e and codes[0, 10] == 0x80
    # scales: the least power of two with a <= 448 of them, at least 2^-127
    for a, s in ((448.0, 127), (448.0001, 128), (1.75, 119), (1.76, 120), (1.0, 119), (0.875, 118),
                 (2.0 ** -119, 0), (2.0 ** -118, 1), (2.0 ** -149, 0), (2.0 ** 127, 246),
                 (3.4e38, 247), (0.0, 0)):
        assert ref.quantize(np.full((1, 3), a))[1].tolist() == [[s]], a
    assert ref.quantize(np.array([[np.nan, 1.0]]))[1].tolist() == [[255]]
    # every code but NaN's comes back as itself
    c = np.array([[k for k in range(256) if k & 127 != 127] + [0x7e, 0]], np.uint8)
    v = ref.dequantize(c, np.full((1, 8), 127, np.uint8))
    v[0, ::32] = 448  # (every block's largest)
    q, s = ref.quantize(v)
    c[0, ::32] = 0x7e
    assert (s == 127).all() and np.array_equal(q, c)


def test_reference_gradients_by_differences():
    rng = np.random.default_rng(0)
    T, D, eps = 4, 7, 0.3
    x, g = rng.standard_normal((T, D)), rng.standard_normal(D)
    dy, dh = rng.standard_normal((T, D)), rng.standard_normal((T, D))

    def total():
        return (dy * ref.norm(x, g, eps)[0]).sum() + (dh * x).sum()

    dx, dg, _, _ = ref.norm_gradients(dy, x, g, ref.norm(x, g, eps)[1], dh)
    for grad, t in ((dx, x), (dg, g)):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + 1e-6
            up = total()
            t[i] = keep - 1e-6
            down = total()
            t[i] = keep
            assert abs((up - down) / 2e-6 - grad[i]) < 1e-7


def norm(**kw):
    a = dict(dtype=BF16, gtype=BF16, T=4, D=70, X=X, ldx=70, R=R, ldr=70, G=G, H=H, ldh=70,
             codes=CODES, ldc=96, scales=SCALES, lds=3, rstd=RSTD)
    a.update(kw)
    return sg.sgemm_validate_rmsnorm(*a.values())


def back(**kw):
    a = dict(dtype=BF16, gtype=BF16, T=4, D=70, dY=DY, lddy=70, H=H, ldh=70, G=G, rstd=RSTD, dH=DH,
             lddh=70, dX=DX, lddx=70, dG=DG)
    a.update(kw)
    return sg.sgemm_validate_rmsnorm_backward(*a.values())


def test_validate_norm():
    assert norm() == sg.SGEMM_OK and norm(dtype=F32, gtype=F32) == sg.SGEMM_OK
    assert norm(gtype=F32) == sg.SGEMM_OK and norm(dtype=F16, gtype=F16) == sg.SGEMM_OK
    assert norm(R=None, ldr=0) == sg.SGEMM_OK and norm(H=None, ldh=0, rstd=None) == sg.SGEMM_OK
    for bad in (-1, 3, 4):
        assert norm(dtype=bad) == sg.SGEMM_ERR_VALUE and norm(gtype=bad) == sg.SGEMM_ERR_VALUE
    assert norm(gtype=F16) == sg.SGEMM_ERR_VALUE and norm(dtype=F32) == sg.SGEMM_ERR_VALUE
    assert norm(T=-1) == sg.SGEMM_ERR_SIZE and norm(D=0) == sg.SGEMM_ERR_SIZE
    assert norm(T=sg.SGEMM_MX_MAX_ROWS + 1) == sg.SGEMM_ERR_SIZE
    assert norm(D=sg.SGEMM_MX_MAX_K + 1, ldx=2 ** 30, ldr=2 ** 30, ldh=2 ** 30, ldc=2 ** 30,
                lds=2 ** 30) == sg.SGEMM_ERR_SIZE
    for name, short in (("ldx", 69), ("ldr", 69), ("ldh", 69), ("ldc", 95), ("lds", 2)):
        assert norm(**{name: short}) == sg.SGEMM_ERR_LD, name
    for name in ("X", "G", "codes", "scales"):
        assert norm(**{name: None}) == sg.SGEMM_ERR_NULL, name
    assert norm(T=0, X=None, G=None, codes=None, scales=None) == sg.SGEMM_OK
    for name, off in (("X", 1), ("R", 1), ("G", 1), ("H", 1), ("rstd", 2)):
        assert norm(**{name: globals()[name.upper()] + off}) == sg.SGEMM_ERR_VALUE, name
    assert norm(gtype=F32, G=G + 2) == sg.SGEMM_ERR_VALUE
    assert norm(codes=CODES + 1, scales=SCALES + 3) == sg.SGEMM_OK  # any byte address
    # in place: the same window of X or R, not another one that meets it
    assert norm(H=X) == sg.SGEMM_OK and norm(H=R) == sg.SGEMM_OK
    assert norm(H=X, ldh=72) == sg.SGEMM_ERR_ALIAS and norm(H=R + 140) == sg.SGEMM_ERR_ALIAS
    assert norm(H=X, R=X) == sg.SGEMM_OK
    assert norm(H=X, ldh=72, T=1) == sg.SGEMM_OK  # (one row has no stride to speak of)
    last = (3 * 70 + 69) * 2
    for out in ("codes", "scales", "rstd"):
        for p in (X + last, R + last, G + 138, H + last):
            if out != "rstd" or p % 4 == 0:
                assert norm(**{out: p}) == sg.SGEMM_ERR_ALIAS, (out, p)
    assert norm(rstd=X) == sg.SGEMM_ERR_ALIAS and norm(rstd=G) == sg.SGEMM_ERR_ALIAS
    assert norm(H=G) == sg.SGEMM_ERR_ALIAS
    assert norm(scales=CODES + 3 * 96 + 95) == sg.SGEMM_ERR_ALIAS
    assert norm(rstd=CODES + 4) == sg.SGEMM_ERR_ALIAS and norm(rstd=SCALES + 8) == sg.SGEMM_ERR_ALIAS


def test_validate_backward():
    assert back() == sg.SGEMM_OK and back(dH=None, lddh=0, dG=None) == sg.SGEMM_OK
    assert back(dtype=F32, gtype=F32) == sg.SGEMM_OK and back(gtype=F32) == sg.SGEMM_OK
    assert back(dtype=3) == sg.SGEMM_ERR_VALUE and back(gtype=F16) == sg.SGEMM_ERR_VALUE
    assert back(T=-1) == sg.SGEMM_ERR_SIZE and back(D=0) == sg.SGEMM_ERR_SIZE
    for name in ("lddy", "ldh", "lddh", "lddx"):
        assert back(**{name: 69}) == sg.SGEMM_ERR_LD, name
    for name in ("dY", "H", "G", "rstd", "dX"):
        assert back(**{name: None}) == sg.SGEMM_ERR_NULL, name
    assert back(T=0, dY=None, H=None, G=None, rstd=None, dX=None) == sg.SGEMM_OK
    for name, off in (("dY", 1), ("H", 1), ("G", 1), ("dH", 1), ("dX", 1), ("dG", 1), ("rstd", 2)):
        assert back(**{name: globals()[name.upper()] + off}) == sg.SGEMM_ERR_VALUE, name
    # dX may stand in dY's or dH's place
    assert back(dX=DY) == sg.SGEMM_OK and back(dX=DH) == sg.SGEMM_OK
    assert back(dX=DY, lddx=72) == sg.SGEMM_ERR_ALIAS and back(dX=DH + 2) == sg.SGEMM_ERR_ALIAS
    for p in (H, G, RSTD, DG):
        assert back(dX=p) == sg.SGEMM_ERR_ALIAS
    for p in (DY, H, DH, G, RSTD, DX):
        assert back(dG=p) == sg.SGEMM_ERR_ALIAS


def test_entries_without_a_device():
    lib = sg.library()
    assert lib.sgemm_mx_byte_quantize(None, F32, 0, 1, 32, X, 32, CODES, 32, SCALES, 1,
                                      None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_mx_byte_dequantize(None, F32, 1, 32, CODES, 32, SCALES, 1, X, 32,
                                        None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_rmsnorm(None, F32, F32, 1, 32, X, 32, None, 0, G, 1e-6, None, 0, CODES, 32,
                             SCALES, 1, None, None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_rmsnorm_backward(None, F32, F32, 1, 32, DY, 32, H, 32, G, RSTD, None, 0, DX, 32,
                                      None, None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_rmsnorm_workspace_size(None, 1, 1, None, None) == sg.SGEMM_ERR_HANDLE
    h = HostHandle()
    at = ctypes.addressof(h)

    def quantize(dtype=BF16, trans=0, R=3, K=40, ldx=40, ldc=64, lds=2, x=X, c=CODES, s=SCALES):
        return lib.sgemm_mx_byte_quantize(at, dtype, trans, R, K, x, ldx, c, ldc, s, lds, None)

    assert quantize() == sg.SGEMM_ERR_DEVICE  # (as far as it gets without one)
    assert quantize(ldc=63) == sg.SGEMM_ERR_LD and quantize(lds=1) == sg.SGEMM_ERR_LD
    assert quantize(dtype=3) == sg.SGEMM_ERR_VALUE and quantize(trans=2) == sg.SGEMM_ERR_VALUE
    assert quantize(x=X + 1) == sg.SGEMM_ERR_VALUE and quantize(c=None) == sg.SGEMM_ERR_NULL
    assert quantize(c=X + 4) == sg.SGEMM_ERR_ALIAS and quantize(s=CODES + 2 * 64 + 63) == sg.SGEMM_ERR_ALIAS
    assert quantize(R=0, x=None) == sg.SGEMM_OK
    # 2^24 workgroups of 512 units of eight values are one too many
    K = 1 << 20
    fits = ((1 << 24) - 1) * 512 * 8 // K
    far = dict(K=K, ldx=K, ldc=K, lds=K // 32, x=1 << 60, c=1 << 52, s=1 << 56)
    assert quantize(R=fits + 1, **far) == sg.SGEMM_ERR_UNSUPPORTED
    assert quantize(R=fits, **far) == sg.SGEMM_ERR_DEVICE
    # the norm's rows are taken in turns: any number
    assert lib.sgemm_rmsnorm(at, F32, F32, sg.SGEMM_MX_MAX_ROWS, 8, 1 << 50, 8, None, 0, G, 1e-6, None,
                             0, 1 << 54, 32, 1 << 56, 1, None, None) == sg.SGEMM_ERR_DEVICE
    least, full = sg.sgemm_rmsnorm_workspace_size(at, 1000, 100)
    assert least == 4 * 100 and full == 63 * least  # (sixteen rows a workgroup)
    assert sg.sgemm_rmsnorm_workspace_size(at, 100000, 4096) == (4 * 4096, h.cus * 4 * 4096)
    assert sg.sgemm_rmsnorm_workspace_size(at, 0, 5000) == (0, 0)
    assert sg.sgemm_rmsnorm_workspace_size(at, 3, 5000) == (20000, 60000)


def test_container():
    torch = pytest.importorskip("torch")
    u8 = dict(dtype=torch.uint8)
    q = sg.Mx8.empty(3, 65, "cpu")
    assert (q.rows, q.K, tuple(q.codes.shape), tuple(q.scales.shape)) == (3, 96, (3, 96), (3, 3))
    assert sg.Mx8.nbytes(3, 65) == q.codes.numel() + q.scales.numel()
    assert sg.Mx4.nbytes(3, 65) == 3 * 17 * 3
    sg.Mx8(torch.zeros(3, 70, **u8)[:, :64], torch.zeros(3, 2, **u8))
    for codes, scales in (((3, 32), (3, 2)), ((3, 64), (4, 2))):
        with pytest.raises(ValueError):
            sg.Mx8(torch.zeros(codes, **u8), torch.zeros(scales, **u8))
    with pytest.raises(TypeError):
        sg.Mx8(torch.zeros(3, 64), torch.zeros(3, 2, **u8))
    with pytest.raises(ValueError):
        sg.Mx8.empty(3, 2 ** 31, "meta")


def test_binding_checks():
    torch = pytest.importorskip("torch")
    bf16 = torch.bfloat16
    assert sg._gain(torch.ones(40), bf16, 40) == F32
    assert sg._gain(torch.ones(40, dtype=bf16), bf16, 40) == BF16
    with pytest.raises(TypeError):
        sg._gain(torch.ones(40, dtype=torch.float16), bf16, 40)
    with pytest.raises(ValueError):
        sg._gain(torch.ones(41), bf16, 40)
    with pytest.raises(ValueError):
        sg._gain(torch.ones(80)[::2], bf16, 40)
    rows = torch.zeros(3, 48, dtype=bf16)[:, :40]
    assert sg._same("H", rows, bf16, (3, 40)) == (rows.data_ptr(), 48)
    for bad in (rows.float(), rows[:2], rows.t()):
        with pytest.raises(ValueError):
            sg._same("H", bad, bf16, (3, 40))


A8, SA, W, SW, C = 0x1000000, 0x2000000, 0x3000000, 0x4000000, 0x8000000  # never touched


def product(**kw):
    a = dict(bits=8, M=4, N=5, K=64, A=A8, lda=64, SA=SA, ldsa=2, B=W, ldb=64, SB=SW, ldsb=2, dtype=BF16,
             C=C, ldc=5)
    a.update(kw)
    return sg.sgemm_validate_mx_byte(*a.values())


def test_validate_product():
    assert product() == sg.SGEMM_OK and product(bits=4, ldb=32) == sg.SGEMM_OK
    assert product(dtype=F32) == sg.SGEMM_OK and product(dtype=F16) == sg.SGEMM_OK
    for bits in (0, 6, 16, -8):
        assert product(bits=bits) == sg.SGEMM_ERR_VALUE
    for bad in (-1, 3, 4, 5):
        assert product(dtype=bad) == sg.SGEMM_ERR_VALUE
    for name in ("M", "N", "K"):
        assert product(**{name: -32}) == sg.SGEMM_ERR_SIZE
    assert product(K=63) == sg.SGEMM_ERR_SIZE
    for name in ("M", "N"):
        assert product(**{name: sg.SGEMM_MX_MAX_ROWS + 1}, ldc=2 ** 31 - 1) == sg.SGEMM_ERR_SIZE
    for name, short in (("lda", 63), ("ldsa", 1), ("ldb", 63), ("ldsb", 1), ("ldc", 4)):
        assert product(**{name: short}) == sg.SGEMM_ERR_LD, name
    assert product(bits=4, ldb=31) == sg.SGEMM_ERR_LD
    for name in ("A", "SA", "B", "SB", "C"):
        assert product(**{name: None}) == sg.SGEMM_ERR_NULL, name
    assert product(A=None, SA=None, B=None, SB=None, K=0) == sg.SGEMM_OK
    assert product(M=0, A=None, C=None) == sg.SGEMM_OK
    assert product(C=C + 1) == sg.SGEMM_ERR_VALUE
    assert product(A=A8 + 1, SA=SA + 1, B=W + 3, SB=SW + 1) == sg.SGEMM_OK  # any byte address
    assert product(C=A8 + 64 * 3 + 62) == sg.SGEMM_ERR_ALIAS
    assert product(C=W + 64 * 4 + 62) == sg.SGEMM_ERR_ALIAS
    assert product(bits=4, ldb=32, C=W + 32 * 4 + 32) == sg.SGEMM_OK
    assert product(C=SA + 6) == sg.SGEMM_ERR_ALIAS and product(C=SW + 8) == sg.SGEMM_ERR_ALIAS


def test_product_entries_without_a_device():
    lib = sg.library()
    assert lib.sgemm_run_mx_byte(None, 8, 1, 1, 32, 1.0, A8, 32, SA, 1, W, 32, SW, 1, 0.0, BF16, C, 1,
                                 None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_run_mx_byte_quant(None, BF16, 8, 1, 1, 32, 1.0, A8, 32, W, 32, SW, 1, 0.0, BF16, C,
                                       1, None) == sg.SGEMM_ERR_HANDLE
    h = HostHandle()
    at = ctypes.addressof(h)

    def quant(xtype=BF16, bits=8, M=3, K=40, x=A8, ldx=40, ldb=64, c=C):
        return lib.sgemm_run_mx_byte_quant(at, xtype, bits, M, 5, K, 1.0, x, ldx, W, ldb, SW, 2, 0.0, BF16,
                                           c, 5, None)

    assert quant() == sg.SGEMM_ERR_DEVICE and quant(bits=4, ldb=32) == sg.SGEMM_ERR_DEVICE
    assert quant(bits=5) == sg.SGEMM_ERR_VALUE and quant(xtype=3) == sg.SGEMM_ERR_VALUE
    assert quant(ldx=39) == sg.SGEMM_ERR_LD and quant(ldb=63) == sg.SGEMM_ERR_LD
    assert quant(x=A8 + 1) == sg.SGEMM_ERR_VALUE and quant(x=None) == sg.SGEMM_ERR_NULL
    assert quant(c=A8 + 8) == sg.SGEMM_ERR_ALIAS and quant(M=0, x=None) == sg.SGEMM_OK
    K = 1 << 20
    fits = ((1 << 24) - 1) * 512 * 8 // K
    assert lib.sgemm_run_mx_byte_quant(at, BF16, 8, fits + 1, 1, K, 1.0, 1 << 60, K, 1 << 50, K, 1 << 52,
                                       K // 32, 0.0, BF16, 1 << 48, 1, None) == sg.SGEMM_ERR_UNSUPPORTED


def grad(**kw):
    a = dict(dtype=BF16, T=4, N=5, D=70, dY=DY, lddy=5, X=CODES, ldx=96, SX=SCALES, ldsx=3, wtype=F32,
             dW=C, lddw=70)
    a.update(kw)
    return sg.sgemm_validate_mx_byte_weight_grad(*a.values())


def test_validate_weight_grad():
    assert grad() == sg.SGEMM_OK and grad(dtype=F16, wtype=F16) == sg.SGEMM_OK
    assert grad(wtype=BF16) == sg.SGEMM_OK
    for bad in (-1, F32, 3, 4):
        assert grad(dtype=bad) == sg.SGEMM_ERR_VALUE
    for bad in (-1, 3, 4):
        assert grad(wtype=bad) == sg.SGEMM_ERR_VALUE
    for name in ("T", "N", "D"):
        assert grad(**{name: -1}) == sg.SGEMM_ERR_SIZE
    for name, short in (("lddy", 4), ("ldx", 95), ("ldsx", 2), ("lddw", 69)):
        assert grad(**{name: short}) == sg.SGEMM_ERR_LD, name
    for name in ("dY", "X", "SX", "dW"):
        assert grad(**{name: None}) == sg.SGEMM_ERR_NULL, name
    assert grad(T=0, dY=None, X=None, SX=None) == sg.SGEMM_OK
    assert grad(N=0, dY=None, dW=None) == sg.SGEMM_OK and grad(D=0, X=None, dW=None) == sg.SGEMM_OK
    assert grad(dY=DY + 1) == sg.SGEMM_ERR_VALUE and grad(dW=C + 2) == sg.SGEMM_ERR_VALUE
    assert grad(X=CODES + 1, SX=SCALES + 1) == sg.SGEMM_OK  # any byte address
    assert grad(dW=DY + 36) == sg.SGEMM_ERR_ALIAS and grad(dW=CODES + 4 * 96 - 4) == sg.SGEMM_ERR_ALIAS
    assert grad(dW=SCALES + 8) == sg.SGEMM_ERR_ALIAS
    # a step of 64 tokens within 32-bit offsets
    far = dict(dY=1 << 50, X=1 << 52, SX=1 << 54, dW=1 << 40)
    assert grad(lddy=1 << 24, ldx=1 << 25, ldsx=1 << 25, **far) == sg.SGEMM_OK
    for name in ("lddy", "ldx", "ldsx"):
        assert grad(**{name: 1 << 27}, **far) == sg.SGEMM_ERR_UNSUPPORTED
        assert grad(**{name: 1 << 27}, T=1, **far) == sg.SGEMM_OK


def test_weight_grad_workspace_size():
    lib = sg.library()
    assert lib.sgemm_mx_byte_weight_grad(None, BF16, 1, 1, 32, 1.0, DY, 1, CODES, 32, SCALES, 1, 0.0, F32,
                                         C, 32, None) == sg.SGEMM_ERR_HANDLE
    h = HostHandle()
    at = ctypes.addressof(h)
    assert lib.sgemm_mx_byte_weight_grad_workspace_size(at, 1, 1, 1, None) == sg.SGEMM_ERR_NULL
    size = lambda *a: sg.sgemm_mx_byte_weight_grad_workspace_size(at, *a)  # noqa: E731
    with pytest.raises(sg.SgemmError):
        size(-1, 1, 1)
    assert size(0, 5, 5) == size(100, 5, 5) == size(1000, 0, 5) == 0
    assert size(4096, 11008, 4096) == 0  # tiles enough
    assert size(16384, 100, 200) >= 2 * 4 * 100 * 200
    # tokens of any number, and sizes at the ends of their ranges
    for T in (1, 63, 64, 127, 128, 129, 1 << 20, sg.SGEMM_MX_MAX_ROWS):
        for N, D in ((1, 1), (1, sg.SGEMM_MX_MAX_K), (sg.SGEMM_MX_MAX_ROWS, 1), (300, 200)):
            parts, rest = divmod(size(T, N, D), 4 * N * -(-D // 4) * 4)
            assert rest == 0 and (parts == 0 or 2 <= parts <= max(T // 128, 1))
