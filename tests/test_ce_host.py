"""The output layer's loss without a GPU: the plain implementation against
differences and closed forms, and every refusal of the C entries and the
binding."""
import ctypes

import numpy as np
import pytest

import fp32_gemm_major_amd as sg
from tests import ce_reference as ref

X, W, Y, LOSS, LSE = 0x10000000, 0x20000000, 0x30000000, 0x31000000, 0x32000000  # never touched
DL, DE, DX, DW = 0x33000000, 0x34000000, 0x40000000, 0x50000000
F32, BF16, F16 = sg.SGEMM_DTYPE_F32, sg.SGEMM_DTYPE_BF16, sg.SGEMM_DTYPE_F16


def test_reference_closed_forms():
    # equal logits: log V; one logit far above: its label costs nothing
    _, loss, lse = ref.forward(np.zeros((2, 3)), np.ones((7, 3)), np.array([0, 6]))
    assert np.allclose(loss, np.log(7)) and np.allclose(lse, np.log(7))
    w = np.zeros((4, 1))
    w[2] = 100.0
    _, loss, lse = ref.forward(np.ones((2, 1)), w, np.array([2, 1]))
    assert np.allclose(loss, [0, 100]) and np.allclose(lse, 100)


def test_reference_gradients_by_differences():
    rng = np.random.default_rng(0)
    T, V, D, alpha = 5, 11, 4, 0.7
    x, w = rng.standard_normal((T, D)), rng.standard_normal((V, D))
    labels = np.array([3, ref.IGNORE, 0, 10, 3])
    a, b = rng.standard_normal(T), rng.standard_normal(T)

    def total(x, w):
        _, loss, lse = ref.forward(x, w, labels, alpha)
        return (a * loss + b * lse).sum()

    z, _, lse = ref.forward(x, w, labels, alpha)
    dx, dw = ref.gradients(x, w, labels, ref.dlogits(z, labels, lse, a, b), alpha)
    h = 1e-6
    for g, t in ((dx, x), (dw, w)):
        for i in np.ndindex(t.shape):
            keep = t[i]
            t[i] = keep + h
            up = total(x, w)
            t[i] = keep - h
            down = total(x, w)
            t[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-7


def fwd(**kw):
    a = dict(dtype=F32, T=4, V=9, D=6, X=X, ldx=6, W=W, ldw=6, labels=Y, loss=LOSS, lse=LSE)
    a.update(kw)
    return sg.sgemm_validate_ce(*a.values())


def bwd(**kw):
    a = dict(dtype=F32, T=4, V=9, D=6, X=X, ldx=6, W=W, ldw=6, labels=Y, lse=LSE, dloss=DL, dlse=DE,
             dX=DX, lddx=6, dW=DW, lddw=6)
    a.update(kw)
    return sg.sgemm_validate_ce_backward(*a.values())


def test_validate():
    for v in (fwd, bwd):
        assert v() == sg.SGEMM_OK
        assert v(dtype=BF16) == sg.SGEMM_OK and v(dtype=F16) == sg.SGEMM_OK
        for bad in (-1, 3, 4):
            assert v(dtype=bad) == sg.SGEMM_ERR_VALUE
        assert v(T=-1) == sg.SGEMM_ERR_SIZE and v(V=0) == sg.SGEMM_ERR_SIZE
        assert v(D=0) == sg.SGEMM_ERR_SIZE and v(V=-3) == sg.SGEMM_ERR_SIZE
        big = sg.SGEMM_CE_MAX_D + 1
        assert v(D=big, ldx=big, ldw=big) == sg.SGEMM_ERR_SIZE
        assert v(T=2 ** 31 - 1) == sg.SGEMM_ERR_SIZE and v(V=2 ** 31 - 1) == sg.SGEMM_ERR_SIZE
        assert v(ldx=5) == sg.SGEMM_ERR_LD and v(ldw=5) == sg.SGEMM_ERR_LD
        for name in ("X", "W", "labels", "lse"):
            assert v(**{name: None}) == sg.SGEMM_ERR_NULL, name
        assert v(T=0, X=None, labels=None) == sg.SGEMM_OK
        assert v(X=X + 2) == sg.SGEMM_ERR_VALUE and v(W=W + 1, dtype=BF16) == sg.SGEMM_ERR_VALUE
        assert v(X=X + 2, dtype=BF16) == sg.SGEMM_OK
        assert v(labels=Y + 4) == sg.SGEMM_ERR_VALUE and v(labels=Y + 8) == sg.SGEMM_OK
        assert v(lse=LSE + 2) == sg.SGEMM_ERR_VALUE and v(lse=LSE + 64) == sg.SGEMM_OK
    assert fwd(loss=LOSS + 1) == sg.SGEMM_ERR_VALUE
    assert bwd(dloss=DL + 2) == sg.SGEMM_ERR_VALUE and bwd(dlse=DE + 1) == sg.SGEMM_ERR_VALUE
    assert fwd(loss=None) == sg.SGEMM_ERR_NULL
    assert fwd(loss=LSE + 12) == sg.SGEMM_ERR_ALIAS and fwd(loss=LSE + 16) == sg.SGEMM_OK
    for a in (X, W, Y):
        assert fwd(loss=a) == sg.SGEMM_ERR_ALIAS and fwd(lse=a + 4) == sg.SGEMM_ERR_ALIAS
    assert bwd(dloss=None) == sg.SGEMM_ERR_NULL
    assert bwd(dlse=None) == sg.SGEMM_OK
    assert bwd(dX=None, lddx=0) == sg.SGEMM_OK and bwd(dW=None, lddw=0) == sg.SGEMM_OK
    assert bwd(lddx=5) == sg.SGEMM_ERR_LD and bwd(lddw=5) == sg.SGEMM_ERR_LD
    assert bwd(dX=DX + 2) == sg.SGEMM_ERR_VALUE
    for a in (X, W, Y, LSE, DL, DE, DW):
        assert bwd(dX=a) == sg.SGEMM_ERR_ALIAS, hex(a)
    for a in (X, W, Y, LSE, DL, DE):
        assert bwd(dW=a) == sg.SGEMM_ERR_ALIAS, hex(a)


def test_sizes_that_a_launch_does_not_hold():
    """Rows or elements whose threads a launch does not count in 32 bits are
    refused before anything is queued."""
    h = HostHandle()
    lib, at = sg.library(), ctypes.addressof(h)
    x, w, y, a, b = (1 << k for k in (60, 56, 54, 52, 53))  # never touched

    def forward(dtype, T, V, D):
        return lib.sgemm_ce_forward(at, dtype, T, V, D, 1.0, x, D, w, D, y, -100, a, b, None)

    def backward(dtype, T, V, D):
        return lib.sgemm_ce_backward(at, dtype, T, V, D, 1.0, x, D, w, D, y, -100, a, b, None, None, 0,
                                     1 << 58, D, None)

    for dtype in (F32, BF16, F16):
        for call in (forward, backward):
            assert call(dtype, 1 << 28, 100, 8) == sg.SGEMM_ERR_UNSUPPORTED
            assert call(dtype, 1 << 20, 100, 1 << 16) == sg.SGEMM_ERR_UNSUPPORTED
            for T in (1, 100, 1 << 20):
                assert call(dtype, T, 100, 8) == sg.SGEMM_ERR_DEVICE
        assert backward(dtype, 0, 1 << 27, 256) == sg.SGEMM_ERR_UNSUPPORTED


def test_null_handle():
    lib = sg.library()
    assert lib.sgemm_ce_workspace_size(None, F32, 1, 1, 1, 0, None, None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_ce_forward(None, F32, 1, 1, 1, 1.0, X, 1, W, 1, Y, -100, LOSS, LSE,
                                None) == sg.SGEMM_ERR_HANDLE
    assert lib.sgemm_ce_backward(None, F32, 1, 1, 1, 1.0, X, 1, W, 1, Y, -100, LSE, DL, None, DX, 1,
                                 DW, 1, None) == sg.SGEMM_ERR_HANDLE


def test_binding_checks():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(3, 8), torch.zeros(5, 8)
    assert sg._ce_shapes(x, w) == (F32, 3, 5, 8, 8, 8)
    with pytest.raises(ValueError):
        sg._ce_shapes(x, w.bfloat16())
    with pytest.raises(ValueError):
        sg._ce_shapes(x, torch.zeros(5, 7))
    with pytest.raises(TypeError):
        sg._vectors(3, torch.int64, labels=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        sg._vectors(3, torch.int64, labels=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        sg._vectors(3, torch.float32, loss=torch.zeros(6)[::2])


class HostHandle(ctypes.Structure):
    """A handle as the library lays it out, for entries that launch nothing: of
    no device, so that any other entry ends at its check of the device."""
    _fields_ = [("device", ctypes.c_int), ("cus", ctypes.c_int), ("variant", ctypes.c_int),
                ("forced_kernel", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("forced_lowp", ctypes.c_int)]

    def __init__(self):
        super().__init__(device=-1, cus=256, forced_kernel=-1, forced_lowp=-1)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("backward", [0, 1])
def test_workspace_size(dtype, backward):
    """An empty batch needs no workspace; other sizes grow with the rows."""
    h = HostHandle()
    at = ctypes.addressof(h)
    for V, D in ((1, 1), (32000, 4096), (300, 7)):
        assert sg.sgemm_ce_workspace_size(at, dtype, 0, V, D, backward) == (0, 0)
        last = (0, 0)
        for T in (1, 16, 17, 511, 512, 5000):
            size = sg.sgemm_ce_workspace_size(at, dtype, T, V, D, backward)
            assert 0 < size[0] <= size[1]
            if T in (16, 511, 5000):  # (with the row before it on one path)
                assert size[0] > last[0]
            last = size
    for bad in (dict(T=-1), dict(V=0), dict(D=0)):
        a = dict(T=0, V=1, D=1) | bad
        with pytest.raises(sg.SgemmError) as e:
            sg.sgemm_ce_workspace_size(at, dtype, a["T"], a["V"], a["D"], backward)
        assert e.value.status == sg.SGEMM_ERR_SIZE
