"""What the weight gradients' workspace query reports, without a GPU."""
import ctypes
import random

import fp32_gemm_major_amd as sg
from tests.test_ce_host import HostHandle


def test_reported_workspace_follows_the_rows_blocks():
    """A gradient over D columns splits its tokens as one over the whole blocks that the
    rows hold does, so that the query made of the rows alone is enough for it."""
    h = HostHandle()
    at = ctypes.addressof(h)
    rng = random.Random(3)
    log = lambda lo, hi: round(lo * (hi / lo) ** rng.random())  # noqa: E731
    splits = 0
    for _ in range(4000):
        T, N, D = log(1, 16384), log(1, 8192), log(1, 8192)
        K = 32 * -(-D // 32)
        own = sg.sgemm_mx_byte_weight_grad_workspace_size(at, T, N, D)
        whole = sg.sgemm_mx_byte_weight_grad_workspace_size(at, T, N, K)
        assert own // (4 * N * (-(-D // 4) * 4)) == whole // (4 * N * K), (T, N, D)
        splits += own > 0
    assert splits > 500


def test_strides_of_a_step_stay_inside_32_bits():
    """The largest strides that a weight gradient takes leave room for 63 of them, a tile's
    256 columns and a lane's sixteen bytes below 2^32."""
    far = dict(dY=1 << 50, X=1 << 52, SX=1 << 54, dW=1 << 40)

    def takes(**strides):
        a = dict(dtype=sg.SGEMM_DTYPE_BF16, T=64, N=8, D=31000, dY=far["dY"], lddy=8, X=far["X"], ldx=31008,
                 SX=far["SX"], ldsx=969, wtype=sg.SGEMM_DTYPE_F32, dW=far["dW"], lddw=31000)
        a.update(strides)
        st = sg.sgemm_validate_mx_byte_weight_grad(*a.values())
        assert st in (sg.SGEMM_OK, sg.SGEMM_ERR_UNSUPPORTED)
        return st == sg.SGEMM_OK

    for name, size in (("lddy", 2), ("ldx", 1), ("ldsx", 1)):
        lo, hi = 1 << 24, 1 << 28
        while hi - lo > 1:
            mid = (lo + hi) // 2
            lo, hi = (mid, hi) if takes(**{name: mid}) else (lo, mid)
        assert 63 * lo * size + 256 * size + 16 < 1 << 32
        assert lo * size > 65 << 20
    assert lo == 68174067
