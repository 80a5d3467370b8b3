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
