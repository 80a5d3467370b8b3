"""Weight gradients of kept rows that lie as far apart as the entry takes them."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests.test_gpu_mx8_grad import gradient, kept  # noqa: E402


@pytest.mark.parametrize("N", [8, 9])  # (a whole step of tokens, and tokens after the last one)
def test_columns_of_the_farthest_token(N):
    """64 tokens whose last one starts just below 2^32 bytes, its later columns past
    them."""
    T, D, ld = 64, 31000, 68174067
    X, dY = kept(T, D, 1), gradient(T, N, 2, "bf16").cuda()
    buf = torch.empty((T - 1) * ld + X.K, dtype=torch.uint8, device="cuda")
    codes = buf.as_strided((T, X.K), (ld, 1))
    codes.copy_(X.codes)
    with sg.Handle() as h:
        got, want = torch.empty(N, D, device="cuda"), torch.empty(N, D, device="cuda")
        h.mx8_weight_grad(dY, sg.Mx8(codes, X.scales), got)
        h.mx8_weight_grad(dY, X, want)
        assert torch.equal(got, want)
