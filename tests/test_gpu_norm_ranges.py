"""The norm's results over its types' whole ranges, against 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests.test_gpu_mx import DTYPES, as_numpy  # noqa: E402
from tests.test_gpu_norm import rows  # noqa: E402

EPS = float(np.float32(1e-5))


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


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
