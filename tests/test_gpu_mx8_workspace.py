"""The workspace that a weight gradient reports is all that it makes use of: with it
the tokens are split as with any larger one, which shows in equal bits (another split
adds the same products in another order)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests.test_gpu_mx8_grad import gradient, kept  # noqa: E402


@pytest.mark.parametrize("T,N,D", [
    # the ranges of a split are whole steps of tokens, so fewer ranges than were asked
    # for may hold all of them
    (5371, 1, 84), (10300, 48, 2410), (1631, 1, 351), (1561, 2, 1803),
    # D ends inside its last block, which the rows' size does not tell
    (1427, 129, 614), (2238, 5017, 44), (3903, 632, 60), (2322, 873, 97),
    (2000, 40, 70), (1500, 300, 200)])
def test_reported_workspace_gives_the_whole_split(T, N, D):
    X, dY = kept(T, D, T), gradient(T, N, T + 1, "bf16").cuda()
    with sg.Handle(workspace=False) as h:
        reported = h.mx8_weight_grad_workspace_size(dY, X)
        own = sg.sgemm_mx_byte_weight_grad_workspace_size(h.h, T, N, D)
        assert own <= reported  # (0: one range)
        results = []
        for size in (own, reported, 1 << 28):
            h.set_workspace(size)
            dW = torch.full((N, D), float("nan"), device="cuda")
            h.mx8_weight_grad(dY, X, dW)
            results.append(dW)
        assert torch.equal(results[0], results[2]) and torch.equal(results[1], results[2])
