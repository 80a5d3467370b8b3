"""Weight gradients from 8-bit rows on the GPU against the plain 64-bit
implementation.

X's values are exact in dY's type, products of two 16-bit values are exact in 32
bits and are summed in 32 bits: off by 4*max(T,1)*2^-24*(|alpha|*sum|dY*X| +
|beta*dW|) and half a step of dW's type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests.test_gpu_mx import DTYPES, as_numpy, half_step, strided, values  # noqa: E402


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


def kept(T, D, seed):
    codes, scales = ref.quantize(values(T, D, seed, spread=3))
    return sg.Mx8(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def gradient(T, N, seed, dt):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((T, N))).to(DTYPES[dt])


def check(got, dy, x, alpha, beta, w, dt, what=""):
    T = dy.shape[0]
    r, t = alpha * (dy.T @ x), abs(alpha) * (np.abs(dy).T @ np.abs(x))
    if beta:
        r, t = r + beta * w, t + np.abs(beta * w)
    bound = 4 * max(T, 1) * 2.0 ** -24 * t
    if dt != "f32":
        bound = bound + half_step(dt) * (np.abs(r) + bound) + (2.0 ** -25 if dt == "f16" else 0)
    err = np.abs(got.double().cpu().numpy() - r)
    assert np.all(err <= bound), (what, float((err - bound).max()), np.argwhere(err > bound)[:3])


SIZES = [(1, 1, 1), (1, 300, 200), (2, 1, 40), (9, 3, 33), (63, 7, 31), (64, 8, 32), (65, 9, 64),
         (128, 128, 128), (200, 129, 1000), (777, 130, 100), (1000, 1, 16), (1000, 5, 300),
         (1100, 250, 130), (4096, 40, 70), (5000, 300, 600), (300, 1500, 1000), (64, 2900, 3050),
         (130, 3500, 3600), (193, 3600, 3501), (1, 3600, 3600), (330, 3500, 3600), (384, 3600, 3501),
         (450, 3500, 3600)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,D", SIZES)
def test_weight_grad(handle, T, N, D, dt):
    X, dy = kept(T, D, T + D), gradient(T, N, T + N, dt)
    x = ref.dequantize(*as_numpy(X))[:, :D]
    for wt, alpha, beta in (("f32", 1.0, 0.0), ("f32", 0.5, 1.0), (dt, 0.125, 0.0), ("bf16", 1.0, 0.5)):
        w0 = torch.from_numpy(np.random.default_rng(N).standard_normal((N, D)) * 4).to(DTYPES[wt])
        if beta == 0.0:
            w0.fill_(float("nan"))  # dW is not read
        outs = []
        for pad in (0, 3):
            dY, _ = strided(dy, pad, fill=float("nan"))
            dW, buf = strided(w0, pad, fill=7.0)
            handle.mx8_weight_grad(dY, X, dW, alpha=alpha, beta=beta)
            check(dW, dy.double().numpy(), x, alpha, beta, w0.double().numpy() if beta else None, wt,
                  (T, N, D, pad))
            assert (buf[:, D:] == 7.0).all()
            outs.append(dW.clone())
        assert torch.equal(*outs)  # same bits, whatever the strides
        if N * D > 10 ** 6:
            break


@pytest.mark.parametrize("T,N,D", [(70, 40, 50), (1000, 200, 300), (100, 3600, 3600)])
def test_integers_are_exact(handle, T, N, D):
    rng = np.random.default_rng(T)
    v, s = rng.integers(-4, 5, (T, 32 * -(-D // 32))), rng.integers(126, 129, (T, -(-D // 32)))
    v[:, D:] = 0
    codes = np.searchsorted(ref.GRID, np.abs(v)).astype(np.uint8) | np.where(v < 0, 128, 0).astype(np.uint8)
    X = sg.Mx8(torch.from_numpy(codes).cuda(), torch.from_numpy(s.astype(np.uint8)).cuda())
    dy = torch.from_numpy(rng.integers(-4, 5, (T, N)).astype(np.float64))
    dW = torch.empty(N, D, device="cuda")
    for dt in ("bf16", "f16"):
        handle.mx8_weight_grad(dy.to(DTYPES[dt]).cuda(), X, dW)
        want = dy.numpy().T @ ref.dequantize(*as_numpy(X))[:, :D]
        assert np.array_equal(dW.double().cpu().numpy(), want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,N,D", [(70, 40, 100), (640, 200, 300), (128, 3600, 3600)])
def test_nan_and_infinity(handle, T, N, D, dt):
    """A block of scale 255 and a NaN code make their columns NaN, an infinity or
    NaN of dY its row; the last token and what lies past the edges count too."""
    X, dy = kept(T, D, 1), gradient(T, N, 2, dt)
    X.codes[:, :64] |= 8  # (no zeros, which an infinity would make NaN)
    X.scales[T - 1, 1] = 255
    X.codes[0, 70] = 0x7F
    dy[T - 1, N - 1] = float("inf")
    dy[3, 5] = float("nan")
    dW = torch.empty(N, D, device="cuda")
    handle.mx8_weight_grad(dy.cuda(), X, dW)
    got = dW.cpu()
    x = ref.dequantize(*as_numpy(X))[:, :D]
    cols = torch.from_numpy(np.isnan(x).any(0))  # (0x77 | 8 is a NaN too)
    assert cols[32:64].all() and cols[70] and not cols.all()
    nan = torch.zeros(N, D, dtype=torch.bool)
    nan[:, cols], nan[5] = True, True
    assert torch.isnan(got[nan]).all()
    rest = got[:N - 1][~nan[:N - 1]]
    assert torch.isfinite(rest).all()
    assert (x[T - 1, :32] != 0).all() and torch.isinf(got[N - 1, :32][~cols[:32]]).all()


def test_extreme_scales(handle):
    """bfloat16 holds every value down to its smallest normal number."""
    T, N, D = 64, 8, 32
    codes = torch.full((T, 32), 0x38, dtype=torch.uint8, device="cuda")
    scales = torch.arange(T, dtype=torch.uint8, device="cuda")[:, None] * 3 + 1  # 2^-126 .. 2^63
    dy = torch.eye(T, N, device="cuda", dtype=torch.bfloat16)
    for first in range(0, T, N):
        dW = torch.empty(N, D, device="cuda")
        handle.mx8_weight_grad(dy.roll(first, 0).contiguous(), sg.Mx8(codes, scales), dW)
        want = torch.exp2((scales[first:first + N].double() - 127)).expand(N, D)
        assert torch.equal(dW.double(), want)


@pytest.mark.parametrize("T,N,D", [(2000, 40, 70), (1500, 300, 200)])
def test_workspace(handle, T, N, D):
    X, dy = kept(T, D, 1), gradient(T, N, 2, "bf16").cuda()
    x = ref.dequantize(*as_numpy(X))[:, :D]
    full = handle.mx8_weight_grad_workspace_size(dy, X)
    part = 4 * N * (-(-D // 4) * 4)
    assert full > 2 * part
    with sg.Handle(workspace=False) as own:
        for size in (0, part, 2 * part, full - 4, full, 2 * full):
            own.set_workspace(size)
            runs = []
            for _ in range(2):
                dW = torch.full((N, D), float("nan"), device="cuda")
                own.mx8_weight_grad(dy, X, dW)
                check(dW, dy.double().cpu().numpy(), x, 1.0, 0.0, None, "f32", size)
                runs.append(dW)
            assert torch.equal(*runs)


def test_empty(handle):
    dW = torch.full((5, 40), 2.0, device="cuda")
    none = torch.empty(0, 5, device="cuda", dtype=torch.bfloat16)
    handle.mx8_weight_grad(none, sg.Mx8.empty(0, 40), dW, beta=0.5)
    assert (dW == 1.0).all()
    dW.fill_(float("nan"))
    handle.mx8_weight_grad(none, sg.Mx8.empty(0, 40), dW)
    assert (dW == 0.0).all()
    X = kept(4, 40, 1)
    handle.mx8_weight_grad(torch.empty(4, 0, device="cuda", dtype=torch.bfloat16), X, dW[:0])


def test_operands_inside_wider_buffers(handle):
    """Odd byte strides of codes and scales, odd element strides of dY whose last
    row ends its buffer."""
    for T, N, D in ((130, 9, 100), (70, 3, 40), (500, 133, 300), (128, 8, 64), (129, 1, 33)):
        X, dy = kept(T, D, 1), gradient(T, N, 2, "bf16")
        want = torch.empty(N, D, device="cuda")
        handle.mx8_weight_grad(dy.cuda(), X, want)
        for pad in (1, 5):
            cb = torch.full((T, X.codes.shape[1] + pad), 255, dtype=torch.uint8, device="cuda")
            sb = torch.full((T, X.scales.shape[1] + pad), 255, dtype=torch.uint8, device="cuda")
            cb[:, :-pad], sb[:, :-pad] = X.codes, X.scales
            buf = torch.full(((T - 1) * (N + pad) + N,), float("nan"), dtype=dy.dtype, device="cuda")
            dY = buf.as_strided((T, N), (N + pad, 1))
            dY.copy_(dy)
            got = torch.empty(N, D, device="cuda")
            handle.mx8_weight_grad(dY, sg.Mx8(cb[:, :-pad], sb[:, :-pad]), got)
            assert torch.equal(got, want)


def test_tokens_past_32_bit_offsets(handle):
    T, N, D, ld = 70000, 40, 64, 32771
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    dY = buf.as_strided((T, N), (ld, 1))
    dY.copy_(gradient(T, N, 1, "bf16"))
    X = kept(T, D, 2)
    got, want = torch.empty(N, D, device="cuda"), torch.empty(N, D, device="cuda")
    handle.mx8_weight_grad(dY, X, got)
    handle.mx8_weight_grad(dY.contiguous(), X, want)
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,N,D", [(1000, 100, 200), (100, 3600, 3600)])
def test_side_stream_and_graph(handle, T, N, D):
    X, dY = kept(T, D, 1), gradient(T, N, 2, "bf16").cuda()
    dW = torch.empty(N, D, device="cuda")
    handle.mx8_weight_grad(dY, X, dW)
    want = dW.clone()
    dW.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    handle.mx8_weight_grad(dY, X, dW, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(dW, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        handle.mx8_weight_grad(dY, X, dW)
    for _ in range(3):
        dY.copy_(torch.randn_like(dY))
        graph.replay()
        got = dW.clone()
        handle.mx8_weight_grad(dY, X, dW)
        assert torch.equal(got, dW)


def test_refusals(handle):
    X, dY = kept(4, 40, 1), gradient(4, 5, 2, "bf16").cuda()
    dW = torch.empty(5, 40, device="cuda")
    with pytest.raises(TypeError):
        handle.mx8_weight_grad(dY.float(), X, dW)
    with pytest.raises(TypeError):
        handle.mx8_weight_grad(dY, handle.mx4_quantize(dW), dW)
    with pytest.raises(ValueError):
        handle.mx8_weight_grad(dY[:3], X, dW)
    with pytest.raises(ValueError):
        handle.mx8_weight_grad(dY, X, dW[:, :32])
    with pytest.raises(TypeError):
        handle.mx8_weight_grad(dY, X, dW.double())
    with pytest.raises(ValueError):
        handle.mx8_weight_grad(dY.cpu(), X, dW)
