"""Products of microscaled 8-bit rows on the GPU against the plain 64-bit
implementation.

A product may be off by 4*max(K,1)*2^-24*(|alpha|*sum|a*b| + |beta*c|) for its
32-bit sums; by the matrix instruction's own sums of 8-bit operands, 2^-9*|alpha|
times the largest |a*b| of every run of 64 (the library's allowance for that
instruction, of which at most a quarter was measured); and by half a step of C's
type.  Integers within the instruction's window are exact."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx8_reference as ref  # noqa: E402
from tests import mx_reference as ref4  # noqa: E402
from tests.test_gpu_mx import DTYPES, as_numpy, half_step, strided, values  # noqa: E402


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


def operand(R, K, seed, bits=8):
    module, kind = (ref, sg.Mx8) if bits == 8 else (ref4, sg.Mx4)
    codes, scales = module.quantize(values(R, K, seed, spread=3))
    return kind(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def numbers(q):
    return (ref if isinstance(q, sg.Mx8) else ref4).dequantize(*as_numpy(q))


def largest(x):
    """The largest magnitude of every run of 64 of the columns."""
    x = np.abs(x)
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % 64)))
    return x.reshape(x.shape[0], -1, 64).max(-1)


def check(got, a, b, alpha, beta, c, dt, what=""):
    K = a.shape[1]
    r, t = ref4.product(alpha, a, b, beta, c)
    bound = 4 * max(K, 1) * 2.0 ** -24 * t + 2.0 ** -9 * abs(alpha) * (largest(a) @ largest(b).T)
    if dt != "f32":
        bound = bound + half_step(dt) * (np.abs(r) + bound)
        if dt == "f16":
            bound = bound + 2.0 ** -25
    err = np.abs(got.double().cpu().numpy() - r)
    assert np.all(err <= bound), (what, float((err - bound).max()), np.argwhere(err > bound)[:3])


PRODUCTS = [(1, 1, 32), (1, 16, 64), (1, 4096, 4096), (2, 17, 96), (4, 100, 512), (16, 333, 4096),
            (17, 40, 544), (33, 65, 32), (64, 64, 256), (100, 128, 1056), (128, 256, 800),
            (200, 300, 160), (256, 512, 512), (257, 511, 288), (1000, 1500, 800), (300, 5000, 96),
            (700, 900, 64), (700, 900, 32), (700, 900, 128), (700, 900, 352),
            (5, 16500, 544), (16, 13000, 2112), (700, 900, 1056), (640, 832, 2048), (650, 840, 1632), (300, 70, 2048), (40, 500, 5000 // 32 * 32),
            # enough tiles for the 128-square and the 256-square ones, K of less
            # than a step, of whole steps (odd and even counts) and ragged
            (2050, 2100, 32), (2050, 2100, 64), (2050, 2100, 160), (2050, 2100, 224), (2050, 2100, 128), (2048, 2176, 1024), (2050, 2100, 1312),
            (2900, 3050, 32), (2900, 3050, 96), (2900, 3050, 160), (2900, 3050, 544), (2900, 3050, 256), (2816, 3328, 512), (2900, 3050, 1568), (2900, 3050, 1184)]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(handle, M, N, K, bits):
    A, B = operand(M, K, 11 * M + K), operand(N, K, 13 * N + K, bits)
    a, b = numbers(A), numbers(B)
    for dt, alpha, beta in (("bf16", 1.0, 0.0), ("f32", 1.5, 0.5), ("f16", 0.125, 0.0), ("bf16", 0.75, 1.0)):
        c0 = torch.from_numpy(np.random.default_rng(M + N).standard_normal((M, N)) * 4).to(DTYPES[dt])
        if beta == 0.0:
            c0.fill_(float("nan"))  # C is not read
        outs = []
        for pad in (0, 3):
            C, buf = strided(c0, pad, fill=7.0)
            handle.gemm_mx8(A, B, C, alpha=alpha, beta=beta)
            check(C, a, b, alpha, beta, c0.double().numpy() if beta else None, dt, (M, N, K, pad))
            assert (buf[:, N:] == 7.0).all()
            outs.append(C.clone())
        assert torch.equal(*outs)  # same bits, whatever C's stride
        if M * N > 10 ** 6:
            break


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(1, 70, 2048), (3, 100, 96), (16, 4200, 512), (130, 190, 1056), (130, 190, 96),
                                   (700, 900, 608), (2900, 3050, 416)])
def test_integer_products_are_exact(handle, M, N, K, bits):
    """Whole numbers from -4 to 4 with scales of one and two: every code, place
    and scale byte counts, and every sum is exact."""
    rng = np.random.default_rng(M + K)
    ops = []
    for R, b in ((M, 8), (N, bits)):
        v = rng.integers(-4, 5, (R, K))
        s = rng.integers(127, 129, (R, K // 32)).astype(np.uint8)
        if b == 8:
            codes = np.searchsorted(ref.GRID, np.abs(v)).astype(np.uint8) | np.where(v < 0, 128, 0).astype(np.uint8)
            q = sg.Mx8(torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda())
        else:
            c = np.searchsorted(ref4.GRID, np.abs(v)).astype(np.uint8) | np.where(v < 0, 8, 0).astype(np.uint8)
            q = sg.Mx4(torch.from_numpy(c[:, 0::2] | (c[:, 1::2] << 4)).cuda(), torch.from_numpy(s).cuda())
        assert np.array_equal(numbers(q), v * np.repeat(np.exp2(s - 127.0), 32, axis=1))
        ops.append(q)
    C = torch.empty(M, N, device="cuda")
    handle.gemm_mx8(*ops, C)
    assert np.array_equal(C.double().cpu().numpy(), numbers(ops[0]) @ numbers(ops[1]).T)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("M,N,K", [(1, 100, 33), (1, 4096, 4096), (2, 40, 1), (3, 70, 5000), (4, 33, 8192),
                                   (4, 9000, 100), (5, 90, 512), (7, 64, 777), (16, 50, 1024), (17, 64, 100),
                                   (40, 200, 4090), (300, 260, 520), (2, 17000, 1000), (3, 13000, 2100)])
def test_product_of_activations(handle, M, N, K, dt, bits):
    x = torch.from_numpy(values(M, K, M + K, spread=2)).to(DTYPES[dt])
    X, _ = strided(x, 7, fill=float("nan"))
    B = operand(N, K, N, bits)
    two, one = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    handle.gemm_mx8(handle.mx8_quantize(X), B, two)
    handle.gemm_mx8(X, B, one)
    assert torch.equal(one, two)
    check(one, ref.dequantize(*ref.quantize(x.double().numpy())), numbers(B), 1.0, 0.0, None, "f32")


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(3, 40, 544), (70, 150, 544), (700, 900, 352), (700, 900, 96)])
def test_nan_stays_in_its_row_and_column(handle, M, N, K, bits):
    """A block of scale 255 and (8 bits) a NaN code make their row or column NaN,
    in the last block of a row too, and nothing else."""
    A, B = operand(M, K, 1), operand(N, K, 2, bits)
    A.scales[1, -1] = 255
    A.codes[2, 5] = 0x7F
    B.scales[N // 2, K // 64] = 255
    if bits == 8:
        B.codes[N - 1, K - 1] = 0xFF
    C = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    handle.gemm_mx8(A, B, C)
    nan = torch.zeros(M, N, dtype=torch.bool)
    nan[1], nan[2], nan[:, N // 2] = True, True, True
    if bits == 8:
        nan[:, N - 1] = True
    assert torch.equal(torch.isnan(C).cpu(), nan)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M,N,K", [(4, 33, 96), (100, 70, 1056), (300, 700, 608)])
def test_operands_inside_wider_buffers(handle, M, N, K, bits):
    """Odd byte strides and addresses; what surrounds the rows is never used."""
    A, B = operand(M, K, 1), operand(N, K, 2, bits)
    want = torch.empty(M, N, device="cuda")
    handle.gemm_mx8(A, B, want)

    def inside(t, pad):
        buf = torch.full((t.shape[0] + 1, t.shape[1] + pad), 255, dtype=torch.uint8, device="cuda")
        view = buf.view(-1)[3:3 + t.shape[0] * buf.shape[1]].view(t.shape[0], -1)[:, :t.shape[1]]
        view.copy_(t)
        return view

    A2 = sg.Mx8(inside(A.codes, 5), inside(A.scales, 3))
    B2 = type(B)(inside(B.codes, 7), inside(B.scales, 4))
    got = torch.empty(M, N, device="cuda")
    handle.gemm_mx8(A2, B2, got)
    assert torch.equal(got, want)


def test_empty_and_k_zero(handle):
    for M, N in ((0, 5), (5, 0)):
        handle.gemm_mx8(sg.Mx8.empty(M, 64), sg.Mx8.empty(N, 64), torch.empty(M, N, device="cuda"))
    for M in (3, 100):
        C = torch.full((M, 40), 2.0, device="cuda")
        handle.gemm_mx8(sg.Mx8.empty(M, 0), sg.Mx8.empty(40, 0), C, beta=0.5)
        assert (C == 1.0).all()
        C.fill_(float("nan"))
        handle.gemm_mx8(torch.empty(M, 0, device="cuda"), sg.Mx4.empty(40, 0), C)
        assert (C == 0.0).all()


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("M", [3, 300])
def test_rows_past_32_bit_offsets(handle, M, bits):
    # B's last rows start past 2^32 bytes of its buffer; strides past a tile's
    # 32-bit offsets take the kernel without tiles
    N, K = 600, 288
    A, B = operand(M, K, 1), operand(N, K, 2, bits)
    for ld in (1 << 23, 1 << 25):
        rows = min(N, (1 << 33) // ld + 70)
        buf = torch.empty(rows * ld, dtype=torch.uint8, device="cuda")
        codes = buf.as_strided((rows, B.codes.shape[1]), (ld, 1))
        codes.copy_(B.codes[:rows])
        got, want = (torch.empty(M, rows, device="cuda") for _ in range(2))
        handle.gemm_mx8(A, type(B)(codes, B.scales[:rows]), got)
        handle.gemm_mx8(A, type(B)(B.codes[:rows].contiguous(), B.scales[:rows].contiguous()), want)
        tol = 2.0 ** -9 * (largest(numbers(A)) @ largest(numbers(B)[:rows]).T)  # (kernels may differ)
        assert (np.abs((got - want).cpu().numpy()) <= tol).all()
        del buf, codes


def test_workspace(handle):
    X, B = torch.randn(40, 200, device="cuda"), operand(30, 200, 1)
    C = torch.empty(40, 30, device="cuda")
    with sg.Handle(workspace=False) as own:
        own.gemm_mx8(X[:4], B, C[:4])
        with pytest.raises(sg.SgemmError) as e:
            own.gemm_mx8(X, B, C)
        assert e.value.status == sg.SGEMM_ERR_SCRATCH
        own.set_workspace(sg.Mx8.nbytes(40, 200) - 1)
        with pytest.raises(sg.SgemmError):
            own.gemm_mx8(X, B, C)
        own.set_workspace(sg.Mx8.nbytes(40, 200))
        own.gemm_mx8(X, B, C)
        own.gemm_mx8(X, B, C, beta=1.0)
    handle.gemm_mx8(X, B, C, beta=0.0)
    want = torch.empty_like(C)
    handle.gemm_mx8(handle.mx8_quantize(X), B, want)
    assert torch.equal(C, want)


@pytest.mark.parametrize("M", [1, 16, 300])
def test_side_stream_and_graph(handle, M):
    X, B = torch.randn(M, 1000, device="cuda", dtype=torch.bfloat16), operand(500, 1000, 1)
    C = torch.empty(M, 500, device="cuda", dtype=torch.bfloat16)
    handle.gemm_mx8(X, B, C)
    want = C.clone()
    C.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    handle.gemm_mx8(X, B, C, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(C, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        handle.gemm_mx8(X, B, C)
    for _ in range(3):
        X.copy_(torch.randn_like(X))
        graph.replay()
        got = C.clone()
        handle.gemm_mx8(X, B, C)
        assert torch.equal(got, C)


def test_refusals(handle):
    A, B, B4 = operand(4, 64, 1), operand(5, 64, 2), operand(5, 64, 3, 4)
    C = torch.empty(4, 5, device="cuda")
    with pytest.raises(ValueError):
        handle.gemm_mx8(A, operand(5, 96, 1), C)
    with pytest.raises(ValueError):
        handle.gemm_mx8(A, B, C[:3])
    with pytest.raises(TypeError):
        handle.gemm_mx8(B4, B, C)
    with pytest.raises(TypeError):
        handle.gemm_mx8(A, C, C)
    with pytest.raises(TypeError):
        handle.gemm_mx4(A, B4, C)
    with pytest.raises(TypeError):
        handle.gemm_mx4(B4, B, C)
    with pytest.raises(TypeError):
        handle.gemm_mx8(A, B, C.double())
    with pytest.raises(ValueError):
        handle.gemm_mx8(A, B, C.cpu())
    with pytest.raises(sg.SgemmError):
        handle.gemm_mx8(A, B, A.codes.view(torch.float32)[:, :5])
