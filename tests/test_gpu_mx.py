"""Microscaled 4-bit quantisation and products on the GPU against the plain
64-bit implementation (mx_reference).

Codes and scales have to be equal, bit for bit.  A product may be off by
4*max(K,1)*2^-24*(|alpha|*sum|a*b| + |beta*c|): every matrix instruction rounds
once to 32 bits (2^-22 of its largest product and partial sum, at most K/64
times, and the waves' partial results are added by 32-bit additions), which is
far inside it; plus half a step of C's type on the result."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import mx_reference as ref  # noqa: E402

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle()
    yield h
    h.close()


def values(R, K, seed, spread=6):
    """Values whose blocks differ in magnitude by up to 2^(2*spread)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, K)) * np.exp2(rng.integers(-spread, spread + 1, (R, 1)))
    return x * np.exp2(rng.integers(-2, 3, (R, K)))


def strided(t, pad, fill=0):
    """A view of t's values inside rows that are `pad` elements longer."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]], buf


def as_numpy(q):
    return q.codes.cpu().numpy(), q.scales.cpu().numpy()


SIZES = [(1, 1), (1, 32), (2, 31), (3, 33), (16, 4096), (64, 256), (65, 777), (130, 2050),
         (257, 64), (1000, 100)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("R,K", SIZES)
def test_quantize(handle, R, K, trans, dt):
    x = torch.from_numpy(values(R, K, 7 * R + K)).to(DTYPES[dt])
    codes, scales = ref.quantize(x.double().numpy())
    stored = x.t().contiguous() if trans else x
    for pad in (0, 5):
        X, _ = strided(stored, pad, fill=float("nan"))
        nb = scales.shape[1]
        cbuf = torch.full((R, 16 * nb + 3), 0xA5, dtype=torch.uint8, device="cuda")
        sbuf = torch.full((R, nb + 1), 0xA5, dtype=torch.uint8, device="cuda")
        q = sg.Mx4(cbuf[:, :16 * nb], sbuf[:, :nb])
        handle.mx4_quantize(X, trans=trans, out=q)
        c, s = as_numpy(q)
        assert np.array_equal(s, scales)
        assert np.array_equal(c, codes)
        assert (cbuf[:, 16 * nb:] == 0xA5).all() and (sbuf[:, nb:] == 0xA5).all()
        Y, ybuf = strided(torch.zeros(R, K, dtype=x.dtype), 3, fill=1.5)
        handle.mx4_dequantize(q, Y)
        want = ref.dequantize(codes, scales)[:, :K]
        assert np.array_equal(Y.double().cpu().numpy(), want)
        assert (ybuf[:, K:] == 1.5).all()


@pytest.mark.parametrize("trans", [False, True])
def test_quantize_special_values(handle, trans):
    rows = []
    tiny = 2.0 ** -149
    for amax in (0.0, tiny, 5 * tiny, 2.0 ** -127, 2.0 ** -126, 3 * 2.0 ** -126, 2.0 ** -125, 1.0,
                 2.0 ** 126, 3.3e38, np.inf, -np.inf, np.nan):
        r = np.zeros(96)
        r[:32] = amax
        # ties and near ties of every pair of codes, in the middle block
        r[32:64] = np.resize([7.99, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5, -3.5, -2.5, -1.75, -1.25,
                              -0.75, -0.25, 6, 7, -7, 0.2499999, 0.2500001, -0.0], 32)
        r[64:] = np.linspace(-1, 1, 32) * (amax if np.isfinite(amax) else 1.0)
        r[70] = amax
        rows.append(r)
    x = np.stack(rows).astype(np.float32)
    codes, scales = ref.quantize(x.astype(np.float64))
    X = torch.from_numpy(x.T.copy() if trans else x).cuda()
    q = handle.mx4_quantize(X, trans=trans)
    c, s = as_numpy(q)
    assert np.array_equal(s, scales)
    assert np.array_equal(c, codes)
    Y = handle.mx4_dequantize(q, torch.empty(x.shape, device="cuda"))
    assert np.array_equal(Y.cpu().numpy(), ref.dequantize(codes, scales), equal_nan=True)


def test_dequantize_fewer_columns(handle):
    x = torch.from_numpy(values(5, 96, 3)).float()
    q = handle.mx4_quantize(x.cuda())
    full = ref.dequantize(*as_numpy(q))
    for K in (1, 8, 31, 33, 64, 95, 96):
        Y = handle.mx4_dequantize(q, torch.empty(5, K, device="cuda"))
        assert np.array_equal(Y.cpu().numpy(), full[:, :K])


def test_quantize_past_32_bit_offsets(handle):
    # the last rows start past 2^32 bytes
    R, K, ld = 70000, 40, 32771
    buf = torch.empty(R * ld, dtype=torch.bfloat16, device="cuda")
    X = buf.as_strided((R, K), (ld, 1))
    X.copy_(torch.from_numpy(values(R, K, 5)))
    q = handle.mx4_quantize(X)
    at = torch.tensor([0, 1, 32767, 32768, 65537, R - 1])
    codes, scales = ref.quantize(X[at.cuda()].double().cpu().numpy())
    c, s = as_numpy(q)
    assert np.array_equal(c[at], codes) and np.array_equal(s[at], scales)
    Y = handle.mx4_dequantize(q, X)
    assert np.array_equal(Y[at.cuda()].double().cpu().numpy(), ref.dequantize(codes, scales)[:, :K])


# ---- products -------------------------------------------------------------------

def operand(R, K, seed):
    codes, scales = ref.quantize(values(R, K, seed, spread=3))
    return sg.Mx4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda())


def half_step(dt):
    return torch.finfo(DTYPES[dt]).eps / 2


def check(got, a, b, K, alpha, beta, c, dt, what=""):
    r, t = ref.product(alpha, a, b, beta, c)
    bound = 4 * max(K, 1) * 2.0 ** -24 * t
    if dt != "f32":
        bound = bound + half_step(dt) * (np.abs(r) + bound)
        if dt == "f16":
            bound = bound + 2.0 ** -25  # half a step of the subnormal numbers
    err = np.abs(got.astype(np.float64) - r)
    assert np.all(err <= bound), (what, float((err - bound).max()), np.argwhere(err > bound)[:3])


PRODUCTS = [(1, 1, 32), (1, 16, 64), (1, 4096, 4096), (2, 17, 96), (4, 100, 512), (16, 333, 4096),
            (17, 40, 544), (33, 65, 32), (64, 64, 256), (100, 128, 1056), (128, 256, 800),
            (200, 300, 160), (256, 512, 512), (257, 511, 288), (1000, 1500, 800),
            # enough tiles for the 128-square and the 256-square ones, K of less
            # than a step, of whole steps (odd and even counts) and ragged
            (2050, 2100, 64), (2050, 2100, 256), (2048, 2176, 1024), (2050, 2100, 1312),
            (2900, 3050, 96), (2900, 3050, 256), (2816, 3328, 512), (2900, 3050, 1568)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("dt,alpha,beta", [("f32", 1.0, 0.0), ("f32", 1.5, 0.5), ("bf16", 1.0, 0.0),
                                           ("bf16", 0.75, 1.0), ("f16", 0.125, 0.0)])
def test_product(handle, M, N, K, dt, alpha, beta):
    A, B = operand(M, K, 11 * M + K), operand(N, K, 13 * N + K)
    a, b = ref.dequantize(*as_numpy(A)), ref.dequantize(*as_numpy(B))
    c0 = torch.from_numpy(np.random.default_rng(M + N).standard_normal((M, N)) * 4).to(DTYPES[dt])
    if beta == 0.0:
        c0.fill_(float("nan"))  # C is not read
    outs = []
    for pad in (0, 3):
        C, buf = strided(c0, pad, fill=7.0)
        handle.gemm_mx4(A, B, C, alpha=alpha, beta=beta)
        c = c0.double().numpy() if beta else None
        check(C.float().cpu().numpy(), a, b, K, alpha, beta, c, dt, (M, N, K, pad))
        assert (buf[:, N:] == 7.0).all()
        outs.append(C.clone())
    assert torch.equal(outs[0], outs[1])  # same bits, whatever C's stride


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("M,N,K", [(1, 100, 33), (1, 4096, 4096), (2, 40, 1), (3, 70, 5000),
                                   (4, 33, 8192), (5, 90, 512), (7, 64, 777), (16, 50, 1024),
                                   (17, 64, 100), (40, 200, 4090), (300, 260, 520)])
def test_product_of_activations(handle, M, N, K, dt):
    x = torch.from_numpy(values(M, K, M + K, spread=2)).to(DTYPES[dt])
    X, _ = strided(x, 7, fill=float("nan"))
    B = operand(N, K, N)
    two, one = (torch.full((M, N), float("nan"), device="cuda") for _ in range(2))
    handle.gemm_mx4(handle.mx4_quantize(X), B, two)
    handle.gemm_mx4(X, B, one)
    assert torch.equal(one, two)
    a = ref.dequantize(*ref.quantize(x.double().numpy()))
    check(one.cpu().numpy(), a, ref.dequantize(*as_numpy(B)), B.K, 1.0, 0.0, None, "f32")


def test_integer_products_are_exact(handle):
    # one scale for all blocks: every product is a multiple of 1/4, every sum exact
    rng = np.random.default_rng(2)
    for M, N, K in ((5, 70, 2048), (130, 190, 1056)):
        q = [sg.Mx4(torch.from_numpy(rng.integers(0, 256, (R, K // 2), dtype=np.uint8)).cuda(),
                    torch.full((R, K // 32), 127, dtype=torch.uint8, device="cuda")) for R in (M, N)]
        C = torch.empty(M, N, device="cuda")
        handle.gemm_mx4(*q, C)
        a, b = (ref.dequantize(*as_numpy(t)) for t in q)
        assert np.array_equal(C.cpu().numpy(), a @ b.T)


@pytest.mark.parametrize("M,N,K", [(3, 40, 544), (70, 150, 544)])
def test_nan_block_stays_in_its_row_and_column(handle, M, N, K):
    A, B = operand(M, K, 1), operand(N, K, 2)
    A.scales[1, K // 32 - 1] = 255
    B.scales[17, 0] = 255
    C = torch.empty(M, N, device="cuda")
    handle.gemm_mx4(A, B, C)
    nan = np.zeros((M, N), bool)
    nan[1], nan[:, 17] = True, True
    got = C.cpu().numpy()
    assert np.array_equal(np.isnan(got), nan)
    a, b = ref.dequantize(*as_numpy(A)), ref.dequantize(*as_numpy(B))
    keep_m, keep_n = [m for m in range(M) if m != 1], [n for n in range(N) if n != 17]
    check(got[np.ix_(keep_m, keep_n)], a[keep_m], b[keep_n], K, 1.0, 0.0, None, "f32")


@pytest.mark.parametrize("M,N,K", [(4, 33, 96), (100, 70, 1056)])
def test_operands_inside_wider_buffers(handle, M, N, K):
    """Odd strides, and bytes around the operands that must not be read into
    the result (scale bytes of 255 behind every row)."""
    A, B = operand(M, K, 3), operand(N, K, 4)
    want = torch.empty(M, N, device="cuda")
    handle.gemm_mx4(A, B, want)
    wide = []
    for q in (A, B):
        c = torch.full((q.rows, K // 2 + 37), 0xFF, dtype=torch.uint8, device="cuda")
        s = torch.full((q.rows, K // 32 + 5), 0xFF, dtype=torch.uint8, device="cuda")
        c[:, 1:1 + K // 2] = q.codes
        s[:, 1:1 + K // 32] = q.scales
        wide.append(sg.Mx4(c[:, 1:1 + K // 2], s[:, 1:1 + K // 32]))
    got = torch.empty(M, N, device="cuda")
    handle.gemm_mx4(*wide, got)
    assert torch.equal(got, want)


def test_empty_and_k_zero(handle):
    for M, N in ((0, 5), (5, 0)):
        handle.gemm_mx4(sg.Mx4.empty(M, 64), sg.Mx4.empty(N, 64), torch.empty(M, N, device="cuda"))
    C = torch.ones(3, 4, device="cuda")
    handle.gemm_mx4(sg.Mx4.empty(3, 0), sg.Mx4.empty(4, 0), C, beta=2.0)
    assert (C == 2).all()
    handle.gemm_mx4(torch.empty(3, 0, device="cuda"), sg.Mx4.empty(4, 0), C)
    assert (C == 0).all()
    q = handle.mx4_quantize(torch.empty(0, 64, device="cuda"))
    handle.mx4_dequantize(q, torch.empty(0, 64, device="cuda"))


@pytest.mark.parametrize("M", [3, 40])
def test_operand_past_32_bit_offsets(handle, M):
    N, K = 70000, 131072  # 4.6 GB of codes
    B = sg.Mx4.empty(N, K)
    B.codes.random_(0, 256)
    B.scales.fill_(120)
    A = operand(M, K, 6)
    C = torch.empty(M, N, device="cuda")
    handle.gemm_mx4(A, B, C)
    at = torch.tensor([0, 1, 65535, 65536, N - 2, N - 1])
    a = ref.dequantize(*as_numpy(A))
    b = ref.dequantize(B.codes[at.cuda()].cpu().numpy(), B.scales[at.cuda()].cpu().numpy())
    check(C[:, at.cuda()].cpu().numpy(), a, b, K, 1.0, 0.0, None, "f32")


def test_calls_on_two_handles_overlap():
    """Calls that use a workspace, on two streams at once: each handle its own."""
    B = operand(512, 1024, 8)
    X = [torch.from_numpy(values(60, 1024, 30 + k, spread=2)).bfloat16().cuda() for k in range(2)]
    with sg.Handle() as one, sg.Handle() as two:
        want = [torch.empty(60, 512, device="cuda") for _ in range(2)]
        for k in range(2):
            one.gemm_mx4(X[k], B, want[k])
        got = [torch.empty_like(w) for w in want]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(50):
            for h, s, x, c in zip((one, two), streams, X, got):
                h.gemm_mx4(x, B, c, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("K", [0, 32])
def test_more_rows_than_a_grid_extent_holds(handle, K):
    M = 65535 * 16 + 40
    A, B = sg.Mx4.empty(M, K), operand(2, 32, 3) if K else sg.Mx4.empty(2, 0)
    rng = np.random.default_rng(0)
    if K:
        A.codes.copy_(torch.from_numpy(rng.integers(0, 256, (M, 16), dtype=np.uint8)))
        A.scales.fill_(127)
    C = torch.ones(M, 2, device="cuda")
    handle.gemm_mx4(A, B, C, beta=0.5)
    a, b = (ref.dequantize(*as_numpy(q)) for q in (A, B))
    want, mag = ref.product(1.0, a, b, 0.5, np.ones((M, 2)))
    assert np.all(np.abs(C.double().cpu().numpy() - want) <= 4 * max(K, 1) * 2.0 ** -24 * mag)


@pytest.mark.parametrize("M,N,K", [(64, 4096, 8192), (33, 3000, 8224), (17, 8190, 8704)])
def test_rows_of_a_long_k(handle, M, N, K):
    """17 to 64 rows straight from memory, four tiles of columns a workgroup."""
    A, B = operand(M, K, 4), operand(N, K, 5)
    C, buf = strided(torch.zeros(M, N), 3, fill=7.0)
    handle.gemm_mx4(A, B, C)
    check(C.cpu().numpy(), ref.dequantize(*as_numpy(A)), ref.dequantize(*as_numpy(B)), K, 1.0, 0.0, None,
          "f32")
    assert (buf[:, N:] == 7.0).all()


@pytest.mark.parametrize("M,N,K,far", [(70, 2100, 96, "A"), (2100, 70, 544, "B")])
def test_rows_past_a_tiles_offsets(handle, M, N, K, far):
    """Rows so far apart that a tile's lie more than 4 GiB from its first: the
    kernel that loads straight from memory takes them."""
    A, B = operand(M, K, 6), operand(N, K, 7)
    q = A if far == "A" else B
    ld = (1 << 32) // 63 + 5  # (a 64-row tile's last row)
    rows = torch.empty((q.rows - 1) * ld + K // 2, dtype=torch.uint8, device="cuda")
    codes = rows.as_strided((q.rows, K // 2), (ld, 1))
    codes.copy_(q.codes)
    wide = sg.Mx4(codes, q.scales)
    C = torch.full((M, N), 7.0, device="cuda")
    handle.gemm_mx4(wide if far == "A" else A, wide if far == "B" else B, C)
    check(C.cpu().numpy(), ref.dequantize(*as_numpy(A)), ref.dequantize(*as_numpy(B)), K, 1.0, 0.0, None,
          "f32")


@pytest.mark.parametrize("M", [1, 20])
def test_more_columns_than_a_grid_extent_holds(handle, M):
    """2^27 and more rows of B: a launch of 16 columns a workgroup holds 2^27 - 16."""
    N, K = (1 << 27) + 100, 32
    A, B = operand(M, K, 3), sg.Mx4.empty(N, K)
    B.codes.random_(0, 256)
    B.scales.fill_(127)
    C = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    handle.gemm_mx4(A, B, C)
    at = torch.tensor([0, 1, (1 << 27) - 18, (1 << 27) - 17, (1 << 27) - 16, (1 << 27) - 15, (1 << 27) - 1,
                       1 << 27, N - 2, N - 1])
    b = ref.dequantize(B.codes[at.cuda()].cpu().numpy(), B.scales[at.cuda()].cpu().numpy())
    check(C[:, at.cuda()].float().cpu().numpy(), ref.dequantize(*as_numpy(A)), b, K, 1.0, 0.0, None,
          "bf16")


def test_refusals(handle):
    A, B = operand(20, 64, 1), operand(5, 64, 2)
    C = torch.empty(20, 5, device="cuda")
    with pytest.raises(ValueError):
        handle.gemm_mx4(A, B, torch.empty(5, 20, device="cuda"))
    with pytest.raises(ValueError):
        handle.gemm_mx4(A, operand(5, 96, 2), C)
    with pytest.raises(ValueError):
        handle.gemm_mx4(A, B, torch.empty(20, 5))
    with pytest.raises(TypeError):
        handle.gemm_mx4(A, B, C.double())
    with pytest.raises(ValueError):
        handle.mx4_quantize(torch.empty(3, 64, device="cuda"), out=A)
    with pytest.raises(ValueError):
        handle.mx4_dequantize(A, torch.empty(20, 65, device="cuda"))
    with sg.Handle(workspace=False) as bare:
        X = torch.randn(20, 64, device="cuda")
        with pytest.raises(sg.SgemmError) as e:
            bare.gemm_mx4(X, B, C)
        assert e.value.status == sg.SGEMM_ERR_SCRATCH
        for m in (3, 5, 16):  # up to 16 rows need none
            want = torch.empty(m, 5, device="cuda")
            handle.gemm_mx4(X[:m], B, want)
            bare.gemm_mx4(X[:m], B, C[:m])
            assert torch.equal(C[:m], want)


@pytest.mark.parametrize("M,N,K", [(1, 256, 1024), (40, 100, 800)])
def test_graph_and_stream(handle, M, N, K):
    """Captured and replayed with eager work in between, and on another
    stream: the eager call's bits every time."""
    B = operand(N, K, 5)
    X = torch.from_numpy(values(M, K, 9, spread=2)).to(torch.bfloat16).cuda()
    C, Y = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    q = sg.Mx4.empty(M, K)

    def work():
        handle.mx4_quantize(X, out=q)
        handle.mx4_dequantize(q, Y)
        handle.gemm_mx4(X, B, C)

    work()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        work()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            work()
    torch.cuda.synchronize()
    for k in range(4):
        X.copy_(torch.from_numpy(values(M, K, 20 + k, spread=2)))
        want = torch.empty_like(C)
        handle.gemm_mx4(handle.mx4_quantize(X), B, want)
        torch.cuda.synchronize()
        C.fill_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)
        assert np.array_equal(Y.float().cpu().numpy(), ref.dequantize(*as_numpy(q))[:, :K])
        with torch.cuda.stream(s):
            C.fill_(-1.0)
            handle.gemm_mx4(handle.mx4_quantize(X), B, C)
        s.synchronize()
        assert torch.equal(C, want)
