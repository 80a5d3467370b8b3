"""Words that a mask takes out of the output layer's loss, and other infinite
logits, on the GPU against the plain 64-bit implementation (ce_reference).

A mask is a column of W that meets a constant column of X: -inf (or, with a
negative alpha, +inf) or the type's lowest value where a word is out, else 0.
Such a word adds nothing to lse, so the reference takes -1e4 in its place,
whose exponential is 0 in 64 bits, and the bounds are those of the other loss
tests.  (dX's column of the mask is the sum of 0 * -inf: NaN.)"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import fp32_gemm_major_amd as sg  # noqa: E402
from tests import ce_reference as ref  # noqa: E402
from tests.test_gpu_ce import DTYPES, U, Problem  # noqa: E402


@pytest.fixture(scope="module")
def handle():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    h = sg.Handle(workspace=False)
    h.set_workspace(1 << 30)
    yield h
    h.close()


def masked(T, V, D, dt, words, value, column=0, alpha=0.5, seed=0, pad=0):
    """A problem whose `words` are out, labels elsewhere; value: "inf" or "lowest"."""
    p = Problem(T, V, D, dt, seed=seed, ignored=0.1, alpha=alpha, pad=pad)
    out = np.zeros(V, bool)
    out[words] = True
    left = np.flatnonzero(~out)
    hit = (p.labels != ref.IGNORE) & out[np.maximum(p.labels, 0)]
    p.labels[hit] = left[p.labels[hit] % len(left)]
    p.Y.copy_(torch.from_numpy(p.labels))
    p.x[:, column], p.w[:, column] = 1.0, 0.0
    sign = -1.0 if alpha > 0 else 1.0
    p.w[out, column] = sign * 1e4
    size = float("inf") if value == "inf" else torch.finfo(DTYPES[dt]).max
    p.X[:, column] = 1.0
    p.W[:, column] = 0.0
    p.W[torch.from_numpy(out).cuda(), column] = sign * size
    p.column, p.infinite = column, value == "inf"
    return p


def check(p, handle):
    p.forward(handle)
    p.check_forward()
    p.backward(handle)
    if p.infinite:
        kept = p.Y != ref.IGNORE
        assert torch.isnan(p.dX[kept, p.column]).all()
        p.dX[kept, p.column] = 0.0
    if p.alpha < 0:  # the same problem with -X and -alpha (check_backward's bounds grow with alpha)
        p.alpha, p.x = -p.alpha, -p.x
        p.dX.neg_()
    p.check_backward()


def runs(V):
    """Sets of words: aligned runs of every reduction's width, ragged ones,
    a vocabulary's padding, every word but one."""
    return {"4": np.arange(8, 12), "64": np.arange(64, 128), "128": np.arange(128, 256),
            "ragged": np.arange(3, 301), "half": np.arange(0, V, 2), "end": np.arange(V - 270, V),
            "but one": np.delete(np.arange(V), V // 3)}


# Over the library's products (up to 16 rows; 32-bit up to 511 rows or few
# tiles): statistics a row.
@pytest.mark.parametrize("value", ["inf", "lowest"])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("words", ["4", "64", "128", "ragged", "half", "end", "but one"])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_masked_words_few_rows(handle, T, words, dt, value):
    V = 18000 if words == "128" else 1300
    check(masked(T, V, 48, dt, runs(V)[words], value), handle)


@pytest.mark.parametrize("value", ["inf", "lowest"])
@pytest.mark.parametrize("words", ["4", "ragged", "but one"])
def test_masked_words_32_bit_library_products(handle, words, value):
    check(masked(90, 1300, 48, "f32", runs(1300)[words], value), handle)


def test_negative_scale_few_rows(handle):
    for dt in DTYPES:
        check(masked(7, 1300, 48, dt, np.arange(3, 301), "inf", alpha=-0.5), handle)
        check(masked(7, 1300, 48, dt, np.arange(3, 301), "lowest", alpha=-0.5), handle)


# Packed rows: parts of 64 and 128 words a wave.
@pytest.mark.parametrize("value", ["inf", "lowest"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("words", ["4", "64", "128", "ragged", "half", "end", "but one"])
@pytest.mark.parametrize("T,D", [(40, 64), (300, 128)])
def test_masked_words_packed_rows(handle, T, D, words, dt, value):
    check(masked(T, 1300, D, dt, runs(1300)[words], value), handle)


@pytest.mark.parametrize("words", ["4", "64", "128", "end", "but one"])
def test_masked_words_big_tiles(handle, words):
    check(masked(300, 20000, 64, "bf16", runs(20000)[words], "inf"), handle)


@pytest.mark.parametrize("words", ["64", "128", "ragged", "but one"])
def test_lowest_words_in_planes(handle, words):
    check(masked(600, 13200, 264, "f32", runs(13200)[words], "lowest"), handle)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_negative_scale_packed_rows(handle, dt):
    for value in ("inf", "lowest"):
        check(masked(40, 1300, 64, dt, np.arange(3, 301), value, alpha=-0.5), handle)


PATHS = [(5, 900, 40, "bf16"), (5, 900, 40, "f16"), (5, 900, 40, "f32"), (90, 900, 40, "f32")]
PACKED = [(40, 900, 64, "bf16"), (40, 900, 64, "f16"), (300, 20000, 64, "bf16")]
PLANES = [(600, 13200, 64, "f32"), (4200, 8200, 520, "f32")]  # (forward; both)


@pytest.mark.parametrize("T,V,D,dt", PATHS + PACKED + PLANES)
def test_no_word_left(handle, T, V, D, dt):
    """Every word at the type's lowest value: lse is it (as far as 32 bits hold
    it), the loss the logarithm of V where the others' part of the logits is
    lost beside it, and every gradient finite but where the sums leave the type;
    at -inf: lse is -inf, the loss NaN."""
    p = masked(T, V, D, dt, np.arange(V - 1), "lowest", seed=2)
    low = torch.finfo(DTYPES[dt]).min
    p.w[:, 0] = low
    p.W[:, 0] = low
    p.forward(handle)
    keep = p.labels != ref.IGNORE
    if dt == "f16":
        p.check_forward()
    else:
        for one in (1.0, 1.0 - 5 * 2.0 ** -7):  # (x w itself is in range)
            p.X[:, 0] = one
            p.forward(handle)
            got = p.lse.double().cpu().numpy()[keep]
            assert np.all(np.abs(got - 0.5 * one * low) <= 4 * U * abs(low)), got[:4]
            got = p.loss.double().cpu().numpy()[keep]
            assert np.all(np.abs(got - np.log(V)) <= p.sum_error() + 8 * U * np.log(V)), got[:4]
    p.backward(handle)
    assert not torch.isnan(p.dW[:, 1:]).any()
    p.W[:, 0] = float("-inf")
    p.forward(handle)
    assert (p.lse.cpu().numpy()[keep] == -np.inf).all()
    assert torch.isnan(p.loss).cpu().numpy()[keep].all()
    assert (p.loss.cpu().numpy()[~keep] == 0).all() and (p.lse.cpu().numpy()[~keep] == 0).all()


@pytest.mark.parametrize("T,V,D,dt", [a for a in PATHS + PACKED if a[3] != "f16"] + PLANES)
def test_gradients_where_no_word_is_left(T, V, D, dt):
    """Logits and lse at the type's lowest value, whose product with log2(e)
    leaves 32 bits: their difference is 0 and exp(z - lse) is 1, so dz is
    dloss + dlse less dloss at the label, off by its rounding to 16 bits."""
    p = masked(T, V, D, dt, np.arange(V - 1), "lowest", alpha=1.0, seed=2)
    p.W[:, 0] = torch.finfo(DTYPES[dt]).min
    with sg.Handle(workspace=False) as h:
        h.set_workspace(max(h.ce_workspace_size(p.X, p.W, backward=b) for b in (False, True)))
        p.forward(h)
        p.backward(h)
    keep = p.labels != ref.IGNORE
    dz = ref.dlogits(np.zeros((T, V)), p.labels, np.zeros(T), p.dloss, p.dlse)
    dx, dw = ref.gradients(p.x, p.w, p.labels, dz)
    half = torch.finfo(DTYPES[dt]).eps / 2
    ez = (half + 4 * U) * np.abs(dz)
    ax, aw = np.abs(np.where(keep[:, None], p.x, 0.0)), np.abs(p.w)
    for got, want, err, mag in ((p.dX, dx, ez @ aw, 4 * V * U * (np.abs(dz) @ aw)),
                                (p.dW, dw, ez.T @ ax, 4 * T * U * (np.abs(dz).T @ ax))):
        bound = err + mag
        bound = bound + half * (np.abs(want) + bound) + 4 * U * np.abs(want)
        off = np.abs(got.double().cpu().numpy() - want)[:, 1:]
        assert np.all(off <= bound[:, 1:]), np.nanmax(off - bound[:, 1:])

@pytest.mark.parametrize("T,V,D,dt", PATHS + PACKED + PLANES)
def test_infinite_and_nan_logits(handle, T, V, D, dt):
    """One word at +inf: lse is +inf, and the loss but for rows labelled with
    that word (inf - inf).  A label at -inf costs +inf.  One word at NaN:
    everything is."""
    p = masked(T, V, D, dt, [V // 2], "inf", seed=3)
    p.labels[:] = np.arange(T) % 5
    p.labels[1] = V // 2
    p.labels[3] = ref.IGNORE
    p.Y.copy_(torch.from_numpy(p.labels))
    keep = p.labels != ref.IGNORE
    p.forward(handle)
    lse, loss = p.lse.cpu().numpy(), p.loss.cpu().numpy()
    assert np.isfinite(lse[keep]).all() and loss[1] == np.inf
    assert np.isfinite(np.delete(loss, 1)).all()
    p.W[V // 2, 0] = float("inf")
    p.forward(handle)
    lse, loss = p.lse.cpu().numpy(), p.loss.cpu().numpy()
    assert (lse[keep] == np.inf).all() and np.isnan(loss[1]) and loss[3] == 0
    assert (np.delete(loss, [1, 3]) == np.inf).all()
    p.W[V // 2, 0] = float("nan")
    p.forward(handle)
    assert np.isnan(p.lse.cpu().numpy()[keep]).all() and np.isnan(p.loss.cpu().numpy()[keep]).all()


# An infinity where D ends inside a K step of the products.
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [8, 40, 72, 120, 200, 264, 1000])
@pytest.mark.parametrize("T", [20, 300])
def test_masks_in_the_last_columns(handle, T, D, dt):
    for column in (D - 1, D - 8):
        check(masked(T, 1300, D, dt, np.arange(60, 400), "inf", column=column, seed=4), handle)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_masks_in_the_last_columns_big_tiles(handle, dt):
    for D in (40, 328):
        check(masked(300, 20001, D, dt, np.arange(60, 400), "inf", column=D - 1, seed=4), handle)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("D", [5, 33, 50, 72, 130, 1030])
@pytest.mark.parametrize("T", [1, 3, 7, 16, 20, 90, 300])
def test_masks_in_the_last_column_of_any_width(handle, T, D, dt):
    check(masked(T, 1300, D, dt, np.arange(60, 400), "inf", column=D - 1, seed=4, pad=T % 4), handle)


# Infinite operands in three planes.
@pytest.mark.parametrize("words", ["64", "128", "ragged", "but one"])
@pytest.mark.parametrize("column", [0, 263])
def test_infinite_words_in_planes(handle, words, column):
    check(masked(600, 13200, 264, "f32", runs(13200)[words], "inf", column=column), handle)


@pytest.mark.parametrize("T", [90, 600])
def test_infinite_operands_with_all_bits_set(handle, T):
    """X's element that meets the infinity has all 24 bits set, of either sign;
    an infinite element of X meets finite ones and an infinity of W."""
    V, D = 13200, 72
    rng = np.random.default_rng(T)
    b = 1 + (rng.integers(0, 1 << 11, T) * 4096 + 2047) * 2.0 ** -23
    sign = np.where(np.arange(T) % 2 == 0, 1.0, -1.0)
    p = Problem(T, V, D, "f32", seed=5, ignored=0.0, alpha=0.5)
    p.labels[:] = 7
    p.Y.copy_(torch.from_numpy(p.labels))
    p.X[:, 0] = torch.from_numpy(b * sign).float()
    p.W[:, 0] = 0.0
    p.W[100:300, 0] = float("-inf")
    p.forward(handle)
    lse, loss = p.lse.cpu().numpy(), p.loss.cpu().numpy()
    assert np.isfinite(lse[sign > 0]).all() and np.isfinite(loss[sign > 0]).all()
    assert (lse[sign < 0] == np.inf).all() and (loss[sign < 0] == np.inf).all()
    # the same column of X at infinity: z is -inf for words whose element is
    # below 0, and for the label
    p.X[:, 0] = float("inf")
    p.W[:, 0] = torch.from_numpy(-(1 + (rng.integers(0, 1 << 11, V) * 4096 + 2047) * 2.0 ** -23)).float()
    p.forward(handle)
    assert (p.lse == float("-inf")).all() and torch.isnan(p.loss).all()
    p.W[5, 0] = float("inf")
    p.forward(handle)
    assert (p.lse == float("inf")).all() and (p.loss == float("inf")).all()


# Left-out rows beside infinities and NaNs of W.
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("T,V,D,dt", PATHS + PACKED + PLANES + [(2000, 220, 100, "f32")])
def test_left_out_rows_of_dx_are_zero(handle, T, V, D, dt, value):
    p = Problem(T, V, D, dt, seed=6, ignored=0.4)
    p.labels[0], p.labels[1] = ref.IGNORE, 3
    p.Y.copy_(torch.from_numpy(p.labels))
    p.forward(handle)
    p.W[V // 2] = value
    p.backward(handle)
    out = p.Y == ref.IGNORE
    assert (p.dX[out] == 0).all()
    assert not torch.isfinite(p.dX[~out]).any()
