"""Cases that time the microscaled 4-bit operators and the output layer's loss.

Two groups of operators around the library's products:

* ``quantise``, ``product``: microscaled 4-bit values (blocks of 32 along K
  share one power-of-two scale, elements are E2M1) made from 16/32-bit
  tensors, and ``C = alpha * A * B^T`` of two such operands.  A product's A is
  either in hand in 4 bits or 16-bit activations that the call quantises.
* ``loss``, ``train``: softmax cross entropy of ``alpha * X * W^T`` against one
  label a row, in pieces of the vocabulary and without keeping the logits; its
  value, and its value with both gradients.

``own`` False computes the plain forms with elementary torch operations in 32
bits, True calls the library.
"""
from __future__ import annotations

import torch

own = False

BLOCK = 32          # values that share a scale
IGNORE = -100       # the label of a row that is left out
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}

_handle = None      # the library handle that a program keeps, and its workspace


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # Activations of a small decode batch, quantised and read back: two
        # small launches, latency.
        {"name": "quantise_16x4096_bf16", "op": "quantise", "rows": 16, "k": 4096,
         "dtype": "bf16", "trans": False, "pad": 0},
        # A weight of the MLP shape stored K x N in 32 bits, quantised along K
        # once when a model is loaded: the stream of a strided source.
        {"name": "quantise_11008x4096_f32_kn", "op": "quantise", "rows": 11008, "k": 4096,
         "dtype": "f32", "trans": True, "pad": 0},
        # Ragged rows inside a wider buffer: K ends inside a block, the stride
        # is odd.
        {"name": "quantise_1000x777_f16", "op": "quantise", "rows": 1000, "k": 777,
         "dtype": "f16", "trans": False, "pad": 6},
        # One token through a square layer: the weight's stream and latency.
        {"name": "product_1x4096x4096_x_bf16", "op": "product", "m": 1, "n": 4096, "k": 4096,
         "a": "bf16", "c": "bf16", "alpha": 1.0},
        # A decode batch through the MLP's up-projection.
        {"name": "product_16x11008x4096_x_bf16", "op": "product", "m": 16, "n": 11008,
         "k": 4096, "a": "bf16", "c": "bf16", "alpha": 1.0},
        # A prompt through the MLP's up-projection, A quantised before.
        {"name": "product_4096x11008x4096", "op": "product", "m": 4096, "n": 11008,
         "k": 4096, "a": "mx4", "c": "bf16", "alpha": 1.0},
        # Ragged sizes, a K that ends inside a K step, 32-bit results.
        {"name": "product_1000x1500x800_f32", "op": "product", "m": 1000, "n": 1500,
         "k": 800, "a": "mx4", "c": "f32", "alpha": 1.5},
        # Scoring one token: the output layer's weight is read once.
        {"name": "loss_1x32000x4096_bf16", "op": "loss", "t": 1, "v": 32000, "d": 4096,
         "dtype": "bf16", "ignored": 0.0},
        # Perplexity of a long prompt over a large vocabulary.
        {"name": "loss_4096x131072x4096_bf16", "op": "loss", "t": 4096, "v": 131072,
         "d": 4096, "dtype": "bf16", "ignored": 0.0},
        # A ragged training batch in binary16 with loss scaling; half its rows
        # are prompt or padding and left out.
        {"name": "train_777x50001x1000_f16", "op": "train", "t": 777, "v": 50001, "d": 1000,
         "dtype": "f16", "ignored": 0.5},
        # A small model trained in 32 bits.
        {"name": "train_1024x32000x1024_f32", "op": "train", "t": 1024, "v": 32000,
         "d": 1024, "dtype": "f32", "ignored": 0.1},
        # A training step's output layer at full size.
        {"name": "train_4096x131072x4096_bf16", "op": "train", "t": 4096, "v": 131072,
         "d": 4096, "dtype": "bf16", "ignored": 0.1},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "loss", "train"])
    if op == "quantise":
        rows, k = _log(rng, 1, 16384), _log(rng, 32, 16384)
        rows = min(rows, max(1, 11008 * 4096 // k))
        return {"op": op, "rows": rows, "k": k, "dtype": rng.choice(["f32", "bf16", "f16"]),
                "trans": rng.random() < 0.4, "pad": rng.choice([0, 0, 1, 6, 64])}
    if op == "product":
        m, n, k = _log(rng, 1, 8192), _log(rng, 1, 16384), 32 * _log(rng, 1, 512)
        m = min(m, max(1, 4096 * 11008 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "a": rng.choice(["mx4", "bf16", "f16"]),
                "c": rng.choice(["bf16", "f16", "f32"]),
                "alpha": round(rng.choice([1.0, rng.uniform(0.25, 2.0)]), 3)}
    t, v, d = _log(rng, 1, 4096), _log(rng, 100, 131072), _log(rng, 16, 4096)
    if op == "loss":
        t = max(t, 4)
    return {"op": op, "t": t, "v": v, "d": d, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]),
            "ignored": rng.choice([0.0, 0.1, 0.5])}


# ---- inputs ---------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, k):
    """Values of a hidden state: unit normal, one channel in sixty-four ten
    times as large, as trained models have them."""
    x = torch.randn(rows, k, generator=g, device="cuda")
    return torch.where(torch.rand(k, generator=g, device="cuda") < 1 / 64, 10.0 * x, x)


def _pack(x):
    """(codes, scales) of a float32 matrix: 4-bit codes two to a byte, the
    even column in the low half, blocks of 32 columns (zeros after the last)
    and one byte a block, the scale's exponent plus 127."""
    mag, sign, e = _elements(x)
    code = (torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4))
            ).to(torch.uint8) + 8 * sign.to(torch.uint8)
    code = code.reshape(x.shape[0], -1)
    return code[:, 0::2] + 16 * code[:, 1::2], (e + 127).to(torch.uint8)


def _elements(x):
    """The quantised blocks of a float32 matrix: magnitudes of E2M1 and signs
    [rows, blocks, 32], and the scales' exponents [rows, blocks]."""
    rows, k = x.shape
    nb = -(-k // BLOCK)
    b = torch.zeros(rows, nb * BLOCK, device=x.device)
    b[:, :k] = x
    b = b.reshape(rows, nb, BLOCK)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - 2, -127).clamp(min=-127)
    # (x / 2 scaled by 2^(1-e): no factor leaves the range of 32 bits)
    m = torch.ldexp(torch.ldexp(b.abs(), -(e // 2)[..., None]), -(e - e // 2)[..., None])
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return (torch.round(m / step) * step).clamp(max=6.0), torch.signbit(b), e


def _unpack(codes, scales):
    """The values that (codes, scales) stand for, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.reshape(codes.shape[0], -1, BLOCK)
    return torch.ldexp(v, (scales.int() - 127)[..., None]).reshape(codes.shape[0], -1)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    if op == "quantise":
        dt = DTYPES[case["dtype"]]
        r, c = (case["k"], case["rows"]) if case["trans"] else (case["rows"], case["k"])
        buf = torch.zeros(r, c + case["pad"], device="cuda", dtype=dt)
        x = buf[:, :c]
        x.copy_(_activations(g, r, c))
        return {"case": case, "x": x,
                "y": torch.empty(case["rows"], case["k"], device="cuda", dtype=dt)}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        w = torch.randn(n, k, generator=g, device="cuda") * (2.0 / k ** 0.5)
        x = _activations(g, m, k)
        s = {"case": case, "b": _pack(w),
             "c": torch.empty(m, n, device="cuda", dtype=DTYPES[case["c"]])}
        s["a"] = _pack(x) if case["a"] == "mx4" else x.to(DTYPES[case["a"]])
        return s
    t, v, d, dt = case["t"], case["v"], case["d"], DTYPES[case["dtype"]]
    w = torch.randn(v, d, generator=g, device="cuda") * (2.0 / d ** 0.5)
    labels = torch.randint(0, v, (t,), generator=g, device="cuda")
    # a trained model: the label's logit is raised, from not at all to plainly
    # the largest
    x = torch.randn(t, d, generator=g, device="cuda")
    x += torch.rand(t, 1, generator=g, device="cuda") * 3.0 * w[labels]
    drop = torch.rand(t, generator=g, device="cuda") < case["ignored"]
    drop[0] = False
    labels = torch.where(drop, IGNORE, labels)
    s = {"case": case, "x": x.to(dt), "w": w.to(dt), "labels": labels}
    s["loss"] = torch.empty(t, device="cuda")
    s["lse"] = torch.empty(t, device="cuda")
    if op == "train":
        # the mean over the rows that count, times the loss scale of binary16
        scale = 1024.0 if case["dtype"] == "f16" else 1.0
        s["dloss"] = torch.where(drop, 0.0, scale / (t - int(drop.sum())))
        s["dx"] = torch.empty_like(s["x"])
        s["dw"] = torch.empty_like(s["w"])
    return s


# ---- one pass -----------------------------------------------------------------------

def run(state):
    case = state["case"]
    return _own(state, case) if own else _plain(state, case)


def _library(state, case):
    """The library and the handle that the program keeps; the handle's
    workspace grows to what the loss asks for."""
    global _handle
    import fp32_gemm_major_amd as sg
    if _handle is None:
        _handle = sg.Handle()
    if case["op"] in ("loss", "train") and "ready" not in state:
        need = _handle.ce_workspace_size(state["x"], state["w"], backward=case["op"] == "train")
        if need > 4 * _handle.workspace.numel():
            _handle.set_workspace(need)
        state["ready"] = True
    return sg, _handle


def _own(state, case):
    sg, h = _library(state, case)
    if case["op"] == "quantise":
        h.mx4_dequantize(h.mx4_quantize(state["x"], trans=case["trans"]), state["y"])
        return state["y"]
    if case["op"] == "product":
        a = state["a"] if torch.is_tensor(state["a"]) else sg.Mx4(*state["a"])
        h.gemm_mx4(a, sg.Mx4(*state["b"]), state["c"], alpha=case["alpha"])
        return state["c"]
    h.ce_forward(state["x"], state["w"], state["labels"], state["loss"], state["lse"],
                 ignore_index=IGNORE)
    if case["op"] == "loss":
        return {"loss": state["loss"], "lse": state["lse"]}
    h.ce_backward(state["x"], state["w"], state["labels"], state["lse"], state["dloss"],
                  state["dx"], state["dw"], ignore_index=IGNORE)
    return {"loss": state["loss"], "lse": state["lse"], "dx": state["dx"], "dw": state["dw"]}


def _plain(state, case):
    if case["op"] == "quantise":
        x = state["x"].float()
        x = x.t() if case["trans"] else x
        mag, sign, e = _elements(x)
        v = torch.ldexp(torch.where(sign, -mag, mag), e[..., None]).reshape(x.shape[0], -1)
        return v[:, :case["k"]].to(state["x"].dtype)
    if case["op"] == "product":
        a = _unpack(*(_pack(state["a"].float()) if torch.is_tensor(state["a"]) else state["a"]))
        return (case["alpha"] * (a @ _unpack(*state["b"]).t())).to(state["c"].dtype)
    x, w, labels = state["x"].float(), state["w"].float(), state["labels"]
    z = x @ w.t()
    keep = labels != IGNORE
    at = torch.where(keep, labels, 0)[:, None]
    top = z.amax(1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
    loss = torch.where(keep, lse - z.gather(1, at)[:, 0], 0.0)
    out = {"loss": loss, "lse": torch.where(keep, lse, 0.0)}
    if case["op"] == "loss":
        return out
    g = torch.where(keep, state["dloss"], 0.0)[:, None]
    p = torch.exp(z.sub_(lse[:, None])).mul_(g)
    p.scatter_add_(1, at, -g)
    out["dx"] = (p @ w).to(state["x"].dtype)
    out["dw"] = (p.t() @ x).to(state["w"].dtype)
    return out


# ---- the definition in 64 bits -------------------------------------------------------

def _rounded(x):
    """Microscaled 4-bit values of a float64 matrix, from the definition: the
    scale is 2^(floor(log2 of the block's largest magnitude) - 2), the
    elements the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (a tie goes to the one
    with the even code, what is larger to 6)."""
    rows, k = x.shape
    out = torch.zeros_like(x)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=x.device, dtype=torch.float64)
    for c in range(0, k, BLOCK * 64):
        part = x[:, c:c + BLOCK * 64]
        pad = -part.shape[1] % BLOCK
        b = torch.nn.functional.pad(part, (0, pad)).reshape(rows, -1, BLOCK)
        amax = b.abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, 2.0 ** -125))) - 2
        s = torch.pow(2.0, e.clamp(min=-127))
        a = b.abs() / s
        code = ((a > .25).int() + (a >= .75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
                + (a >= 3.5) + (a > 5))
        v = (grid[code] * torch.sign(b) * s).reshape(rows, -1)
        out[:, c:c + BLOCK * 64] = v[:, :part.shape[1]]
    return out


def _stands_for(codes, scales):
    """The float64 values of packed codes and scale bytes."""
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64,
                      device=codes.device)
    for half in (0, 1):
        c = (codes >> (4 * half)).int() & 15
        ex, man = (c >> 1) & 3, (c & 1).double()
        mag = torch.where(ex == 0, man / 2, (1 + man / 2) * torch.pow(2.0, ex.double() - 1))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    return out * torch.pow(2.0, scales.double() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        x = s["x"].double()
        return _rounded(x.t().contiguous() if case["trans"] else x)
    if case["op"] == "product":
        a = _rounded(s["a"].double()) if torch.is_tensor(s["a"]) else _stands_for(*s["a"])
        return case["alpha"] * torch.mm(a, _stands_for(*s["b"]).t())
    x, w, keep = s["x"].double(), s["w"].double(), s["labels"] != IGNORE
    t = case["t"]
    rows = torch.arange(t, device="cuda")
    hit = s["labels"].clamp(min=0)
    z = torch.mm(x, w.t())
    lse = torch.logsumexp(z, 1)
    zero = torch.zeros_like(lse)
    out = {"loss": torch.where(keep, lse - z[rows, hit], zero),
           "lse": torch.where(keep, lse, zero)}
    if case["op"] == "train":
        z -= lse[:, None]
        z.exp_()
        z[rows, hit] -= 1.0
        z *= torch.where(keep, s["dloss"].double(), zero)[:, None]
        out["dx"] = torch.mm(z, w)
        out["dw"] = torch.mm(z.t(), x)
    return out


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    if case["op"] == "quantise":
        n, nb = case["rows"] * case["k"], case["rows"] * -(-case["k"] // BLOCK)
        q = 17 * nb  # sixteen bytes of codes and one of scale a block
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 2 * q, "flops": 4 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = m * k * 17 / 32 if case["a"] == "mx4" else m * k * SIZE[case["a"]]
        return {"bytes": a + n * k * 17 / 32 + m * n * SIZE[case["c"]], "flops": 2 * m * n * k}
    t, v, d, size = case["t"], case["v"], case["d"], SIZE[case["dtype"]]
    if case["op"] == "loss":
        return {"bytes": (t + v) * d * size + 16 * t, "flops": 2 * t * v * d}
    # the logits once, and a product for each gradient
    return {"bytes": 2 * (t + v) * d * size + 20 * t, "flops": 6 * t * v * d}
