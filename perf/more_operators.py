"""Cases that time the microscaled 8-bit operators.

Blocks of 32 values along a row share one power-of-two scale, the elements are
E4M3.  Four groups of operators make such rows and use them:

* ``checkpoint``: activations kept in 8 bits and read back.
* ``norm``, ``norm_train``: root-mean-square norm of a residual stream with the
  addition of a block's output to it, its result in 8 bits; with the norm's
  gradients.
* ``product``: ``C = alpha * A * W^T`` of 8-bit activations (in hand, or 16-bit
  ones that the call quantises) and a weight in 8 or in 4 bits.
* ``weight_grad``: ``dW = alpha * dY^T * X`` from 16-bit ``dY`` and the
  activations that a forward pass kept in 8 bits.

``own`` False computes the plain forms with elementary torch operations in 32
bits, True calls the library.
"""
from __future__ import annotations

import torch

own = False

BLOCK = 32          # values that share a scale
EPS = 1e-6          # of the norm
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}

_handle = None      # the library handle that a program keeps, and its workspace


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # What a training step of 16384 tokens keeps of a layer's input.
        {"name": "checkpoint_16384x4096_bf16", "op": "checkpoint", "rows": 16384, "k": 4096,
         "dtype": "bf16", "trans": False, "pad": 0},
        # Ragged rows inside a wider buffer: K ends inside a block, the stride
        # is odd.
        {"name": "checkpoint_1000x777_f16", "op": "checkpoint", "rows": 1000, "k": 777,
         "dtype": "f16", "trans": False, "pad": 6},
        # One token of a decode step before a layer: latency.
        {"name": "norm_1x4096_bf16", "op": "norm", "t": 1, "d": 4096, "dtype": "bf16",
         "residual": True},
        # A long prompt's rows before a layer: the stream.
        {"name": "norm_8192x4096_bf16", "op": "norm", "t": 8192, "d": 4096, "dtype": "bf16",
         "residual": True},
        # A stack's first norm, 32-bit states, nothing to add, an odd width.
        {"name": "norm_1000x1501_f32", "op": "norm", "t": 1000, "d": 1501, "dtype": "f32",
         "residual": False},
        # A training batch's norm, forward and backward.
        {"name": "norm_train_8192x4096_bf16", "op": "norm_train", "t": 8192, "d": 4096,
         "dtype": "bf16", "residual": True},
        # A small ragged batch in binary16.
        {"name": "norm_train_777x1000_f16", "op": "norm_train", "t": 777, "d": 1000,
         "dtype": "f16", "residual": True},
        # One token through a square layer: the weight's stream and latency.
        {"name": "product_1x4096x4096_x_bf16_w8", "op": "product", "m": 1, "n": 4096, "k": 4096,
         "a": "bf16", "w": "mx8", "c": "bf16", "alpha": 1.0},
        # A decode batch through the MLP's up-projection, its weight in 4 bits.
        {"name": "product_16x11008x4096_x_bf16_w4", "op": "product", "m": 16, "n": 11008,
         "k": 4096, "a": "bf16", "w": "mx4", "c": "bf16", "alpha": 1.0},
        # A prompt through the MLP's up-projection, its rows from the norm.
        {"name": "product_4096x11008x4096_w8", "op": "product", "m": 4096, "n": 11008,
         "k": 4096, "a": "mx8", "w": "mx8", "c": "bf16", "alpha": 1.0},
        # The gradient of that projection's weight, for 32-bit accumulation.
        {"name": "weight_grad_4096x11008x4096_bf16", "op": "weight_grad", "t": 4096,
         "n": 11008, "d": 4096, "dy": "bf16", "dw": "f32", "alpha": 1.0},
        # A ragged one in binary16, with the loss's scale taken out.
        {"name": "weight_grad_777x1500x1000_f16", "op": "weight_grad", "t": 777, "n": 1500,
         "d": 1000, "dy": "f16", "dw": "f16", "alpha": 0.125},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even in its logarithm."""
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["checkpoint", "norm", "norm_train", "product", "product", "weight_grad"])
    if op == "checkpoint":
        rows, k = _log(rng, 1, 16384), _log(rng, 32, 16384)
        rows = min(rows, max(1, 16384 * 4096 // k))
        dtype = rng.choice(["f32", "bf16", "f16"])
        rows = max(1, rows // 2) if dtype == "f32" else rows
        return {"op": op, "rows": rows, "k": k, "dtype": dtype,
                "trans": rng.random() < 0.3, "pad": rng.choice([0, 0, 1, 6, 64])}
    if op in ("norm", "norm_train"):
        t, d = _log(rng, 1, 16384), _log(rng, 16, 16384)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        t = min(t, max(1, 8192 * 4096 // (d * SIZE[dtype] // 2)))
        return {"op": op, "t": t, "d": d, "dtype": dtype, "residual": rng.random() < 0.7}
    alpha = round(rng.choice([1.0, rng.uniform(0.25, 2.0)]), 3)
    if op == "product":
        m, n, k = _log(rng, 1, 8192), _log(rng, 1, 16384), _log(rng, 32, 16384)
        m = min(m, max(1, 4096 * 11008 * 4096 // (n * k)))
        a = rng.choice(["mx8", "bf16", "f16"])
        k = k if a != "mx8" else BLOCK * -(-k // BLOCK)
        return {"op": op, "m": m, "n": n, "k": k, "a": a, "w": rng.choice(["mx8", "mx4"]),
                "c": rng.choice(["bf16", "f16"]), "alpha": alpha}
    t, n, d = _log(rng, 1, 16384), _log(rng, 1, 16384), _log(rng, 16, 16384)
    t = min(t, max(1, 4096 * 11008 * 4096 // (n * d)))
    return {"op": op, "t": t, "n": n, "d": d, "dy": rng.choice(["bf16", "bf16", "f16"]),
            "dw": rng.choice(["f32", "bf16", "f16"]), "alpha": alpha}


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


def _blocks(x):
    """A float32 matrix as [rows, blocks, 32] (zeros after the last column)
    and the largest magnitude of every block."""
    rows, k = x.shape
    nb = -(-k // BLOCK)
    b = torch.zeros(rows, nb * BLOCK, device=x.device)
    b[:, :k] = x
    b = b.reshape(rows, nb, BLOCK)
    return b, b.abs().amax(-1)


def _times(v, n):
    """v * 2^n, exactly: two powers of two put together from their bits, none
    of which leaves the range of 32 bits."""
    half = n // 2
    return v * ((half + 127) << 23).view(torch.float32) * ((n - half + 127) << 23).view(torch.float32)


def _elements8(x):
    """The quantised blocks of a float32 matrix in E4M3, [rows, blocks, 32],
    and the exponents of their scales: the least one, of at least -127, with
    which the block's largest magnitude is at most 448."""
    b, amax = _blocks(x)
    m, ex = torch.frexp(amax)
    e = torch.where(amax > 0, ex - 9 + (m > 0.875).int(), -127).clamp(min=-127)
    v = _times(b, -e[..., None])
    step = torch.frexp(v)[1].sub(1).clamp(min=-6) - 3
    return _times(torch.round(_times(v, -step)), step), e


def _values8(x):
    """What the 8-bit rows of a float32 matrix stand for, in 32 bits."""
    v, e = _elements8(x)
    return _times(v, e[..., None]).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _pack8(x):
    """(codes, scales) of a float32 matrix: a byte an element and one byte a
    block, the scale's exponent plus 127."""
    v, e = _elements8(x)
    codes = v.reshape(x.shape[0], -1).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8)


def _pack4(x):
    """The same in 4 bits (E2M1, the largest magnitude's binade at 4), two
    codes a byte, the even column in the low half."""
    b, amax = _blocks(x)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(min=-127)
    m = _times(b.abs(), -e[..., None])
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6.0)
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8)
    code = (code + 8 * torch.signbit(b).to(torch.uint8)).reshape(x.shape[0], -1)
    return code[:, 0::2] + 16 * code[:, 1::2], (e + 127).to(torch.uint8)


def _unpack(codes, scales):
    """The values that 8- or 4-bit (codes, scales) stand for, in 32 bits."""
    if codes.shape[1] == BLOCK * scales.shape[1]:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                             device=codes.device)
        v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.reshape(codes.shape[0], -1, BLOCK)
    return _times(v, (scales.int() - 127)[..., None]).reshape(codes.shape[0], -1)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "checkpoint":
        dt = DTYPES[case["dtype"]]
        r, c = (case["k"], case["rows"]) if case["trans"] else (case["rows"], case["k"])
        buf = torch.zeros(r, c + case["pad"], device="cuda", dtype=dt)
        s["x"] = buf[:, :c]
        s["x"].copy_(_activations(g, r, c))
        s["y"] = torch.empty(case["rows"], case["k"], device="cuda", dtype=dt)
        return s
    if op in ("norm", "norm_train"):
        t, d, dt = case["t"], case["d"], DTYPES[case["dtype"]]
        # the stream, and the output of the block before that is added to it
        s["r"] = _activations(g, t, d).to(dt) if case["residual"] else None
        x = torch.randn(t, d, generator=g, device="cuda") * 0.5
        s["x"] = (x if case["residual"] else x + _activations(g, t, d)).to(dt)
        s["g"] = (1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt)
        s["h"] = torch.empty(t, d, device="cuda", dtype=dt) if case["residual"] else None
        # (bfloat16 holds every value of 8-bit rows)
        s["y"] = torch.empty(t, d, device="cuda", dtype=torch.bfloat16)
        s["rstd"] = torch.empty(t, device="cuda")
        if op == "norm_train":
            s["dy"] = (torch.randn(t, d, generator=g, device="cuda") * 0.1).to(dt)
            s["dh"] = (torch.randn(t, d, generator=g, device="cuda") * 0.1).to(dt) \
                if case["residual"] else None
            s["dx"] = torch.empty(t, d, device="cuda", dtype=dt)
            s["dg"] = torch.empty(d, device="cuda", dtype=dt)
        return s
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        w = torch.randn(n, k, generator=g, device="cuda") * (2.0 / k ** 0.5)
        x = _activations(g, m, k)
        s["w"] = _pack8(w) if case["w"] == "mx8" else _pack4(w)
        s["a"] = _pack8(x) if case["a"] == "mx8" else x.to(DTYPES[case["a"]])
        s["c"] = torch.empty(m, n, device="cuda", dtype=DTYPES[case["c"]])
        return s
    t, n, d = case["t"], case["n"], case["d"]
    s["x"] = _pack8(_activations(g, t, d))
    s["dy"] = (torch.randn(t, n, generator=g, device="cuda") * 0.1).to(DTYPES[case["dy"]])
    s["dw"] = torch.empty(n, d, device="cuda", dtype=DTYPES[case["dw"]])
    return s


# ---- one pass -----------------------------------------------------------------------

def run(state):
    case = state["case"]
    return _own(state, case) if own else _plain(state, case)


def _library(state, case):
    """The library and the handle that the program keeps; the handle's
    workspace grows to what a call asks for."""
    global _handle
    import fp32_gemm_major_amd as sg
    if _handle is None:
        _handle = sg.Handle()
    if "ready" not in state:
        need = 0
        if case["op"] == "product" and torch.is_tensor(state["a"]):
            need = sg.Mx8.nbytes(case["m"], case["k"])
        elif case["op"] == "weight_grad":
            need = _handle.mx8_weight_grad_workspace_size(state["dy"], sg.Mx8(*state["x"]))
        if need > 4 * _handle.workspace.numel():
            _handle.set_workspace(need)
        if case["op"] in ("norm", "norm_train"):
            state["q"] = sg.Mx8.empty(case["t"], case["d"])
        state["ready"] = True
    return sg, _handle


def _own(s, case):
    sg, h = _library(s, case)
    if case["op"] == "checkpoint":
        return h.mx8_dequantize(h.mx8_quantize(s["x"], trans=case["trans"]), s["y"])
    if case["op"] == "product":
        a = s["a"] if torch.is_tensor(s["a"]) else sg.Mx8(*s["a"])
        w = (sg.Mx8 if case["w"] == "mx8" else sg.Mx4)(*s["w"])
        h.gemm_mx8(a, w, s["c"], alpha=case["alpha"])
        return s["c"]
    if case["op"] == "weight_grad":
        h.mx8_weight_grad(s["dy"], sg.Mx8(*s["x"]), s["dw"], alpha=case["alpha"])
        return s["dw"]
    q = h.rmsnorm_mx8(s["x"], s["g"], residual=s["r"], H=s["h"], rstd=s["rstd"], eps=EPS,
                      out=s["q"])
    out = {"y": h.mx8_dequantize(q, s["y"]), "rstd": s["rstd"]}
    if case["residual"]:
        out["h"] = s["h"]
    if case["op"] == "norm_train":
        stream = s["h"] if case["residual"] else s["x"]
        h.rmsnorm_backward(s["dy"], stream, s["g"], s["rstd"], s["dx"], dG=s["dg"], dH=s["dh"])
        out["dx"], out["dg"] = s["dx"], s["dg"]
    return out


def _plain(s, case):
    if case["op"] == "checkpoint":
        x = s["x"].float()
        return _values8(x.t() if case["trans"] else x).to(s["x"].dtype)
    if case["op"] == "product":
        a = _values8(s["a"].float()) if torch.is_tensor(s["a"]) else _unpack(*s["a"])
        w = _unpack(*s["w"])[:, :case["k"]]
        return (case["alpha"] * (a @ w.t())).to(s["c"].dtype)
    if case["op"] == "weight_grad":
        x = _unpack(*s["x"])[:, :case["d"]]
        return (case["alpha"] * (s["dy"].float().t() @ x)).to(s["dw"].dtype)
    x, gain = s["x"].float(), s["g"].float()
    out = {}
    if case["residual"]:
        out["h"] = (x + s["r"].float()).to(s["x"].dtype)
        x = out["h"].float()
    rstd = torch.rsqrt((x * x).mean(1) + EPS)
    n = x * rstd[:, None]
    out["y"] = _values8(n * gain).to(torch.bfloat16)
    out["rstd"] = rstd
    if case["op"] == "norm_train":
        dy = s["dy"].float()
        dn = dy * gain
        dx = rstd[:, None] * (dn - n * (dn * n).mean(1, keepdim=True))
        if case["residual"]:
            dx = dx + s["dh"].float()
        out["dx"], out["dg"] = dx.to(s["x"].dtype), (dy * n).sum(0).to(s["g"].dtype)
    return out


# ---- the definition in 64 bits -------------------------------------------------------

def _power(n):
    """2^n in 64 bits (a library's power of two may be off in its last bit,
    which the ties of a rounding show)."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def _rounded(x):
    """Microscaled 8-bit values of a float64 matrix, from the definition: the
    scale is the least power of two, of at least 2^-127, that leaves no
    magnitude over 448; the elements are the nearest numbers of 4 bits (a
    leading one and three more) that are multiples of 2^-9, ties to even."""
    rows, k = x.shape
    out = torch.zeros_like(x)
    for c in range(0, k, BLOCK * 64):
        part = x[:, c:c + BLOCK * 64]
        pad = -part.shape[1] % BLOCK
        b = torch.nn.functional.pad(part, (0, pad)).reshape(rows, -1, BLOCK)
        m, e = torch.frexp(b.abs().amax(-1, keepdim=True) / 448.0)
        s = _power(torch.where(m > 0.5, e, torch.where(m > 0, e - 1, -127)).clamp(min=-127))
        a = b / s
        unit = _power(torch.frexp(a)[1].sub(1).clamp(min=-6) - 3)
        v = (torch.round(a / unit) * unit * s).reshape(rows, -1)
        out[:, c:c + BLOCK * 64] = v[:, :part.shape[1]]
    return out


def _stands_for(codes, scales):
    """The float64 values of codes and scale bytes, read bit by bit."""
    if codes.shape[1] == BLOCK * scales.shape[1]:
        c = codes.int()
        ex, man = (c >> 3) & 15, (c & 7).double()
        mag = torch.where(ex == 0, man / 512, (1 + man / 8) * _power(ex - 7))
        out = torch.where(c >= 128, -mag, mag)
    else:
        out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64,
                          device=codes.device)
        for half in (0, 1):
            c = (codes >> (4 * half)).int() & 15
            ex, man = (c >> 1) & 3, (c & 1).double()
            mag = torch.where(ex == 0, man / 2, (1 + man / 2) * _power(ex - 1))
            out[:, half::2] = torch.where(c >= 8, -mag, mag)
    return out * _power(scales.int() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        x = s["x"].double()
        return _rounded(x.t().contiguous() if case["trans"] else x)
    if case["op"] == "product":
        a = _rounded(s["a"].double()) if torch.is_tensor(s["a"]) else _stands_for(*s["a"])
        w = _stands_for(*s["w"])[:, :case["k"]].contiguous()
        return case["alpha"] * torch.mm(a, w.t())
    if case["op"] == "weight_grad":
        x = _stands_for(*s["x"])[:, :case["d"]].contiguous()
        return case["alpha"] * torch.mm(s["dy"].double().t(), x)
    h, gain, out = s["x"].double(), s["g"].double(), {}
    if case["residual"]:
        # (what is kept is the sum rounded to the stream's type)
        out["h"] = (h + s["r"].double()).to(s["x"].dtype).double()
        h = out["h"]
    d = case["d"]
    root = torch.sqrt((h * h).sum(1, keepdim=True) / d + EPS)
    out["y"], out["rstd"] = _rounded(gain * h / root), 1.0 / root[:, 0]
    if case["op"] == "norm_train":
        dy = s["dy"].double()
        # d/dh of gain * h / root, row by row
        along = (dy * gain * h).sum(1, keepdim=True) / (d * root ** 3)
        out["dx"] = dy * gain / root - h * along
        if case["residual"]:
            out["dx"] += s["dh"].double()
        out["dg"] = (dy * h / root).sum(0)
    return out


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    if case["op"] == "checkpoint":
        n, nb = case["rows"] * case["k"], case["rows"] * -(-case["k"] // BLOCK)
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 2 * 33 * nb, "flops": 4 * n}
    if case["op"] in ("norm", "norm_train"):
        t, d, size = case["t"], case["d"], SIZE[case["dtype"]]
        n, q = t * d, 33 * t * -(-d // BLOCK)
        # the states (and what is added to them, and their sum), the gain, the
        # 8-bit rows written and read back as 16-bit values
        byte = (3 if case["residual"] else 1) * n * size + d * size + 4 * t + 2 * q + 2 * n
        flops = 8 * n
        if case["op"] == "norm_train":
            # dy and the stream (and its gradient) to dx
            byte += (4 if case["residual"] else 3) * n * size + 2 * d * size + 4 * t
            flops += 10 * n
        return {"bytes": byte, "flops": flops}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        nb = -(-k // BLOCK)
        a = 33 * m * nb if case["a"] == "mx8" else m * k * SIZE[case["a"]]
        w = (33 if case["w"] == "mx8" else 17) * n * nb
        return {"bytes": a + w + m * n * SIZE[case["c"]], "flops": 2 * m * n * k}
    t, n, d = case["t"], case["n"], case["d"]
    return {"bytes": t * n * SIZE[case["dy"]] + 33 * t * -(-d // BLOCK)
            + n * d * SIZE[case["dw"]], "flops": 2 * t * n * d}
