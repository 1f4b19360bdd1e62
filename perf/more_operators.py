"""Cases of the operators around RMS norm and 4-bit linear layers.

    norm      RMS norm of the rows of a residual stream: s = x + residual, y = s rstd w with rstd =
              (mean s^2 + eps)^-1/2.  To a layer with 8-bit weights it hands y as E4M3 codes with one
              E8M0 scale per 128 values of a row, to one with 4-bit weights y itself and its largest
              magnitude.  Backward: the gradient of s, to which the gradient that comes along the
              residual stream is added, and the gradient of w
    quantise  an activation as NVFP4 codes: its largest magnitude, then E2M1 codes with one E4M3 scale
              per 16 values, along its rows and along its columns (that copy lies transposed), and
              the values of both copies
    product   D = A B^T (+ C) of two NVFP4 operands: a linear layer's output, its input's gradient
              and its weight's gradient
    linear    a 4-bit linear layer's training step: both activations quantised, three products

Conventions.  E4M3 with E8M0: e = floor(log2(amax)) - 8 clamped at -127, byte e + 127 (0xFF for a block
with a NaN or an infinity), code = E4M3(y * 2^-e), nearest-even, saturating at 448.  NVFP4: S = 2688 / G
with G the tensor's largest magnitude (1 for G = 0, at most the largest float), block scale s =
E4M3((A / 6) S) with A the block's, code = E2M1(x (S / s)) (0 where s is 0), nearest-even, saturating at 6,
every step rounded to 32 bits; a code stands for code * s * (1 / S).  Codes lie two to a byte, the
even column in the low half; an operand's rows have a pitch of whole 16-byte units.  Scales lie in 128x4
tiles of 512 bytes: entry (r, c) of a tile at byte (r % 32) * 16 + (r / 32) * 4 + c.
"""
import math

import torch

own = False

EPS = 1e-5
LARGEST = 3.4028234663852886e38  # the largest float


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # serving: one new token in front of a layer with 8-bit weights
        {"name": "norm one token", "op": "norm", "dir": "forward", "rows": 1, "cols": 4096, "dtype": "bf16",
         "to": "codes"},
        # a prompt, or one long training micro-batch, in front of a layer with 8-bit weights
        {"name": "norm forward", "op": "norm", "dir": "forward", "rows": 16384, "cols": 6144, "dtype": "bf16",
         "to": "codes"},
        # odd sizes in 32 bits, in front of a layer with 4-bit weights
        {"name": "norm forward odd", "op": "norm", "dir": "forward", "rows": 4001, "cols": 1023, "dtype": "f32",
         "to": "values"},
        # the backward pass of the long micro-batch, inside a residual stream
        {"name": "norm backward", "op": "norm", "dir": "backward", "rows": 16384, "cols": 6144, "dtype": "bf16"},
        # the smallest weight-sized matrix of the package's workloads: latency-bound calls
        {"name": "quantise small", "op": "quantise", "rows": 160, "cols": 96, "dtype": "f32"},
        # the activations of one long training micro-batch
        {"name": "quantise large", "op": "quantise", "rows": 16384, "cols": 6144, "dtype": "bf16"},
        # serving: one new token through a square layer
        {"name": "product one token", "op": "product", "kind": "output", "tokens": 1, "outs": 4096, "ins": 4096,
         "dtype": "bf16"},
        # serving: a batch of decoding sequences through a wide layer
        {"name": "product 64 tokens", "op": "product", "kind": "output", "tokens": 64, "outs": 8192, "ins": 8192,
         "dtype": "bf16"},
        # nothing divides anything: ragged tiles, a contraction that ends inside a byte
        {"name": "product ragged", "op": "product", "kind": "input_grad", "tokens": 1000, "outs": 999, "ins": 1111,
         "dtype": "f32"},
        # a prompt, or one training micro-batch, through a square layer
        {"name": "product 4096", "op": "product", "kind": "output", "tokens": 4096, "outs": 4096, "ins": 4096,
         "dtype": "bf16"},
        # a weight's gradient added to the gradient of the micro-batches before
        {"name": "product weight gradient", "op": "product", "kind": "weight_grad", "tokens": 8192, "outs": 2048,
         "ins": 8192, "dtype": "f32"},
        # one training step of a large linear layer
        {"name": "linear step", "op": "linear", "tokens": 8192, "outs": 8192, "ins": 8192, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer width: as often a multiple of 32 as not."""
    w = _log_int(rng, lo, hi)
    return max(lo, w // 32 * 32) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["norm", "norm", "norm", "quantise", "quantise", "product", "product", "product", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        case = {"op": op, "dir": rng.choice(["forward", "forward", "backward"]), "rows": _log_int(rng, 1, 16384),
                "cols": _width(rng, 64, 6144), "dtype": dtype}
        if case["dir"] == "forward":
            case["to"] = rng.choice(["codes", "values"])
        return case
    if op == "quantise":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _width(rng, 16, 6144), "dtype": dtype}
    if op == "product":
        kind = rng.choice(["output", "output", "input_grad", "weight_grad"])
        return {"op": op, "kind": kind, "tokens": _log_int(rng, 1, 8192), "outs": _width(rng, 64, 8192),
                "ins": _width(rng, 64, 8192), "dtype": "f32" if kind == "weight_grad" else dtype}
    return {"op": op, "tokens": _log_int(rng, 16, 8192), "outs": _width(rng, 64, 8192),
            "ins": _width(rng, 64, 8192), "dtype": dtype}


# ------------------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pitch(n):
    """Row stride of a buffer of bytes: whole 16-byte units."""
    return (n + 15) // 16 * 16


def _scale_bytes(rows, cols):
    return (rows + 127) // 128 * 128 * ((cols + 3) // 4 * 4)


def _rows(n, cols, g, dtype, std, outliers=False):
    """Activations: normal values, a few channels 20 times the others."""
    x = torch.randn(n, cols, generator=g, device="cuda") * std
    if outliers:
        x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(dtype)


def _power(e):
    """2^e as a float, from its bits, for whole e in [-127, 127]; NaN past that."""
    bits = torch.where(e > -127, (e + 127) << 23, 1 << 22)
    return torch.where(e > 127, 0x7FC00000, bits).to(torch.int32).view(torch.float32)


def _blocks(x, block):
    """The columns of x in blocks, the last one filled up with zeros."""
    r, c = x.shape
    nb = (c + block - 1) // block
    return torch.nn.functional.pad(x, (0, nb * block - c)).view(r, nb, block)


def _kept8(y):
    """What E4M3 codes with a scale per 128 values of a row keep of y."""
    b = _blocks(y, 128)
    top = b.abs().amax(2).view(torch.int32) >> 23
    byte = torch.where(top == 255, 255, (top - 8).clamp(min=0))
    mul = torch.where(byte == 255, math.nan, _power(127 - byte))
    q = (b * mul[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return (q * _power(byte.int() - 127)[:, :, None]).flatten(1)[:, :y.shape[1]]


def _tensor_scale(top):
    """S of the tensor whose largest magnitude is `top`."""
    # quotients in 64 bits, rounded: with a number on one side torch multiplies by a rounded reciprocal
    return torch.where(top == 0, 1.0, (2688.0 / top.double()).clamp(max=LARGEST).float())


def _encode4(x, top):
    """(E2M1 values of x's codes, E4M3 scales), in blocks of 16 along the rows."""
    b = _blocks(x.float(), 16)
    S = _tensor_scale(top)
    s = ((b.abs().amax(2).double() / 6.0).float() * S).clamp(max=448.0).to(torch.float8_e4m3fn)
    f = s.float()
    v = b * torch.where(f == 0, 0.0, S / f)[:, :, None]
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = ((v / step).round() * step).clamp(-6.0, 6.0)
    return q.flatten(1)[:, :x.shape[1]], s


def _values4(q, s, top):
    """The values that codes of E2M1 values q and scales s stand for."""
    f = s.float().repeat_interleave(16, 1)[:, :q.shape[1]]
    return q * f * (1.0 / _tensor_scale(top))


def _kept4(x, top):
    return _values4(*_encode4(x, top), top)


def _packed(q):
    """Codes of E2M1 values in a buffer, two to a byte."""
    r, c = q.shape
    a = (q.abs() * 2).to(torch.uint8)  # 0 1 2 3 4 6 8 12
    code = a - (a > 4).to(torch.uint8) - (a > 6).to(torch.uint8) - 3 * (a > 8).to(torch.uint8)
    code |= torch.signbit(q).to(torch.uint8) << 3
    two = torch.nn.functional.pad(code, (0, c % 2)).view(r, -1, 2)
    buf = torch.zeros(r, _pitch((c + 1) // 2), dtype=torch.uint8, device="cuda")
    buf[:, :two.shape[1]] = two[:, :, 0] | (two[:, :, 1] << 4)
    return buf


def _tiled(grid):
    """A scale grid [rows][blocks] in 128x4 tiles, padded with zero bytes."""
    r, c = grid.shape
    R, C = (r + 127) // 128, (c + 3) // 4
    g = torch.nn.functional.pad(grid.view(torch.uint8), (0, 4 * C - c, 0, 128 * R - r))
    return g.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _grid(tiled, r, c):
    """The scale grid that lies in 128x4 tiles."""
    R, C = (r + 127) // 128, (c + 3) // 4
    return tiled.view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * R, 4 * C)[:r, :c]


def _u8(*shape):
    return torch.empty(*shape, dtype=torch.uint8, device="cuda")


def _operand(x):
    """An operand in hand: codes, scales, largest magnitude."""
    top = x.float().abs().amax().view(1)
    q, s = _encode4(x, top)
    return {"codes": _packed(q), "scale": _tiled(s), "top": top}


def _empty_operand(rows, cols):
    return {"codes": _u8(rows, _pitch((cols + 1) // 2)), "scale": _u8(_scale_bytes(rows, (cols + 15) // 16))}


def _sizes(case):
    """(m, n, k) of a product."""
    t, o, i = case["tokens"], case["outs"], case["ins"]
    return {"output": (t, o, i), "input_grad": (t, i, o), "weight_grad": (o, i, t)}[case["kind"]]


def _activations(case, seed):
    """The values that a case starts from."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    if case["op"] == "quantise":
        return {"x": _rows(case["rows"], case["cols"], g, dt, 1.0, True)}
    if case["op"] in ("product", "linear"):
        t, o, i = case["tokens"], case["outs"], case["ins"]
        got = {"x": _rows(t, i, g, dt, 1.0, True), "dy": _rows(t, o, g, dt, 1e-3),
               "w": _rows(o, i, g, torch.bfloat16, 0.02)}
        if case.get("kind") == "weight_grad" or case["op"] == "linear":
            got["c"] = _rows(o, i, g, torch.float32, 0.05)
        return got
    r, c = case["rows"], case["cols"]
    got = {"weight": 1 + 0.1 * torch.randn(c, generator=g, device="cuda"), "x": _rows(r, c, g, dt, 1.0, True)}
    if case["dir"] == "forward":
        got["residual"] = _rows(r, c, g, dt, 2.0)
    else:
        got |= {"dy": _rows(r, c, g, dt, 1e-2), "dsum": _rows(r, c, g, dt, 1e-2)}
    return got


def prepare(case, seed):
    s = {"case": case, **_activations(case, seed)}
    dt = _TYPES[case["dtype"]]
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        if case["dir"] == "forward":
            s |= {"sum": torch.empty(r, c, dtype=dt, device="cuda"), "rstd": torch.empty(r, device="cuda")}
            if case["to"] == "codes":
                s |= {"codes": _u8(r, _pitch(c)), "scale": _u8(_scale_bytes(r, (c + 127) // 128)),
                      "y": torch.empty(r, c, dtype=torch.bfloat16, device="cuda")}
            else:
                s |= {"y": torch.empty(r, c, dtype=dt, device="cuda"), "top": torch.empty(1, device="cuda")}
        else:
            s["rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt()
            s |= {"dx": torch.empty(r, c, dtype=dt, device="cuda"), "dweight": torch.empty(c, device="cuda")}
    elif case["op"] == "quantise":
        r, c = case["rows"], case["cols"]
        s |= {"r": _empty_operand(r, c), "c": _empty_operand(c, r), "top": torch.empty(1, device="cuda"),
              "y_r": torch.empty(r, c, dtype=dt, device="cuda"), "y_c": torch.empty(c, r, dtype=dt, device="cuda")}
    elif case["op"] == "product":
        kind = case["kind"]
        s["a"] = _operand({"output": s["x"], "input_grad": s["dy"], "weight_grad": s["dy"].t()}[kind])
        # a weight's columnwise codes are laid out as rows of the contraction once
        s["b"] = _operand({"output": s["w"], "input_grad": s["w"].t(), "weight_grad": s["x"].t()}[kind])
        m, n, _ = _sizes(case)
        s["out"] = torch.empty(m, n, dtype=dt, device="cuda")
        for name in ("x", "dy", "w"):
            del s[name]
    else:
        t, o, i = case["tokens"], case["outs"], case["ins"]
        s["w_r"], s["w_c"] = _operand(s["w"]), _operand(s["w"].t())
        del s["w"]
        for name, width in (("x", i), ("dy", o)):
            s[name + "_r"], s[name + "_c"] = _empty_operand(t, width), _empty_operand(width, t)
            s[name + "_top"] = torch.empty(1, device="cuda")
        s |= {"y": torch.empty(t, o, dtype=dt, device="cuda"), "dx": torch.empty(t, i, dtype=dt, device="cuda"),
              "dw": torch.empty(o, i, device="cuda")}
    if own:
        s["calls"] = _calls(case, s)
    return s


def _calls(case, s):
    """The framework's calls of one pass, their arguments marshalled once."""
    from mxfp8_master_weight_gb300 import api

    def quantise(x, top, rowwise, colwise, r, c):
        return [api.prepare_nvfp4_tensor_amax(x, top, r, c),
                api.prepare_nvfp4_quantize(x, top, rowwise["codes"], rowwise["scale"], colwise["codes"],
                                           colwise["scale"], r, c)]

    def product(a, a_top, b, b_top, addend, out, m, n, k):
        return api.prepare_nvfp4_gemm(a["codes"], a["scale"], a_top, b["codes"], b["scale"], b_top, addend, out, m, n, k)

    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        if case["dir"] == "backward":
            s["workspace"] = _u8(max(1, api.mxfp8_rms_norm_workspace_size(r, c)))
            return [api.prepare_rms_norm_backward(s["dy"], s["dsum"], s["x"], s["weight"], s["rstd"], s["dx"],
                                                  s["dweight"], s["workspace"], r, c)]
        if case["to"] == "values":
            return [api.prepare_rms_norm_forward(s["x"], s["residual"], s["weight"], s["sum"], s["y"], None, None,
                                                 s["top"], s["rstd"], r, c, EPS)]
        return [api.prepare_rms_norm_forward(s["x"], s["residual"], s["weight"], s["sum"], None, s["codes"], s["scale"],
                                             None, s["rstd"], r, c, EPS),
                api.prepare_checkpoint_restore(s["codes"], s["scale"], s["y"], r, c)]
    if case["op"] == "quantise":
        r, c = case["rows"], case["cols"]
        return quantise(s["x"], s["top"], s["r"], s["c"], r, c) + [
            api.prepare_nvfp4_restore(s["r"]["codes"], s["r"]["scale"], s["top"], s["y_r"], r, c),
            api.prepare_nvfp4_restore(s["c"]["codes"], s["c"]["scale"], s["top"], s["y_c"], c, r)]
    if case["op"] == "product":
        m, n, k = _sizes(case)
        return [product(s["a"], s["a"]["top"], s["b"], s["b"]["top"], s.get("c"), s["out"], m, n, k)]
    t, o, i = case["tokens"], case["outs"], case["ins"]
    return (quantise(s["x"], s["x_top"], s["x_r"], s["x_c"], t, i)
            + [product(s["x_r"], s["x_top"], s["w_r"], s["w_r"]["top"], None, s["y"], t, o, i)]
            + quantise(s["dy"], s["dy_top"], s["dy_r"], s["dy_c"], t, o)
            + [product(s["dy_r"], s["dy_top"], s["w_c"], s["w_c"]["top"], None, s["dx"], t, i, o),
               product(s["dy_c"], s["dy_top"], s["x_c"], s["x_top"], s["c"], s["dw"], o, i, t)])


# ------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        if case["op"] == "norm" and case.get("to") == "values":
            s["top"].zero_()  # the largest magnitude is accumulated over calls
        [c.call() for c in s["calls"]]
        if case["op"] == "norm":
            if case["dir"] == "backward":
                return {"dx": s["dx"], "dweight": s["dweight"]}
            return {k: s[k] for k in ("sum", "rstd", "y") + (("top",) if case["to"] == "values" else ())}
        if case["op"] == "quantise":
            return {"top": s["top"], "r": s["y_r"], "c": s["y_c"]}
        if case["op"] == "product":
            return s["out"]
        return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    dt = _TYPES[case["dtype"]]
    if case["op"] == "norm":
        w, x = s["weight"], s["x"].float()
        if case["dir"] == "backward":
            rstd, dy = s["rstd"][:, None], s["dy"].float()
            xh = x * rstd
            g = dy * w
            dx = rstd * (g - xh * (g * xh).mean(1, keepdim=True)) + s["dsum"].float()
            return {"dx": dx.to(dt), "dweight": (dy * xh).sum(0)}
        x = x + s["residual"].float()
        rstd = (x.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = x * rstd * w
        got = {"sum": x.to(dt), "rstd": rstd[:, 0]}
        if case["to"] == "codes":  # exact in BF16: four bits and a power of two
            return got | {"y": _kept8(y).to(torch.bfloat16)}
        y = y.to(dt)
        return got | {"y": y, "top": y.float().abs().amax().view(1)}
    if case["op"] == "quantise":
        top = s["x"].float().abs().amax().view(1)
        return {"top": top, "r": _kept4(s["x"], top).to(dt), "c": _kept4(s["x"].t(), top).to(dt)}
    if case["op"] == "product":
        m, n, k = _sizes(case)
        d = _decoded(s["a"], m, k) @ _decoded(s["b"], n, k).t()
        return (d + s["c"] if "c" in s else d).to(dt)
    t, o, i = case["tokens"], case["outs"], case["ins"]
    x_top, dy_top = s["x"].float().abs().amax().view(1), s["dy"].float().abs().amax().view(1)
    return {"y": (_kept4(s["x"], x_top) @ _decoded(s["w_r"], o, i).t()).to(dt),
            "dx": (_kept4(s["dy"], dy_top) @ _decoded(s["w_c"], i, o).t()).to(dt),
            "dw": s["c"] + _kept4(s["dy"].t(), dy_top) @ _kept4(s["x"].t(), x_top).t()}


def _decoded(a, rows, k):
    """The values, [rows][k], of an operand in hand."""
    two = a["codes"][:, :(k + 1) // 2]
    code = torch.stack((two & 15, two >> 4), 2).flatten(1)[:, :k].int()
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    table = torch.cat((table, -table))
    s = _grid(a["scale"], rows, (k + 15) // 16).contiguous().view(torch.float8_e4m3fn)
    return _values4(table[code], s, a["top"])


# ------------------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4

    def codes(r, c):  # a 4-bit copy's codes and scales
        return r * ((c + 1) // 2) + r * ((c + 15) // 16)

    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        if case["dir"] == "backward":  # dy, dsum, x, dx
            return {"bytes": 4 * r * c * e + 8 * c + 4 * r, "flops": 10 * r * c}
        if case["to"] == "values":  # x, residual, sum, y
            return {"bytes": 4 * r * c * e + 4 * c + 4 * r + 4, "flops": 5 * r * c}
        # x, residual, sum, codes and scales written and read, the values in BF16
        return {"bytes": 3 * r * c * e + 2 * (r * c + r * ((c + 127) // 128)) + 2 * r * c + 4 * c + 4 * r, "flops": 7 * r * c}
    if case["op"] == "quantise":
        r, c = case["rows"], case["cols"]
        # the input twice (its largest magnitude decides every code), both copies written and read, both restored
        return {"bytes": 2 * r * c * e + 2 * (codes(r, c) + codes(c, r)) + 2 * r * c * e, "flops": 8 * r * c}
    if case["op"] == "product":
        m, n, k = _sizes(case)
        b = codes(m, k) + codes(n, k) + m * n * e
        return {"bytes": b + (m * n * 4 if case["kind"] == "weight_grad" else 0), "flops": 2 * m * n * k}
    t, o, i = case["tokens"], case["outs"], case["ins"]
    b = 2 * t * (o + i) * e + 2 * (codes(t, i) + codes(i, t) + codes(t, o) + codes(o, t))
    return {"bytes": b + codes(o, i) + codes(i, o) + t * (o + i) * e + 2 * o * i * 4, "flops": 6 * t * o * i}


# ------------------------------------------------------------------------------ in 64 bits
def _nearest(v, bits, least, most):
    """The nearest multiples of a quantum, ties to even: 2^(bits - 1) quanta to a value's power of two,
    `least` the smallest quantum, saturating at `most`."""
    v = v.clamp(-most, most)
    power = torch.where(v == 0, 0.0, v.abs() / torch.frexp(v.abs()).mantissa)  # in (|v|, 2 |v|]
    quantum = (power * 2.0 ** -bits).clamp(min=least)
    return (v / quantum).round().mul(quantum).clamp(-most, most)


def _r32(v):
    return v.float().double()


def _exact8(y):
    """Values kept by E4M3 codes, a scale 2^max(p - 8, -127) per 128 values of largest magnitude in [2^p, 2^(p+1))."""
    kept = torch.empty_like(y)
    for k in range(0, y.shape[1], 128):
        part = y[:, k:k + 128]
        top = part.abs().amax(1, keepdim=True)
        scale = (torch.where(top == 0, 0.0, top / torch.frexp(top).mantissa) * 2.0 ** -9).clamp(min=2.0 ** -127)
        kept[:, k:k + 128] = _nearest(part / scale, 4, 2.0 ** -9, 448.0) * scale
    return kept


def _exact4(x):
    """Values kept by NVFP4 codes, in blocks of 16 along the rows; the definition's roundings to 32 bits are made."""
    x = x.double()
    top = x.abs().amax()
    S = _r32(2688.0 / top).clamp(max=LARGEST) if float(top) else torch.ones_like(top)
    kept = torch.empty_like(x)
    for k in range(0, x.shape[1], 2048):
        c = min(2048, x.shape[1] - k)
        part = torch.nn.functional.pad(x[:, k:k + c], (0, -c % 16)).unflatten(1, (-1, 16))
        s = _nearest(_r32(_r32(part.abs().amax(2, keepdim=True) / 6.0) * S), 4, 2.0 ** -9, 448.0)
        q = _nearest(_r32(part * torch.where(s == 0, 0.0, _r32(S / s))), 2, 0.5, 6.0)
        kept[:, k:k + c] = (q * s / S).flatten(1)[:, :c]
    return kept


def exact(case, seed):
    s = _activations(case, seed)
    if case["op"] == "norm":
        x, w = s["x"].double(), s["weight"].double()
        if case["dir"] == "forward":
            x = x + s["residual"].double()
            rstd = 1 / torch.sqrt(torch.linalg.vector_norm(x, dim=1).square() / x.shape[1] + EPS)
            got = {"sum": x, "rstd": rstd}
            y = torch.einsum("rc,r,c->rc", x, rstd, w)
            if case["to"] == "codes":
                return got | {"y": _exact8(y)}
            return got | {"y": y, "top": y.to(s["x"].dtype).double().abs().amax().view(1)}  # of y as it is stored
        # the saved statistic is an input: what the forward pass left in 32 bits
        rstd = (s["x"].float().square().mean(1) + EPS).rsqrt().double()
        dy = s["dy"].double()
        along = torch.einsum("rc,c,rc->r", dy, w, x) * rstd ** 3 / x.shape[1]
        dx = torch.einsum("rc,c,r->rc", dy, w, rstd) - x * along[:, None] + s["dsum"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc,r->c", dy, x, rstd)}
    if case["op"] == "quantise":
        return {"top": s["x"].double().abs().amax().view(1), "r": _exact4(s["x"]), "c": _exact4(s["x"].t())}
    if case["op"] == "product":
        if case["kind"] == "output":
            return torch.einsum("tk,nk->tn", _exact4(s["x"]), _exact4(s["w"]))
        if case["kind"] == "input_grad":
            return torch.einsum("tk,nk->tn", _exact4(s["dy"]), _exact4(s["w"].t()))
        return s["c"].double() + torch.einsum("mt,nt->mn", _exact4(s["dy"].t()), _exact4(s["x"].t()))
    return {"y": torch.einsum("tk,nk->tn", _exact4(s["x"]), _exact4(s["w"])),
            "dx": torch.einsum("tk,nk->tn", _exact4(s["dy"]), _exact4(s["w"].t())),
            "dw": s["c"].double() + torch.einsum("mt,nt->mn", _exact4(s["dy"].t()), _exact4(s["x"].t()))}
