"""Cases of the training operators around the MXFP8 weights: 8-bit activation checkpoints,
the block-scaled 8-bit matrix product, and layer norm.

    checkpoint  an activation (or gradient) is kept as E4M3 codes with one E8M0 scale per 128
                values, along its rows and along its columns, and both copies are restored
    product     D = A B^T (+ C) of 8-bit operands with a scale per block along the contraction
                (128 values; 32 for the weights the master-weight cast writes): a linear
                layer's output, its input's gradient and its weight's gradient
    linear      a linear layer's training step: both activations' checkpoints, three products
    norm        layer norm forward; backward with the gradients of weight and bias, from the
                saved input or from its 8-bit checkpoint

Scale convention: e = floor(log2(amax)) - 8 clamped at -127, byte e + 127 (0xFF for a block
with a NaN or an infinity), code = E4M3(x * 2^-e), nearest-even, saturating at 448.  Scales lie
in 128x4 tiles of 512 bytes: entry (r, c) of a tile at byte (r % 32) * 16 + (r / 32) * 4 + c.
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest weight-sized matrix of the package's workloads: a latency-bound call
        {"name": "checkpoint small", "op": "checkpoint", "rows": 160, "cols": 96, "dtype": "f32"},
        # the activations of one long training micro-batch
        {"name": "checkpoint large", "op": "checkpoint", "rows": 16384, "cols": 6144, "dtype": "bf16"},
        # serving: one new token through a square layer
        {"name": "product one token", "op": "product", "kind": "output", "tokens": 1, "outs": 4096,
         "ins": 4096, "block": 32, "dtype": "bf16"},
        # serving: a batch of decoding sequences through a wide layer
        {"name": "product 64 tokens", "op": "product", "kind": "output", "tokens": 64, "outs": 8192,
         "ins": 8192, "block": 32, "dtype": "bf16"},
        # nothing divides anything: ragged tiles, rows that no 16-byte load can follow
        {"name": "product ragged", "op": "product", "kind": "input_grad", "tokens": 1000, "outs": 999,
         "ins": 1111, "block": 128, "dtype": "f32"},
        # a prompt, or one training micro-batch, through a square layer
        {"name": "product 4096", "op": "product", "kind": "output", "tokens": 4096, "outs": 4096,
         "ins": 4096, "block": 128, "dtype": "bf16"},
        # a weight's gradient added to the gradient of the micro-batches before
        {"name": "product weight gradient", "op": "product", "kind": "weight_grad", "tokens": 8192,
         "outs": 2048, "ins": 8192, "block": 128, "dtype": "f32"},
        # one training step of a large linear layer
        {"name": "linear step", "op": "linear", "tokens": 8192, "outs": 8192, "ins": 8192, "block": 32,
         "dtype": "bf16"},
        # serving: one new token
        {"name": "norm one token", "op": "norm", "dir": "forward", "rows": 1, "cols": 4096, "dtype": "bf16"},
        # training forward over a long micro-batch
        {"name": "norm forward", "op": "norm", "dir": "forward", "rows": 16384, "cols": 6144, "dtype": "bf16"},
        # its backward, the input kept as an 8-bit checkpoint
        {"name": "norm backward", "op": "norm", "dir": "backward", "rows": 16384, "cols": 6144,
         "dtype": "bf16", "saved": "checkpoint"},
        # odd sizes in 32 bits, the input kept as it is
        {"name": "norm backward odd", "op": "norm", "dir": "backward", "rows": 1001, "cols": 1023,
         "dtype": "f32", "saved": "input"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer width: as often a multiple of 16 as not."""
    w = _log_int(rng, lo, hi)
    return max(lo, w // 16 * 16) if rng.random() < 0.5 else w


def draw(rng):
    op = rng.choice(["checkpoint", "product", "product", "product", "linear", "norm", "norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "checkpoint":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": _width(rng, 16, 6144), "dtype": dtype}
    if op == "product":
        kind = rng.choice(["output", "output", "input_grad", "weight_grad"])
        return {"op": op, "kind": kind, "tokens": _log_int(rng, 1, 8192), "outs": _width(rng, 64, 8192),
                "ins": _width(rng, 64, 8192), "block": 128 if kind == "weight_grad" else rng.choice([32, 128]),
                "dtype": "f32" if kind == "weight_grad" else dtype}
    if op == "linear":
        return {"op": op, "tokens": _log_int(rng, 16, 8192), "outs": _width(rng, 64, 8192),
                "ins": _width(rng, 64, 8192), "block": 32, "dtype": dtype}
    case = {"op": op, "dir": rng.choice(["forward", "backward"]), "rows": _log_int(rng, 1, 16384),
            "cols": _width(rng, 64, 6144), "dtype": dtype}
    if case["dir"] == "backward":
        case["saved"] = rng.choice(["input", "checkpoint"])
    return case


# ------------------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pitch(n):
    """Row stride of a buffer that the program lays out itself: whole 16-byte units."""
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


def _encode(x, block, dim):
    """(E4M3 codes, scale grid) of a matrix, in blocks of `block` along `dim`."""
    x = x.float() if dim == 1 else x.float().t()
    r, c = x.shape
    nb = (c + block - 1) // block
    b = torch.nn.functional.pad(x, (0, nb * block - c)).view(r, nb, block)
    top = b.abs().amax(2).view(torch.int32) >> 23
    byte = torch.where(top == 255, 255, (top - 8).clamp(min=0))
    mul = torch.where(byte == 255, math.nan, _power(127 - byte))
    q = (b * mul[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(r, nb * block)[:, :c]
    return (q if dim == 1 else q.t()), byte.to(torch.uint8)


def _tiled(grid):
    """A scale grid [rows][blocks] in 128x4 tiles, padded with zero bytes."""
    r, c = grid.shape
    R, C = (r + 127) // 128, (c + 3) // 4
    g = torch.nn.functional.pad(grid, (0, 4 * C - c, 0, 128 * R - r))
    return g.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _grid(tiled, r, c):
    """The scale grid that lies in 128x4 tiles."""
    R, C = (r + 127) // 128, (c + 3) // 4
    return tiled.view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * R, 4 * C)[:r, :c]


def _buffer(codes, pitch):
    """`codes` as the first columns of a buffer with the row stride `pitch`."""
    q = torch.zeros(codes.shape[0], pitch, dtype=torch.uint8, device="cuda")
    q[:, :codes.shape[1]] = codes.view(torch.uint8) if codes.is_contiguous() else codes.contiguous().view(torch.uint8)
    return q


def _u8(*shape):
    return torch.empty(*shape, dtype=torch.uint8, device="cuda")


def _sizes(case):
    """(m, n, k) of a product."""
    t, o, i = case["tokens"], case["outs"], case["ins"]
    return {"output": (t, o, i), "input_grad": (t, i, o), "weight_grad": (o, i, t)}[case["kind"]]


def _activations(case, seed):
    """The values that a case starts from."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]
    if case["op"] == "checkpoint":
        return {"x": _rows(case["rows"], case["cols"], g, dt, 1.0, True)}
    if case["op"] in ("product", "linear"):
        t, o, i = case["tokens"], case["outs"], case["ins"]
        got = {"x": _rows(t, i, g, dt, 1.0, True), "dy": _rows(t, o, g, dt, 1e-3),
               "w": _rows(o, i, g, torch.float32, 0.02)}
        if case.get("kind") == "weight_grad":
            got["c"] = _rows(o, i, g, torch.float32, 0.05)
        return got
    r, c = case["rows"], case["cols"]
    x = torch.randn(r, c, generator=g, device="cuda") * 1.5 + torch.randn(c, generator=g, device="cuda")
    got = {"x": x.to(dt), "weight": 1 + 0.1 * torch.randn(c, generator=g, device="cuda"),
           "bias": 0.1 * torch.randn(c, generator=g, device="cuda")}
    if case["dir"] == "backward":
        got["dy"] = _rows(r, c, g, dt, 1e-2)
    return got


def prepare(case, seed):
    s = {"case": case, **_activations(case, seed)}
    dt = _TYPES[case["dtype"]]
    if case["op"] == "checkpoint":
        r, c = case["rows"], case["cols"]
        s |= {"q_r": _u8(r, _pitch(c)), "q_c": _u8(r, _pitch(c)), "s_r": _u8(_scale_bytes(r, (c + 127) // 128)),
              "s_c": _u8(_scale_bytes(c, (r + 127) // 128)),
              "y_r": torch.empty(r, c, dtype=dt, device="cuda"), "y_c": torch.empty(r, c, dtype=dt, device="cuda")}
    elif case["op"] == "product":
        m, n, k = _sizes(case)
        kind, blk = case["kind"], case["block"]
        left = s["x"] if kind == "output" else s["dy"]
        right = s["x"] if kind == "weight_grad" else s["w"]
        # contraction along the rows of a stored matrix: its columnwise copy
        s["a_col"], s["b_col"] = kind == "weight_grad", kind != "output"
        qa, ga = _encode(left, 128, 0 if s["a_col"] else 1)
        qb, gb = _encode(right, blk, 0 if s["b_col"] else 1)
        s["a"], s["a_scale"] = _buffer(qa, _pitch(qa.shape[1])), _tiled(ga)
        # a weight's codes lie densely, as the cast writes them
        s["b"], s["b_scale"] = _buffer(qb, _pitch(qb.shape[1]) if kind == "weight_grad" else qb.shape[1]), _tiled(gb)
        s["out"] = torch.empty(m, n, dtype=dt, device="cuda")
        for name in ("x", "dy", "w"):
            del s[name]
    elif case["op"] == "linear":
        t, o, i, blk = case["tokens"], case["outs"], case["ins"], case["block"]
        for name, dim in (("w_r", 1), ("w_c", 0)):
            q, g = _encode(s["w"], blk, dim)
            s[name], s[name + "_scale"] = _buffer(q, i), _tiled(g)
        del s["w"]
        for name, width in (("x", i), ("dy", o)):
            s[name + "_r"], s[name + "_c"] = _u8(t, _pitch(width)), _u8(t, _pitch(width))
            s[name + "_r_scale"] = _u8(_scale_bytes(t, (width + 127) // 128))
            s[name + "_c_scale"] = _u8(_scale_bytes(width, (t + 127) // 128))
        s |= {"y": torch.empty(t, o, dtype=dt, device="cuda"), "dx": torch.empty(t, i, dtype=dt, device="cuda"),
              "dw": torch.empty(o, i, device="cuda")}
    else:
        r, c = case["rows"], case["cols"]
        x = s["x"].float()
        s |= {"mean": torch.empty(r, device="cuda"), "rstd": torch.empty(r, device="cuda")}
        if case["dir"] == "forward":
            s["y"] = torch.empty(r, c, dtype=dt, device="cuda")
        else:
            s["mean"] = x.mean(1)
            s["rstd"] = ((x - s["mean"][:, None]).square().mean(1) + EPS).rsqrt()
            s |= {"dx": torch.empty(r, c, dtype=dt, device="cuda"), "dweight": torch.empty(c, device="cuda"),
                  "dbias": torch.empty(c, device="cuda"), "saved": s["x"], "saved_scale": None}
            if case["saved"] == "checkpoint":
                q, g = _encode(x, 128, 1)
                s["saved"], s["saved_scale"] = _buffer(q, _pitch(c)), _tiled(g)
            del s["x"]
    if own:
        s["calls"] = _calls(case, s)
    return s


def _calls(case, s):
    """The framework's calls of one pass, their arguments marshalled once."""
    from mxfp8_master_weight_gb300 import api
    if case["op"] == "checkpoint":
        r, c = case["rows"], case["cols"]
        return [api.prepare_checkpoint_save(s["x"], s["q_r"], s["s_r"], s["q_c"], s["s_c"], r, c),
                api.prepare_checkpoint_restore(s["q_r"], s["s_r"], s["y_r"], r, c),
                api.prepare_checkpoint_restore(s["q_c"], s["s_c"], s["y_c"], r, c, colwise=True)]
    if case["op"] == "product":
        m, n, k = _sizes(case)
        return [api.prepare_gemm(s["a"], s["a_scale"], s["b"], s["b_scale"], s.get("c"), s["out"], m, n, k,
                                 a_colwise=s["a_col"], b_colwise=s["b_col"], a_block=128, b_block=case["block"])]
    if case["op"] == "linear":
        t, o, i, blk = case["tokens"], case["outs"], case["ins"], case["block"]
        return [api.prepare_checkpoint_save(s["x"], s["x_r"], s["x_r_scale"], s["x_c"], s["x_c_scale"], t, i),
                api.prepare_gemm(s["x_r"], s["x_r_scale"], s["w_r"], s["w_r_scale"], None, s["y"], t, o, i,
                                 b_block=blk),
                api.prepare_checkpoint_save(s["dy"], s["dy_r"], s["dy_r_scale"], s["dy_c"], s["dy_c_scale"], t, o),
                api.prepare_gemm(s["dy_r"], s["dy_r_scale"], s["w_c"], s["w_c_scale"], None, s["dx"], t, i, o,
                                 b_colwise=True, b_block=blk),
                api.prepare_gemm(s["dy_c"], s["dy_c_scale"], s["x_c"], s["x_c_scale"], None, s["dw"], o, i, t,
                                 a_colwise=True, b_colwise=True)]
    r, c = case["rows"], case["cols"]
    if case["dir"] == "forward":
        return [api.prepare_layer_norm_forward(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], r, c, EPS)]
    s["workspace"] = _u8(max(1, api.mxfp8_layer_norm_workspace_size(r, c)))
    return [api.prepare_layer_norm_backward(s["dy"], s["saved"], s["saved_scale"], s["weight"], s["mean"], s["rstd"],
                                            s["dx"], s["dweight"], s["dbias"], s["workspace"], r, c)]


# ------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        [c.call() for c in s["calls"]]
        if case["op"] == "checkpoint":
            return [s["y_r"], s["y_c"]]
        if case["op"] == "product":
            return s["out"]
        if case["op"] == "linear":
            return {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
        if case["dir"] == "forward":
            return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    dt = _TYPES[case["dtype"]]
    if case["op"] == "checkpoint":
        return [_kept(s["x"], 1).to(dt), _kept(s["x"], 0).to(dt)]
    if case["op"] == "product":
        m, n, k = _sizes(case)
        a = _values(s["a"], s["a_scale"], m, k, 128, s["a_col"])
        b = _values(s["b"], s["b_scale"], n, k, case["block"], s["b_col"])
        d = a @ b.t()
        return (d + s["c"] if "c" in s else d).to(dt)
    if case["op"] == "linear":
        t, o, i, blk = case["tokens"], case["outs"], case["ins"], case["block"]
        return {"y": (_kept(s["x"], 1) @ _values(s["w_r"], s["w_r_scale"], o, i, blk, False).t()).to(dt),
                "dx": (_kept(s["dy"], 1) @ _values(s["w_c"], s["w_c_scale"], i, o, blk, True).t()).to(dt),
                "dw": _kept(s["dy"], 0).t() @ _kept(s["x"], 0)}
    w = s["weight"]
    if case["dir"] == "forward":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        rstd = ((x - mean).square().mean(1, keepdim=True) + EPS).rsqrt()
        return {"y": ((x - mean) * rstd * w + s["bias"]).to(dt), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    r, c = case["rows"], case["cols"]
    x = s["saved"].float() if s["saved_scale"] is None else _values(s["saved"], s["saved_scale"], r, c, 128, False)
    rstd, dy = s["rstd"][:, None], s["dy"].float()
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _values(buffer, tiled, rows, k, block, colwise):
    """The values, [rows][k], that codes and scales stand for (colwise: stored [k][rows])."""
    q = buffer[:, :rows].t() if colwise else buffer[:, :k]
    v = q.contiguous().view(torch.float8_e4m3fn).float()
    nb = (k + block - 1) // block
    f = _power(_grid(tiled, rows, nb).int() - 127)
    return v * f.repeat_interleave(block, 1)[:, :k]


def _kept(x, dim):
    """What a checkpoint with blocks along `dim` keeps of x."""
    q, byte = _encode(x, 128, dim)
    f = _power(byte.int() - 127).repeat_interleave(128, 1)
    return q.float() * (f[:, :x.shape[1]] if dim == 1 else f[:, :x.shape[0]].t())


# ------------------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4

    def copies(r, c):  # both directions' codes and scales
        return 2 * r * c + r * ((c + 127) // 128) + c * ((r + 127) // 128)

    if case["op"] == "checkpoint":
        r, c = case["rows"], case["cols"]
        # the input, both copies written and read, both restored matrices
        return {"bytes": r * c * e + 2 * copies(r, c) + 2 * r * c * e, "flops": 4 * r * c}
    if case["op"] == "product":
        m, n, k = _sizes(case)
        b = m * k + m * ((k + 127) // 128) + n * k + n * ((k + case["block"] - 1) // case["block"]) + m * n * e
        return {"bytes": b + (m * n * 4 if case["kind"] == "weight_grad" else 0), "flops": 2 * m * n * k}
    if case["op"] == "linear":
        t, o, i, blk = case["tokens"], case["outs"], case["ins"], case["block"]
        b = t * (o + i) * e + 2 * copies(t, i) + 2 * copies(t, o) + t * (o + i) * e + o * i * 4
        return {"bytes": b + 2 * o * i + o * ((i + blk - 1) // blk) + i * ((o + blk - 1) // blk), "flops": 6 * t * o * i}
    r, c = case["rows"], case["cols"]
    if case["dir"] == "forward":
        return {"bytes": 2 * r * c * e + 8 * c + 8 * r, "flops": 8 * r * c}
    x = r * c + r * ((c + 127) // 128) if case["saved"] == "checkpoint" else r * c * e
    return {"bytes": 2 * r * c * e + x + 12 * c + 8 * r, "flops": 14 * r * c}


# ------------------------------------------------------------------------------ in 64 bits
def _exact_blocks(x, block, dim):
    """The values kept of a matrix, from the definition: a block with the largest magnitude in
    [2^p, 2^(p+1)) has the scale 2^max(p - 8, -127); each value becomes the nearest multiple of
    its quantum (2^-9 under 2^-6, else an eighth of its power of two), ties to even, at most 448."""
    x = x.double() if dim == 1 else x.double().t()
    kept = torch.empty_like(x)

    def power(v):  # the power of two in (|v|, 2|v|], exactly; 0 for 0
        return torch.where(v == 0, 0.0, v.abs() / torch.frexp(v.abs()).mantissa)

    for k in range(0, x.shape[1], block):
        part = x[:, k:k + block]
        scale = (power(part.abs().max(1, keepdim=True).values) * 2.0 ** -9).clamp(min=2.0 ** -127)
        v = part / scale
        quantum = (power(v.clamp(-448.0, 448.0)) * 2.0 ** -4).clamp(min=2.0 ** -9)
        kept[:, k:k + block] = (v / quantum).round().mul(quantum).clamp(-448.0, 448.0) * scale
    return kept if dim == 1 else kept.t()


def exact(case, seed):
    s = _activations(case, seed)
    if case["op"] == "checkpoint":
        return [_exact_blocks(s["x"], 128, 1), _exact_blocks(s["x"], 128, 0)]
    if case["op"] == "product":
        blk = case["block"]
        if case["kind"] == "output":
            return torch.einsum("tk,nk->tn", _exact_blocks(s["x"], 128, 1), _exact_blocks(s["w"], blk, 1))
        if case["kind"] == "input_grad":
            return torch.einsum("tk,kn->tn", _exact_blocks(s["dy"], 128, 1), _exact_blocks(s["w"], blk, 0))
        return s["c"].double() + torch.einsum("tm,tn->mn", _exact_blocks(s["dy"], 128, 0), _exact_blocks(s["x"], 128, 0))
    if case["op"] == "linear":
        blk = case["block"]
        return {"y": torch.einsum("tk,nk->tn", _exact_blocks(s["x"], 128, 1), _exact_blocks(s["w"], blk, 1)),
                "dx": torch.einsum("tk,kn->tn", _exact_blocks(s["dy"], 128, 1), _exact_blocks(s["w"], blk, 0)),
                "dw": torch.einsum("tm,tn->mn", _exact_blocks(s["dy"], 128, 0), _exact_blocks(s["x"], 128, 0))}
    x, w = s["x"].double(), s["weight"].double()
    if case["dir"] == "forward":
        var, mean = torch.var_mean(x, dim=1, correction=0)
        xh = (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None]
        return {"y": torch.addcmul(s["bias"].double(), xh, w), "mean": mean, "rstd": 1 / torch.sqrt(var + EPS)}
    # the saved statistics are inputs: what the forward pass left in 32 bits
    x32 = s["x"].float()
    mean = x32.mean(1)
    rstd = ((x32 - mean[:, None]).square().mean(1) + EPS).rsqrt()
    if case["saved"] == "checkpoint":
        x = _exact_blocks(s["x"], 128, 1)
    xh = (x - mean.double()[:, None]) * rstd.double()[:, None]
    dy = s["dy"].double()
    dxh = dy * w
    n = case["cols"]
    dx = (n * dxh - dxh.sum(1, keepdim=True) - xh * (dxh * xh).sum(1, keepdim=True)) * rstd.double()[:, None] / n
    return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xh), "dbias": dy.sum(0)}
