"""Cases of what a training step runs between its products and the optimizer: the root-mean-square norm with the
residual's addition and an 8-bit operand, forward and backward; the global gradient norm with clipping into the
shard's flat gradient; microscaled 4-bit quantisation and product, alone and as a layer's backward pass.

Where `own` is false every case runs in elementary torch operations (fp32, long sums in fp64); where it is true it
makes the calls of the library's Python binding.  Byte buffers in the library's layouts:

* 8-bit operand: rows of codes with a pitch of the next multiple of 128, from the next multiple of 256 bytes on one
  scale byte (exponent + 127) per row and block of 128 columns, with a pitch of the next multiple of 4;
* 4-bit operand (e2m1): rows of codes, two in a byte with the even column in the low half and a pitch of the next
  multiple of 256 codes, from the next multiple of 256 bytes on one scale byte (exponent + 127) per row and block of
  32 columns, with a pitch of the next multiple of 16.
"""
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 9, "e5m2": 16}  # the largest value of a format is 0.875 * 2^TOP
EPS = 1e-6
WORKSPACE = 64 << 20  # bytes: covers every call


def listed():
    return [
        # one token's hidden state on its way into a projection: a call's latency
        {"name": "norm-one-token", "op": "norm", "rows": 1, "cols": 2048, "dtype": "bf16", "residual": True, "out": "operand", "fmt": "e4m3"},
        # 16384 tokens of the 1B decoder in training: residual stream, statistics, both orientations of the operand
        {"name": "norm-training-16384", "op": "norm", "rows": 16384, "cols": 2048, "dtype": "bf16", "residual": True, "out": "both", "fmt": "e4m3"},
        # its backward pass: gradient of both paths, weight gradient added into the shard's
        {"name": "norm-backward-16384", "op": "norm_backward", "rows": 16384, "cols": 2048, "dtype": "bf16", "residual": True},
        # backward on 13 images of 197 tokens at width 768, fp32
        {"name": "norm-backward-vit-f32", "op": "norm_backward", "rows": 2561, "cols": 768, "dtype": "f32", "residual": True},
        # the norm weights of the 1B decoder alone, 64 vectors of 2048: latency over many small tensors
        {"name": "clip-vectors", "op": "clip", "layers": 16, "width": 2048, "inner": 0, "squares": 0, "flat": 0, "dtype": "f32", "clipped": True},
        # bf16 gradients of four decoder layers, 44 tensors, into the fp32 gradient that the optimizer step reads
        {"name": "clip-layers-bf16", "op": "clip", "layers": 4, "width": 2048, "inner": 8192, "squares": 4, "flat": 0, "dtype": "bf16", "clipped": True},
        # the flat fp32 gradient of the 1B decoder's half shard
        {"name": "clip-half-shard", "op": "clip", "layers": 0, "width": 0, "inner": 0, "squares": 0, "flat": 639697920, "dtype": "f32", "clipped": True},
        # the fp32 master weight of an MLP projection after an optimizer step, both directions, and the values it now has
        {"name": "mx-weight-f32", "op": "mx_values", "rows": 8192, "cols": 2048, "dtype": "f32", "tile": True},
        # one token through the MLP's down projection
        {"name": "mx-one-token", "op": "mx_matmul", "m": 1, "n": 2048, "k": 8192, "out": "bf16", "addend": False},
        # MLP up projection of the 1B decoder on 4096 tokens
        {"name": "mx-mlp-up", "op": "mx_matmul", "m": 4096, "n": 8192, "k": 2048, "out": "bf16", "addend": False},
        # qkv weight gradient over 2561 tokens (no multiple of a block), added into the fp32 gradient shard
        {"name": "mx-weight-gradient-vit", "op": "mx_matmul", "m": 2304, "n": 768, "k": 2561, "out": "f32", "addend": True},
        # backward of the down projection on 8192 tokens, fp16: quantise the gradient, input gradient, weight gradient
        {"name": "mx-backward-8192", "op": "mx_backward", "m": 8192, "n": 2048, "k": 8192, "dtype": "f16"},
    ]


def _size(rng, low, high):
    """A size spread over its logarithm; every other one a multiple of 64 where that fits."""
    n = int(round(low * (high / low) ** rng.random()))
    return max(64, n // 64 * 64) if n > 64 and rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_backward", "norm_backward", "clip", "clip", "mx_values", "mx_matmul", "mx_matmul", "mx_backward"])
    dtype = rng.choice(sorted(DT))
    if op in ("norm", "norm_backward", "mx_values"):
        rows, cols = _size(rng, 1, 16384), _size(rng, 64, 16384)
        while rows * cols > 1 << 25:
            rows = rows // 2
        if op == "mx_values":
            return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "tile": rng.random() < 0.5}
        case = {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "residual": rng.random() < 0.6}
        return {**case, "out": rng.choice(["y", "operand", "both"]), "fmt": rng.choice(sorted(FP8))} if op == "norm" else case
    if op == "clip":
        case = {"op": op, "layers": 0, "width": 0, "inner": 0, "squares": 0, "flat": 0, "dtype": dtype, "clipped": rng.random() < 0.7}
        if rng.random() < 0.3:
            return {**case, "flat": _size(rng, 1000, 1 << 28)}
        width, inner, layers = _size(rng, 64, 4096), rng.choice([0, _size(rng, 64, 8192)]), _size(rng, 1, 24)
        squares = rng.choice([0, 4])
        while layers > 1 and layers * (squares * width + 3 * inner) * width > 1 << 28:
            layers //= 2
        return {**case, "layers": layers, "width": width, "inner": inner, "squares": squares}
    m, n, k = _size(rng, 1, 16384), _size(rng, 64, 16384), _size(rng, 64, 16384)
    while m * n * k > 1 << (37 if op == "mx_backward" else 38) or m * max(n, k) > 1 << 27:
        m = m // 2
    if op == "mx_matmul":
        return {"op": op, "m": m, "n": n, "k": k, "out": dtype, "addend": rng.random() < 0.5}
    return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["bf16", "f16"])}


# --- layouts ------------------------------------------------------------------------------------------------

def _up(x, a):
    return (x + a - 1) // a * a


def _layout8(rows, cols):
    pitch, scale_pitch = _up(cols, 128), _up(_up(cols, 128) // 128, 4)
    scale_off = _up(rows * pitch, 256)
    return pitch, scale_off, scale_pitch, _up(scale_off + rows * scale_pitch, 256)


def _layout4(rows, cols):
    pitch, scale_pitch = _up(cols, 256) // 2, _up(_up(cols, 256) // 32, 16)
    scale_off = _up(rows * pitch, 256)
    return pitch, scale_off, scale_pitch, _up(scale_off + rows * scale_pitch, 256)


def _buffer(layout):
    return torch.zeros(layout[3], dtype=torch.uint8, device="cuda")


def _views8(buf, rows, cols, fmt):
    """(codes [rows, cols] as 8-bit floats, scales [rows, blocks] as 8-bit powers of two) of an 8-bit operand."""
    pitch, scale_off, scale_pitch, _ = _layout8(rows, cols)
    codes = buf[: rows * pitch].view(FP8[fmt]).view(rows, pitch)[:, :cols]
    scales = buf[scale_off: scale_off + rows * scale_pitch].view(rows, scale_pitch)[:, : _up(cols, 128) // 128]
    return codes, scales.view(torch.float8_e8m0fnu)


# --- plain forms --------------------------------------------------------------------------------------------

def _power(e):
    """2^e in fp32 for integers -127 <= e <= 127."""
    return torch.where(e == -127, 0x400000, (e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x, width, tile, over):
    """A matrix in fp32 padded to whole blocks, as [block rows, rows, block columns, columns], and the exponent of each
    block's scale: its largest magnitude a = m 2^e, 0.5 <= m < 1, at most `over` times the scale."""
    rows, cols = x.shape
    high = width if tile else 1
    z = torch.zeros(_up(rows, high), _up(cols, width), device=x.device)
    z[:rows, :cols] = x
    z = z.view(-1, high, z.shape[1] // width, width)
    a = z.abs().amax((1, 3))
    m, e = torch.frexp(a)
    most, top = over
    return z, torch.where(a > 0, e - top + (m > most).to(e.dtype), -127).clamp(min=-127)


def _quantize8(x, fmt):
    """(codes, scales) of a matrix, blocks of 128 along its rows."""
    z, e = _blocks(x, 128, False, (0.875, TOP[fmt]))
    codes = (z * _power(-e)[:, None, :, None]).view(-1, _up(x.shape[1], 128)).to(FP8[fmt])
    return codes[:, : x.shape[1]], (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _quantize4(x, tile):
    """(values over their scales, exponents [rows, blocks]) of a matrix, blocks of 32 along its rows or 32 x 32."""
    rows, cols = x.shape
    z, e = _blocks(x, 32, tile, (0.75, 3))
    v = z * _power(-e)[:, None, :, None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    v = torch.round(v / step) * step
    return v.view(-1, _up(cols, 32))[:rows, :cols], e.repeat_interleave(32 if tile else 1, 0)[:rows]


def _values4(x, tile):
    v, e = _quantize4(x, tile)
    return v * _power(e).repeat_interleave(32, 1)[:, : x.shape[1]]


def _pack4(x, tile):
    """The 4-bit operand's bytes of a matrix."""
    rows, cols = x.shape
    pitch, scale_off, scale_pitch, _ = layout = _layout4(rows, cols)
    v, e = _quantize4(x.float(), tile)
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    full = torch.zeros(rows, pitch * 2, dtype=torch.uint8, device=x.device)
    full[:, :cols] = code
    buf = _buffer(layout)
    buf[: rows * pitch].view(rows, pitch).copy_(full[:, 0::2] | full[:, 1::2] << 4)
    buf[scale_off: scale_off + rows * scale_pitch].view(rows, scale_pitch)[:, : e.shape[1]] = (e + 127).to(torch.uint8)
    return buf


def _unpack4(buf, rows, cols):
    """fp32 values of a 4-bit operand."""
    pitch, scale_off, scale_pitch, _ = _layout4(rows, cols)
    q = buf[: rows * pitch].view(rows, pitch)
    code = torch.stack([q & 15, q >> 4], 2).view(rows, pitch * 2)[:, :cols].to(torch.int32)
    a = (code & 7).float()
    a = torch.where(a < 4, a / 2, torch.where(a < 6, a - 2, a * 2 - 8))
    e = buf[scale_off: scale_off + rows * scale_pitch].view(rows, scale_pitch).to(torch.int32) - 127
    return torch.where(code >= 8, -a, a) * _power(e).repeat_interleave(32, 1)[:, :cols]


def _norm(x, residual, weight, dtype):
    """(h, 1 / root mean square, normalised and weighted in fp32)."""
    h = x if residual is None else (x.float() + residual.float()).to(dtype)
    v = h.float()
    r = torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    return h, r, v * r * weight


# --- inputs -------------------------------------------------------------------------------------------------

def _normal(gen, rows, cols, std, dtype="f32"):
    return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(DT[dtype])


def _activations(gen, rows, cols, dtype):
    """Normal values with a few channels some 20 times larger, as hidden states have them."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    big = torch.rand(cols, generator=gen, device="cuda") < 0.004
    return (x * torch.where(big, 20.0, 1.0)).to(DT[dtype])


def _sizes(case):
    """Elements of each gradient: a flat piece, or layers of square and inner matrices and four vectors."""
    w = case["width"]
    layer = [w * w] * case["squares"] + [w * case["inner"]] * (3 if case["inner"] else 0) + [w] * 4
    return [case["flat"]] if case["flat"] else layer * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 2 + 1)
    s, op = dict(case), case["op"]
    s["workspace"] = torch.empty(WORKSPACE, dtype=torch.uint8, device="cuda")
    if op in ("norm", "norm_backward"):
        r, c, d = case["rows"], case["cols"], case["dtype"]
        s["weight"] = 1 + torch.randn(c, generator=gen, device="cuda") * 0.2
        s["x"] = _activations(gen, r, c, d)
        if op == "norm":
            s["residual"] = _activations(gen, r, c, d) if case["residual"] else None
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["y"], s["rstd"] = torch.empty_like(s["x"]), torch.empty(r, device="cuda")
            s["q"], s["qt"] = _buffer(_layout8(r, c)), _buffer(_layout8(c, r))
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = _normal(gen, r, c, 0.01, d)
            s["dresidual"] = _normal(gen, r, c, 0.01, d) if case["residual"] else None
            s["grad"] = torch.randn(c, generator=gen, device="cuda") * 0.05  # the shard's gradient so far
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty(c, device="cuda")
    elif op == "clip":
        sizes, d = _sizes(case), DT[case["dtype"]]
        spread = torch.rand(len(sizes), generator=gen, device="cuda").mul_(1.5).add_(0.5).mul_(1e-3).tolist()
        s["grads"] = [torch.randn(n, generator=gen, device="cuda").mul_(a).to(d) for n, a in zip(sizes, spread)]
        s["flat_grad"] = torch.empty(sum(sizes), device="cuda")
        size = sum(n * a * a for n, a in zip(sizes, spread)) ** 0.5  # about the norm
        s["max_norm"] = size * (0.5 if case["clipped"] else 2.0)
        s["sumsq"] = torch.empty(1, dtype=torch.float64, device="cuda")
        s["norm"] = torch.empty(1, device="cuda")
    elif op == "mx_values":
        r, c = case["rows"], case["cols"]
        s["x"] = _normal(gen, r, c, 0.02, case["dtype"]) if case["tile"] else _activations(gen, r, c, case["dtype"])
        s["q"], s["qt"] = _buffer(_layout4(r, c)), _buffer(_layout4(c, r))
        s["v"] = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
        s["vt"] = torch.empty(c, r, dtype=torch.bfloat16, device="cuda")
    elif op == "mx_matmul":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"] = _pack4(_activations(gen, m, k, "bf16"), False)
        s["b"] = _pack4(_normal(gen, n, k, 0.02), True)
        s["addend"] = _normal(gen, m, n, 1.0, case["out"]) if case["addend"] else None
        s["c"] = torch.empty(m, n, dtype=DT[case["out"]], device="cuda")
    else:
        m, n, k, d = case["m"], case["n"], case["k"], case["dtype"]
        s["wt"] = _pack4(_normal(gen, n, k, 0.02).t(), True)
        s["xt"] = _pack4(_activations(gen, m, k, d).t(), False)
        s["dy"] = _normal(gen, m, n, 0.01, d)
        s["grad"] = _normal(gen, n, k, 0.05)  # the shard's gradient so far
        s["gq"], s["gt"] = _buffer(_layout4(m, n)), _buffer(_layout4(n, m))
        s["dx"] = torch.empty(m, k, dtype=DT[d], device="cuda")
        s["dw"] = torch.empty(n, k, device="cuda")
    if op == "clip" and own:
        from communication_compressed_optimizer_elt_amd import binding as L

        # the lists of gradients and of their places in the flat gradient, which a program makes once
        s["src"] = L.Tensors(s["grads"])
        s["dst"] = L.Tensors(s["flat_grad"].split([g.numel() for g in s["grads"]]))
    return s


# --- one pass -----------------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "norm":
        h, r, y = _norm(s["x"], s["residual"], s["weight"], s["x"].dtype)
        out = {"h": h} if s["residual"] is not None else {}
        if s["out"] == "y":
            return {**out, "y": y.to(h.dtype), "rstd": r[:, 0]}
        out["q"], out["scale"] = _quantize8(y, s["fmt"])
        if s["out"] == "both":
            out["rstd"] = r[:, 0]
            out["qt"], out["scale_t"] = _quantize8(y.t(), s["fmt"])
        return out
    if op == "norm_backward":
        r, g = s["rstd"][:, None], s["dy"].float()
        n = s["x"].float() * r
        gw = g * s["weight"]
        dx = (gw - n * (gw * n).mean(1, keepdim=True)) * r
        dx = dx if s["dresidual"] is None else dx + s["dresidual"].float()
        return {"dx": dx.to(s["x"].dtype), "dw": s["grad"] + (g * n).double().sum(0).float()}
    if op == "clip":
        norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt()
        scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
        return {"flat": torch.cat([g.float() * scale for g in s["grads"]]), "norm": norm.float()[None]}
    if op == "mx_values":
        x = s["x"].float()
        return {"v": _values4(x, s["tile"]).bfloat16(), "vt": _values4(x.t(), s["tile"]).bfloat16()}
    m, n, k = s["m"], s["n"], s["k"]
    if op == "mx_matmul":
        c = _unpack4(s["a"], m, k) @ _unpack4(s["b"], n, k).t()
        return (c if s["addend"] is None else s["addend"].float() + c).to(DT[s["out"]])
    g = s["dy"].float()
    dx = _values4(g, False) @ _unpack4(s["wt"], k, n).t()
    dw = _values4(g.t(), False) @ _unpack4(s["xt"], k, m).t()
    return {"dx": dx.to(DT[s["dtype"]]), "dw": s["grad"] + dw}


def _run_own(s):
    from communication_compressed_optimizer_elt_amd import binding as L

    op, ws = s["op"], s["workspace"]
    if op == "norm":
        cfg = L.Norm(eps=EPS, fmt={"e4m3": L.FMT_E4M3, "e5m2": L.FMT_E5M2}[s["fmt"]])
        x, (rows, cols) = s["x"], s["x"].shape
        out = {"h": s["h"]} if s["residual"] is not None else {}
        if s["out"] == "y":
            L.demo_rms_norm(cfg, x, s["weight"], y=s["y"], residual=s["residual"], h=s["h"], rstd=s["rstd"])
            return {**out, "y": s["y"], "rstd": s["rstd"]}
        if s["out"] == "operand":
            L.demo_rms_norm(cfg, x, s["weight"], residual=s["residual"], h=s["h"], operand=s["q"])
        else:
            L.demo_rms_norm(cfg, x, s["weight"], residual=s["residual"], h=s["h"], rstd=s["rstd"], operand=s["q"], operand_t=s["qt"])
            out["rstd"] = s["rstd"]
            out["qt"], out["scale_t"] = _views8(s["qt"], cols, rows, s["fmt"])
        out["q"], out["scale"] = _views8(s["q"], rows, cols, s["fmt"])
        return out
    if op == "norm_backward":
        L.demo_rms_norm_backward(L.Norm(eps=EPS), s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], dresidual=s["dresidual"],
                                 dweight=s["dw"], addend=s["grad"], workspace=ws)
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "clip":
        L.demo_grad_norm(s["src"], s["sumsq"], workspace=ws)
        L.demo_grad_clip(s["src"], s["sumsq"], s["max_norm"], dst=s["dst"], norm=s["norm"])
        return {"flat": s["flat_grad"], "norm": s["norm"]}
    if op == "mx_values":
        L.demo_mx_quantize(L.Mx(tile=int(s["tile"])), s["x"], s["q"], s["qt"])
        L.demo_mx_dequantize(s["q"], s["v"])
        L.demo_mx_dequantize(s["qt"], s["vt"])
        return {"v": s["v"], "vt": s["vt"]}
    m, n, k = s["m"], s["n"], s["k"]
    if op == "mx_matmul":
        L.demo_mx_matmul(L.Mx(), m, n, k, s["a"], s["b"], s["c"], addend=s["addend"], workspace=ws)
        return s["c"]
    L.demo_mx_quantize(L.Mx(), s["dy"], s["gq"], s["gt"])
    L.demo_mx_matmul(L.Mx(), m, k, n, s["gq"], s["wt"], s["dx"], workspace=ws)
    L.demo_mx_matmul(L.Mx(), n, k, m, s["gt"], s["xt"], s["dw"], addend=s["grad"], workspace=ws)
    return {"dx": s["dx"], "dw": s["dw"]}


# --- what a pass cannot do without --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, b, res = case["rows"] * case["cols"], BYTES[case["dtype"]], case["residual"]
        if op == "norm":
            out = {"y": b, "operand": 129 / 128, "both": 2 * 129 / 128}[case["out"]]
            return {"bytes": n * (b * (3 if res else 1) + out) + 4 * case["cols"], "flops": 5 * n}
        return {"bytes": n * b * (4 if res else 3) + 4 * case["rows"] + 12 * case["cols"], "flops": 10 * n}
    if op == "clip":
        n = sum(_sizes(case))
        return {"bytes": n * (BYTES[case["dtype"]] + 4), "flops": 3 * n}
    code = 17 / 32  # bytes of a 4-bit value with its share of the scale
    if op == "mx_values":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (BYTES[case["dtype"]] + 4 * code + 4), "flops": 3 * n}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "mx_matmul":
        return {"bytes": (m + n) * k * code + m * n * BYTES[case["out"]] * (2 if case["addend"] else 1), "flops": 2 * m * n * k}
    return {"bytes": m * n * 2 + n * k * code + m * k * code + m * k * 2 + n * k * 8, "flops": 4 * m * n * k}


# --- the definitions in 64 bits -----------------------------------------------------------------------------

def _scales64(x, width, tile, limit):
    """Exponents [rows, blocks] in fp64: the smallest from -127 on that keep a block within limit * 2^e."""
    h = width if tile else 1
    full = torch.nn.functional.pad(x, (0, -x.shape[1] % width, 0, -x.shape[0] % h))
    a = full.abs().unflatten(1, (-1, width)).unflatten(0, (-1, h)).amax((1, 3)) / limit
    e = torch.ceil(torch.log2(a)).clamp(min=-127)  # fp64's log2 is exact at powers of two, and no value here lies nearer to one than 2^-24
    return torch.where(a == 0, torch.full_like(e, -127), e).repeat_interleave(h, 0)[: x.shape[0]]


def _codes64(x, fmt):
    """(rounded codes, scales) of 8-bit blocks along the rows."""
    limit, digits, low = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}[fmt]
    e = _scales64(x, 128, False, limit)
    v = x * torch.exp2(-e).repeat_interleave(128, 1)[:, : x.shape[1]]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low) * (1 + 2.0 ** -40))) - digits)
    return torch.round(v / step) * step, torch.exp2(e)


def _values64(x, tile):
    """What 4-bit codes of a matrix stand for, by the middles between the format's values."""
    e = torch.exp2(_scales64(x, 32, tile, 6.0)).repeat_interleave(32, 1)[:, : x.shape[1]]
    a = (x / e).abs()
    middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    below, above = torch.bucketize(a, middle), torch.bucketize(a, middle, right=True)
    code = torch.where(below % 2 == 1, above, below)  # in the middle: the even one
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    return torch.copysign(grid[code], x) * e


def _operand64(buf, rows, cols):
    pitch, scale_off, scale_pitch, _ = _layout4(rows, cols)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=buf.device)
    q = buf[: rows * pitch].view(rows, pitch).long()
    v = torch.cat([grid, -grid])[torch.stack([q % 16, q // 16], 2).flatten(1)[:, :cols]]
    e = buf[scale_off: scale_off + rows * scale_pitch].view(rows, scale_pitch).double() - 127
    return v * torch.exp2(e).repeat_interleave(32, 1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        x = s["x"].double()
        h = x if s["residual"] is None else x + s["residual"].double()
        v = h.float().to(s["x"].dtype).double()  # statistics are of h as it is stored
        r = ((v * v).sum(1, keepdim=True) / case["cols"] + EPS) ** -0.5
        y = v * r * s["weight"].double()
        out = {"h": h} if s["residual"] is not None else {}
        if case["out"] == "y":
            return {**out, "y": y, "rstd": r[:, 0]}
        out["q"], out["scale"] = _codes64(y, case["fmt"])
        if case["out"] == "both":
            out["rstd"] = r[:, 0]
            out["qt"], out["scale_t"] = _codes64(y.t().contiguous(), case["fmt"])
        return out
    if op == "norm_backward":
        r, g, h, w = s["rstd"].double()[:, None], s["dy"].double(), s["x"].double(), s["weight"].double()
        along = (g * w * h).sum(1, keepdim=True) / case["cols"]
        dx = r * g * w - h * along * r ** 3
        return {"dx": dx if s["dresidual"] is None else dx + s["dresidual"].double(),
                "dw": s["grad"].double() + (g * h * r).sum(0)}
    if op == "clip":
        norm = sum(float((g.double() ** 2).sum()) for g in s["grads"]) ** 0.5
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"flat": torch.cat([g.double() * scale for g in s["grads"]]), "norm": torch.tensor([norm], dtype=torch.float64)}
    if op == "mx_values":
        x = s["x"].double()
        return {"v": _values64(x, case["tile"]), "vt": _values64(x.t().contiguous(), case["tile"])}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "mx_matmul":
        c = _operand64(s["a"], m, k) @ _operand64(s["b"], n, k).t()
        return c if s["addend"] is None else c + s["addend"].double()
    g = s["dy"].double()
    dx = _values64(g, False) @ _operand64(s["wt"], k, n).t()
    dw = _values64(g.t().contiguous(), False) @ _operand64(s["xt"], k, m).t()
    return {"dx": dx, "dw": s["grad"].double() + dw}
