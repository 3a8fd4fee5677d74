"""Plain 64-bit forms of the norm, of gradient clipping and of the 4-bit operands (numpy), for their tests."""
import linear_forms as F
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def norm(h, weight, eps):
    """(1 / root mean square [rows], normalised and weighted)."""
    r = 1 / np.sqrt((h * h).mean(1) + eps)
    return r, h * r[:, None] * weight


def norm_backward(dy, h, weight, r, dresidual=0.0):
    """(dx, dweight) and the magnitudes that bound their roundings: mean|g n| and sum|dy n|."""
    n = h * r[:, None]
    g = dy * weight
    along = (g * n).mean(1, keepdims=True)
    dx = r[:, None] * (g - n * along) + dresidual
    return dx, (dy * n).sum(0), np.abs(g * n).mean(1, keepdims=True), np.abs(dy * n).sum(0)


def mx_round(v):
    """v rounded to the nearest e2m1 value, halves to the even code (|v| <= 6)."""
    a = np.abs(v)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    return np.copysign(np.rint(a / step) * step, v)


def mx_quantize(x, tile):
    """(codes' values, exponents [rows, blocks]) of a matrix; exponent 128 and zeros where a block is not finite."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    kb, h = -(-cols // 32), 32 if tile else 1
    full = np.zeros((-(-rows // h) * h, kb * 32))
    full[:rows, :cols] = np.abs(x)
    a = full.reshape(-1, h, kb, 32).max((1, 3))
    odd = ~np.isfinite(a)
    m, e = np.frexp(np.where(odd, 0, a) / 6.0)
    e = np.where(a > 0, e - (m == 0.5), -127).clip(-127).astype(np.int64)
    e = np.repeat(np.where(odd, 128, e), h, 0)[:rows]
    wide = np.repeat(e, 32, 1)[:, :cols]
    with np.errstate(invalid="ignore"):
        return np.where(wide == 128, 0.0, mx_round(np.ldexp(np.where(wide == 128, 0.0, x), -wide))), e


def mx_value(codes, e):
    wide = np.repeat(e, 32, 1)[:, : codes.shape[1]]
    return np.where(wide == 128, np.nan, np.ldexp(codes, wide))


def mx_layout(rows, cols):
    pitch = -(-cols // 256) * 128
    sp = -(-(pitch // 16) // 16) * 16
    so = -(-rows * pitch // 256) * 256
    return pitch, so, sp, -(-(so + rows * sp) // 256) * 256


def mx_pack(codes, e):
    """Operand bytes of code values and exponents."""
    rows, cols = codes.shape
    pitch, so, sp, total = mx_layout(rows, cols)
    code = np.zeros((rows, pitch * 2), np.uint8)
    code[:, :cols] = np.searchsorted(GRID, np.abs(codes)) + 8 * np.signbit(codes)
    buf = np.zeros(total, np.uint8)
    buf[: rows * pitch] = (code[:, 0::2] | code[:, 1::2] << 4).reshape(-1)
    s = np.zeros((rows, sp), np.uint8)
    s[:, : e.shape[1]] = e + 127
    buf[so: so + rows * sp] = s.reshape(-1)
    return buf


def mx_unpack(buf, rows, cols):
    """(codes' values, exponents, padding codes and bytes all zero) of operand bytes."""
    pitch, so, sp, _ = mx_layout(rows, cols)
    q = buf[: rows * pitch].reshape(rows, pitch)
    code = np.stack([q & 15, q >> 4], 2).reshape(rows, pitch * 2)
    s = buf[so: so + rows * sp].reshape(rows, sp)
    kb = -(-cols // 32)
    clean = not code[:, cols:].any() and not s[:, kb:].any()
    v = np.where(code & 8, -1.0, 1.0) * GRID[code & 7]
    return v[:, :cols], s[:, :kb].astype(np.int64) - 127, clean


def dropped(x, p, **kw):
    """x through a dropout's gradient, in fp32 as the kernels multiply."""
    mask = F.keep(x.size, p, **kw).reshape(x.shape)
    return np.where(mask, np.float32(x) * np.float32(F.scale(p)), np.float32(0)).astype(np.float64)
