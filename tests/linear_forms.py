"""Plain 64-bit forms of the low-precision linear layer (numpy), for its tests."""
import numpy as np

M32 = np.uint64(0xFFFFFFFF)
FORMATS = {0: (448.0, 3, -6), 1: (57344.0, 2, -14)}  # largest value, mantissa bits, smallest normal exponent


def philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 on arrays of uint64 that hold 32-bit words."""
    c0, c1, c2, c3 = (np.asarray(c, dtype=np.uint64) for c in (c0, c1, c2, c3))
    for r in range(10):
        ka = np.uint64((k0 + r * 0x9E3779B9) & 0xFFFFFFFF)
        kb = np.uint64((k1 + r * 0xBB67AE85) & 0xFFFFFFFF)
        p0, p1 = c0 * np.uint64(0xD2511F53), c2 * np.uint64(0xCD9E8D57)
        c0, c1, c2, c3 = (p1 >> np.uint64(32)) ^ c1 ^ ka, p1 & M32, (p0 >> np.uint64(32)) ^ c3 ^ kb, p0 & M32
    return c0, c1, c2, c3


def threshold(p):
    return int(np.floor(float(np.float32(p)) * 65536 + 0.5))


def scale(p):
    t = threshold(p)
    return 0.0 if t == 65536 else float(np.float32(65536 / (65536 - t)))


def keep(n, p, seed=0, step=0, site=0, chunk_offset=0):
    b = np.arange((n + 7) // 8, dtype=np.uint64) + np.uint64(4 * chunk_offset)
    full = np.ones_like(b)
    w = philox(b & M32, b >> np.uint64(32), full * np.uint64(step & 0xFFFFFFFF), full * np.uint64(2 << 24 | site),
               seed & 0xFFFFFFFF, seed >> 32)
    draws = np.stack([np.stack([x & np.uint64(0xFFFF), x >> np.uint64(16)], 1) for x in w], 1).reshape(-1)[:n]
    return draws >= threshold(p)


def round_to(v, fmt):
    """v rounded to nearest even in the format (|v| within its range)."""
    _, digits, low = FORMATS[fmt]
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, low) - digits)
    return np.rint(v / step) * step


def quantize(x, fmt, tile):
    """(codes' values, exponents [rows, blocks]) of a matrix; NaN for what is not finite."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    kb, h = -(-cols // 128), 128 if tile else 1
    full = np.zeros((-(-rows // h) * h, kb * 128))
    full[:rows, :cols] = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = full.reshape(-1, h, kb, 128).max((1, 3))
    m, e = np.frexp(a / FORMATS[fmt][0])
    e = np.where(a > 0, e - (m == 0.5), -127).clip(-127).astype(np.int64)
    e = np.repeat(e, h, 0)[:rows]
    wide = np.repeat(e, 128, 1)[:, :cols]
    v = np.where(np.isfinite(x), x, 0.0)
    return np.where(np.isfinite(x), round_to(np.ldexp(v, -wide), fmt), np.nan), e


def value(codes, e):
    return np.ldexp(codes, np.repeat(e, 128, 1)[:, : codes.shape[1]])


def decode_codes(u, fmt):
    """Values of 8-bit codes."""
    u = np.asarray(u, dtype=np.int64)
    _, digits, low = FORMATS[fmt]
    bits = 7 - digits
    bias = (1 << (bits - 1)) - 1
    e, m = (u >> digits) & ((1 << bits) - 1), u & ((1 << digits) - 1)
    v = np.where(e == 0, np.ldexp(m.astype(float), low - digits), np.ldexp(1.0 + m / (1 << digits), e - bias))
    if fmt == 0:
        v = np.where((u & 0x7F) == 0x7F, np.nan, v)
    else:
        v = np.where(e == 31, np.where(m == 0, np.inf, np.nan), v)
    return np.where(u & 0x80, -v, v)


def encode_values(v, fmt):
    """Codes of values of the format."""
    table = decode_codes(np.arange(128), fmt)
    order = np.argsort(np.where(np.isfinite(table), table, np.inf), kind="stable")
    at = order[np.searchsorted(table[order], np.abs(v))]
    assert np.array_equal(table[at], np.abs(v))
    return (at + 128 * np.signbit(v)).astype(np.uint8)


def layout(rows, cols):
    pitch = -(-cols // 128) * 128
    sp = -(-(pitch // 128) // 4) * 4
    so = -(-rows * pitch // 256) * 256
    return pitch, so, sp, -(-(so + rows * sp) // 256) * 256


def pack(codes, e, fmt):
    """Operand bytes of code values and exponents."""
    rows, cols = codes.shape
    pitch, so, sp, total = layout(rows, cols)
    buf = np.zeros(total, np.uint8)
    q = np.zeros((rows, pitch), np.uint8)
    q[:, :cols] = encode_values(codes, fmt)
    buf[: rows * pitch] = q.reshape(-1)
    s = np.zeros((rows, sp), np.uint8)
    s[:, : e.shape[1]] = e + 127
    buf[so: so + rows * sp] = s.reshape(-1)
    return buf


def unpack(buf, rows, cols, fmt):
    """(codes' values, exponents, padding bytes all zero) of operand bytes."""
    pitch, so, sp, _ = layout(rows, cols)
    q = buf[: rows * pitch].reshape(rows, pitch)
    s = buf[so: so + rows * sp].reshape(rows, sp)
    kb = pitch // 128
    clean = not q[:, cols:].any() and not s[:, kb:].any()
    return decode_codes(q[:, :cols], fmt), s[:, :kb].astype(np.int64) - 127, clean
