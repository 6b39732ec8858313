"""Packed cache rows by their definition, in numpy: every operation rounded to fp32, as the header states it."""
import numpy as np

F16, F32 = np.float16, np.float32
DIMS = (32, 64, 96, 128, 160, 192, 224, 256)


def row_bytes(bits, dim):
    return -(-(dim * bits // 8 + dim // 32 * 4) // 16) * 16


def toward(x, up):
    """The nearest fp16 not below (up) or not above x (fp32 within +-65504)."""
    h = x.astype(F16)
    back = h.astype(np.float64)
    off = back < x if up else back > x
    with np.errstate(over="ignore"):  # (the step from the largest one is not taken)
        return np.where(off, np.nextafter(h, F16(np.inf if up else -np.inf)), h).astype(F16)


def pack(x, bits):
    """(codes uint8 [..., dim], steps fp16, bases fp16 [..., dim/32]) of x [..., dim] fp32."""
    top = F32((1 << bits) - 1)
    shape = x.shape
    x = x.astype(F32).reshape(*shape[:-1], shape[-1] // 32, 32)
    nan = np.isnan(x).any(-1)
    x = np.clip(np.where(np.isnan(x), F32(0), x), F32(-65504), F32(65504))
    m = toward(x.min(-1), False)
    d = toward((x.max(-1) - m.astype(F32)) / top, True)
    d = np.where(nan, F16(0), d)
    with np.errstate(divide="ignore"):
        r = np.where(d == 0, F32(0), F32(1) / d.astype(F32)).astype(F32)
    c = np.minimum(np.rint((x - m.astype(F32)[..., None]) * r[..., None]), top).astype(np.uint8)
    return c.reshape(shape), d, np.where(nan, F16(np.nan), m)


def to_bytes(codes, d, m, bits):
    """Rows uint8 [..., row_bytes] (unused bytes 0)."""
    if bits == 4:
        codes = codes[..., 0::2] | codes[..., 1::2] << 4
    row = np.concatenate([codes, d.view(np.uint8), m.view(np.uint8)], -1)
    pad = -row.shape[-1] % 16
    return np.concatenate([row, np.zeros((*row.shape[:-1], pad), np.uint8)], -1)


def parts(rows, bits, dim):
    """(codes, steps, bases) that rows of bytes hold, the codes as whole numbers."""
    n, g = dim * bits // 8, dim // 32
    b = rows[..., :n]
    codes = b if bits == 8 else np.stack([b & 15, b >> 4], -1).reshape(*rows.shape[:-1], dim)
    scale = np.ascontiguousarray(rows[..., n:n + 4 * g]).view(F16)
    return codes, scale[..., :g], scale[..., g:]


def values(rows, bits, dim):
    """The values of rows, in 64 bits (exact)."""
    c, d, m = parts(rows, bits, dim)
    return c.astype(np.float64) * np.repeat(d.astype(np.float64), 32, -1) + np.repeat(m.astype(np.float64), 32, -1)
