"""Float64 numpy oracle of the dense FP4 operators.

Written from the definitions.  Test infrastructure only: it shares no code with
the GPU path."""
import numpy as np

NVFP4, MXFP4 = 0, 1
BLOCK = {NVFP4: 16, MXFP4: 32}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_value(byte):
    """E4M3 (no infinities; 0x7F is NaN) of bytes without a sign."""
    b = np.asarray(byte, dtype=np.int64)
    e, m = b >> 3, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0))
    return np.where(b == 0x7F, np.nan, v)


def nearest(x, table):
    """Index of the entry of an ascending table that is nearest to x >= 0, ties to the even index."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    low, high = x - table[lo], table[hi] - x
    return np.where((low < high) | ((low == high) & (lo % 2 == 0)), lo, hi)


E4M3 = e4m3_value(np.arange(0x7F))  # 0 to 448


def scale_value(byte, format):
    byte = np.asarray(byte)
    if format == NVFP4:
        return e4m3_value(byte)
    return np.where(byte == 255, np.nan, 2.0 ** (byte.astype(np.float64) - 127))


def quantize(x, format):
    """x [rows, cols] (FP32 values) -> codes [rows, cols] (0..15), scales
    [rows, blocks] bytes, row scales [rows] or None."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    g = BLOCK[format]
    codes = np.zeros((rows, cols), dtype=np.uint8)
    scales = np.zeros((rows, cols // g), dtype=np.uint8)
    row_scale = np.ones(rows) if format == NVFP4 else None
    for r in range(rows):
        if format == NVFP4:
            if not np.isfinite(x[r]).all():
                row_scale[r] = np.nan
                continue
            top, e = float(np.abs(x[r]).max()), -126
            while 2688.0 * 2.0 ** e < top:
                e += 1
            row_scale[r] = 2.0 ** e
            y = np.ldexp(x[r], -e).astype(np.float32).reshape(-1, g)
            big = np.abs(y).max(1)
            scales[r] = nearest((big / np.float32(6)).astype(np.float64), E4M3)
            s = E4M3[scales[r]].astype(np.float32)
            q = y / np.where(s == 0, np.float32(np.inf), s)[:, None]
            keep = (s != 0)[:, None]
        else:
            y = x[r].reshape(-1, g).astype(np.float64)
            big = np.abs(y).max(1)
            with np.errstate(invalid="ignore"):
                fine = np.isfinite(big)
                e = np.full(len(big), -127)
                while (fine & (6.0 * 2.0 ** e.astype(np.float64) < big)).any():
                    e = e + (fine & (6.0 * 2.0 ** e.astype(np.float64) < big))
                scales[r] = np.where(fine, e + 127, 255)
                q = y / (2.0 ** e.astype(np.float64))[:, None]
            keep = fine[:, None]
        with np.errstate(invalid="ignore"):
            c = nearest(np.abs(q.astype(np.float64)), E2M1[:8]) + 8 * np.signbit(q)
        codes[r] = np.where(keep, c, 0).reshape(-1)
    return codes, scales, row_scale


def values(codes, scales, row_scale, format):
    v = E2M1[codes].reshape(codes.shape[0], -1, BLOCK[format]) * scale_value(scales, format)[..., None]
    v = v.reshape(codes.shape)
    return v if row_scale is None else v * np.asarray(row_scale, dtype=np.float64)[:, None]


def pack(codes):
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(packed):
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def tile(scales, fill=0):
    """Row-major scales [rows, blocks] in tiles of 128 rows x 4 blocks."""
    rows, blocks = scales.shape
    kt, rt = -(-blocks // 4), -(-rows // 128)
    full = np.full((rt * 128, kt * 4), fill, dtype=np.uint8)
    full[:rows] = 0
    full[:rows, :blocks] = scales
    return full.reshape(rt, 4, 32, kt, 4).transpose(0, 3, 2, 1, 4).reshape(-1)


def untile(tiled, rows, blocks):
    kt, rt = -(-blocks // 4), -(-rows // 128)
    return tiled.reshape(rt, kt, 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :blocks]


def swiglu(gate, up):
    g = np.asarray(gate, dtype=np.float64)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * np.asarray(up, dtype=np.float64)


def norm(x, weight, eps):
    x = np.asarray(x, dtype=np.float64)
    x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x if weight is None else x * np.asarray(weight, dtype=np.float64)


def block_norm(r, y, post_weight, gate, scale, weight, eps):
    r = np.asarray(r, dtype=np.float64)
    if y is not None:
        y = np.asarray(y, dtype=np.float64)
        if post_weight is not None:
            y = norm(y, post_weight, eps)
        r = r + scale * (y if gate is None else y * np.asarray(gate, dtype=np.float64))
    return r, norm(r, weight, eps)
