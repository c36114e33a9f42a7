"""Matrices on the device as the oracle sees them, and what may separate the two."""
import numpy as np
import torch

from block_scaled_fp4_softmax_gb300 import fp4
from oracle import fp4 as O

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
STEP = {BF: 2.0 ** -8, FP: 2.0 ** -11, F32: 2.0 ** -24}      # half a step, relative
LEAST = {BF: 2.0 ** -134, FP: 2.0 ** -25, F32: 2.0 ** -150}  # half a step of the subnormals


def f64(t):
    return t.detach().double().cpu().numpy()


def parts(m):
    """codes [rows, cols], scales [rows, blocks] bytes, row scales or None of a matrix on the device."""
    codes = O.unpack(m.codes.cpu().numpy())
    scales = O.untile(m.scales.cpu().numpy(), m.rows, m.cols // O.BLOCK[m.format])
    return codes, scales, None if m.row_scale is None else f64(m.row_scale)


def held(m):
    """The values of a matrix's elements in 64 bits."""
    return O.values(*parts(m), m.format)


def random_matrix(rows, cols, format, seed, spread=1.0, row_scale=True):
    """Any codes, scales over many magnitudes (subnormal E4M3 among them)."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    if format == fp4.NVFP4:
        scales = rng.integers(0, 0x7F, (rows, cols // 16)).astype(np.uint8)
    else:
        scales = rng.integers(127 - int(8 * spread), 128 + int(8 * spread), (rows, cols // 32)).astype(np.uint8)
    factor = rng.lognormal(size=rows).astype(np.float32) if row_scale else None
    m = fp4.fp4_matrix(torch.from_numpy(O.pack(codes)).cuda(), torch.from_numpy(scales).cuda(),
                       None if factor is None else torch.from_numpy(factor).cuda(), format)
    return m, codes, scales, factor


def rounded(want, dtype, slack):
    """How far a result may be from `want`: `slack` before its rounding, and the rounding."""
    return slack + (np.abs(want) + slack) * STEP[dtype] + LEAST[dtype]


def check_fp4(m, x, rel):
    """That m is what fp4_quantize makes of values within `rel` of x (relative).

    With s a block's scale and 2^E its row's, each may be what either end of that
    range gives, and a value is within half of its gap of x, and `rel`."""
    codes, scales, row = parts(m)
    x = np.asarray(x, dtype=np.float64)
    g = O.BLOCK[m.format]
    if m.format == fp4.NVFP4:
        top = np.abs(x).max(1)
        e = np.log2(row)
        assert (e == np.round(e)).all() and (e >= -126).all()
        assert (2688 * row >= top * (1 - rel)).all()
        assert ((1344 * row < top * (1 + rel)) | (e == -126)).all()
    else:
        row = np.ones(m.rows)
    big = np.abs(x).reshape(m.rows, -1, g).max(2) / row[:, None]
    if m.format == fp4.NVFP4:
        lo, hi = O.nearest(big * (1 - rel) / 6, O.E4M3), O.nearest(big * (1 + rel) / 6, O.E4M3)
        assert ((scales == lo) | (scales == hi)).all()
    else:
        s = O.scale_value(scales, m.format)
        assert (6 * s >= big * (1 - rel)).all() and ((3 * s < big * (1 + rel)) | (scales == 0)).all()
    s = np.repeat(O.scale_value(scales, m.format), g, 1) * row[:, None]
    v = np.abs(O.E2M1[codes])
    # (rounded up from below 6: the next step down is 2, and nothing lies above)
    gap = np.where(v < 2, 0.25, np.where(v < 4, 0.5, 1.0))
    below = np.where(v == 2, 0.25, np.where(v == 4, 0.5, gap))
    size = np.abs(x)
    assert (size <= (v + gap) * s * (1 + rel) + 1e-300).all()
    assert (size >= (v - below) * s * (1 - rel)).all()
    sure = size > 0.25 * s * (1 + rel)
    assert (np.signbit(x) == (codes >= 8))[sure].all()
