"""fp4_quantize, fp4_dequantize, fp4_tile_scales, fp4_swiglu and fp4_block_norm against the oracle."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_softmax_gb300 import fp4, moe
from fp4_helpers import BF, F32, FP, check_fp4, f64, held, parts, random_matrix, rounded
from oracle import fp4 as O

pytestmark = pytest.mark.gpu
NV, MX = fp4.NVFP4, fp4.MXFP4
COLS = [32, 64, 96, 256, 288, 1056, 2048, 2560, 4128, 8192, 8224, 16384]


def rows_of(rows, cols, dtype, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= (torch.randn(rows, 1, generator=g, device="cuda") * 2).exp()
    x[:, ::17] *= 20
    x[:, 5 * 32:7 * 32] *= 1e-3
    return x.to(dtype)[:, :cols]


def same(m, x):
    """m is, bit by bit, the oracle's quantisation of x."""
    codes, scales, row = O.quantize(x.float().cpu().numpy(), m.format)
    got, got_scales, got_row = parts(m)
    assert np.array_equal(got_scales, scales)
    assert np.array_equal(got, codes)
    if m.format == NV:
        assert np.array_equal(got_row, row, equal_nan=True)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("cols", COLS)
def test_quantize(cols, dtype, format):
    """Quotients in FP32 are the definition, so nothing may differ."""
    for rows, pad in ((1, 0), (37, 32)):
        x = rows_of(rows, cols, dtype, cols + rows, pad)
        same(fp4.fp4_quantize(x, format), x)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("cols", [16416, 24576, 32736, 32768])
def test_quantize_the_longest_rows(cols, dtype, format):
    for rows, pad in ((1, 0), (5, 32)):
        x = rows_of(rows, cols, dtype, cols + rows, pad)
        x[rows - 1, cols - 5] *= 30
        same(fp4.fp4_quantize(x, format), x)


@pytest.mark.parametrize("format", [NV, MX])
def test_quantize_many_rows(format):
    x = rows_of(700, 160, BF, 1)
    same(fp4.fp4_quantize(x, format), x)


@pytest.mark.parametrize("format", [NV, MX])
def test_quantize_ties_and_extremes(format):
    """Every tie of e2m1, ties of E4M3, rows of zeros, of one element, of the
    largest and the smallest numbers."""
    ties = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5, -6.0])
    rows = [ties.repeat(8) * 2.0 ** e for e in (-120, -3, 0, 7, 100)]
    rows += [torch.zeros(128), -torch.zeros(128)]
    for at in (0, 127):
        for v in (1.0, 2688.0, 2689.0, 3e38, 1e-38, 2.0 ** -133, -1.5):
            r = torch.zeros(128)
            r[at] = v
            rows.append(r)
    # block maxima half way between two E4M3 scales, the row's largest 2688
    steps = torch.zeros(8, 16)
    steps[:, 3] = 6 * torch.tensor([448, 17, 19, 34, 2.0 ** -9 * 0.5, 2.0 ** -9 * 1.5, 2.0 ** -9 * 2.5, 15.5])
    steps[:, 7] = steps[:, 3] * 0.37
    rows.append(steps.flatten())
    x = torch.stack(rows).cuda()
    same(fp4.fp4_quantize(x, format), x)
    same(fp4.fp4_quantize(x.to(BF), format), x.to(BF))


@pytest.mark.parametrize("power", [0, 40, -100, -119, -126])
def test_quantize_every_scale_and_tie(power):
    """Blocks of each E4M3 scale, with every tie of e2m1 and its neighbours in FP32: what the
    products that stand for quotients have to get right.  `power`: of the row."""
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    around = [np.nextafter(ties, np.float32(0)), ties, np.nextafter(ties, np.float32(9))]
    for near in around:
        x = np.zeros((1, 127, 16), dtype=np.float32)
        for code in range(1, 127):
            s = np.float32(O.E4M3[code])
            x[0, code, 0], x[0, code, 1:8], x[0, code, 8:15] = 6 * s, near * s, -near * s
        x[0, 0, 0] = 2688
        x = np.ldexp(np.concatenate([x.reshape(1, -1), np.zeros((1, 16), np.float32)], 1), power).astype(np.float32)
        rows = torch.from_numpy(x).cuda()
        same(fp4.fp4_quantize(rows, NV), rows)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("format", [NV, MX])
def test_quantize_not_finite(dtype, format):
    x = rows_of(6, 320, dtype, 3)
    x[1, 70], x[2, 319], x[3, 0], x[4, 100] = float("nan"), float("inf"), -float("inf"), -float("nan")
    m = fp4.fp4_quantize(x, format)
    same(m, x)
    v = fp4.fp4_dequantize(m)
    if format == NV:
        assert torch.isnan(v[1:5]).all() and torch.isfinite(v[[0, 5]]).all()
    else:
        for r, c in ((1, 70), (2, 319), (3, 0), (4, 100)):
            b = c // 32 * 32
            assert torch.isnan(v[r, b:b + 32]).all()
            assert torch.isnan(v[r]).sum() == 32


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (33, 160), (129, 288), (300, 2560), (2, 32768)])
def test_tiles_and_values(rows, cols, format):
    m, codes, scales, factor = random_matrix(rows, cols, format, rows + cols)
    tiled = m.scales.cpu().numpy()
    want = O.tile(scales)
    assert tiled.shape == want.shape
    assert np.array_equal(O.untile(tiled, rows, scales.shape[1]), scales)
    # blocks past a row's end are 0
    kt = -(-scales.shape[1] // 4)
    full = O.untile(tiled, rows, kt * 4)
    assert not full[:, scales.shape[1]:].any()
    v = O.values(codes, scales, factor, format)
    for dtype in (BF, FP, F32):
        got = f64(fp4.fp4_dequantize(m, dtype))
        fits = np.abs(v) < 65000
        # code * scale is exact, the row's factor one rounding in FP32
        assert (np.abs(got - v) <= rounded(v, dtype, np.abs(v) * 2.0 ** -24))[fits].all()


@pytest.mark.parametrize("format", [NV, MX])
def test_values_of_quantised_rows_are_exact_in_bf16(format):
    x = rows_of(50, 512, BF, 9)
    m = fp4.fp4_quantize(x, format)
    assert np.array_equal(f64(fp4.fp4_dequantize(m)), held(m))
    out = torch.full((50, 600), 7.0, device="cuda", dtype=BF)
    fp4.fp4_dequantize(m, out=out[:, :512])
    assert np.array_equal(f64(out[:, :512]), held(m)) and (out[:, 512:] == 7).all()


@pytest.mark.parametrize("format", [NV, MX])
def test_values_of_extreme_scales_and_factors(format):
    """Every code under the smallest and the largest scales, in rows whose factors bring them back among
    the numbers or carry them out of them: a zero stays zero, and nothing between overflows."""
    block = O.BLOCK[format]
    bytes_ = [0, 1, 8, 56, 0x7E, 17, 119, 2] if format == NV else [0, 1, 2, 127, 252, 253, 254, 64]
    factors = [1.0, 2.0, 4.0, 0.75, 1e38, 3e38, -2.0 ** 100, 2.0 ** -100, 1.3 * 2.0 ** -126, 2.0 ** -140, 3 * 2.0 ** -149]
    factors = np.array(factors, dtype=np.float32)
    codes = np.tile(np.arange(block, dtype=np.uint8) % 16, (len(factors), len(bytes_)))
    scales = np.tile(np.array(bytes_, dtype=np.uint8), (len(factors), 1))
    m = fp4.fp4_matrix(torch.from_numpy(O.pack(codes)).cuda(), torch.from_numpy(scales).cuda(), torch.from_numpy(factors).cuda(), format)
    want = O.values(codes, scales, factors, format)
    for dtype in (F32, BF, FP):
        got = f64(fp4.fp4_dequantize(m, dtype))
        # the least that rounds to infinity: half a step past the largest number
        top = {F32: 2.0 ** 128 * (1 - 2.0 ** -25), BF: 2.0 ** 128 * (1 - 2.0 ** -9), FP: 65520.0}[dtype]
        # code * scale is exact, the row's factor one rounding in FP32 (a subnormal result: half of 2^-149)
        slack = np.abs(want) * 2.0 ** -24 + 2.0 ** -150
        near = 0 if dtype == F32 else slack  # (in FP32 there is that rounding alone, and `want` is exact)
        over, under = np.abs(want) - near >= top, np.abs(want) + near < top
        assert (over | under).all()
        assert (got[over] == np.copysign(np.inf, want[over])).all()
        assert (np.abs(got - want)[under] <= rounded(want, dtype, slack)[under]).all()
        assert (got[want == 0] == 0).all()


def test_nothing_is_written_behind_the_rows():
    x = rows_of(37, 288, BF, 11)
    big = [torch.full((200, 144), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((fp4.fp4_scale_bytes(200, 288, NV),), 0xA5, dtype=torch.uint8, device="cuda"),
           torch.full((200,), -3.0, device="cuda")]
    size = fp4.fp4_scale_bytes(37, 288, NV)
    m = fp4.Fp4Matrix(big[0][:37], big[1][:size], big[2][:37], 37, 288, NV)
    same(fp4.fp4_quantize(x, NV, out=m), x)
    assert (big[0][37:] == 0xA5).all() and (big[2][37:] == -3).all()
    assert (big[1][size:] == 0xA5).all()


# ---------------------------------------------------------------------------
# SwiGLU
# ---------------------------------------------------------------------------

# exp(-g) by __expf: (2 + |1.173 g|) ulp, which the sum 1 + exp(-g) takes over at most
# whole; then a rounding of the sum, a quotient within 2 ulp and a product.  An ulp
# is at most 2^-23 of the value.
def swiglu_slack(g, want):
    return np.abs(want) * (2 + 1.173 * np.abs(g) + 0.5 + 2 + 0.5) * 2.0 ** -23 + 2.0 ** -126


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("rows,cols", [(1, 64), (5, 2880), (260, 96), (2, 16416)])
def test_swiglu(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    both = (torch.randn(rows, 2 * cols, generator=g, device="cuda") * 4).to(dtype)
    gate, up = both[:, :cols], both[:, cols:]
    want = O.swiglu(f64(gate), f64(up))
    slack = swiglu_slack(f64(gate), want)
    for out_type in (BF, FP):
        a, none = fp4.fp4_swiglu(gate, up, dtype=out_type)
        assert none is None and a.dtype == out_type
        assert (np.abs(f64(a) - want) <= rounded(want, out_type, slack)).all()
    for format in (NV, MX):
        a, m = fp4.fp4_swiglu(gate, up, dtype=BF, format=format)
        assert (np.abs(f64(a) - want) <= rounded(want, BF, slack)).all()
        check_fp4(m, want, 40 * 2.0 ** -23)  # |g| < 30: the largest of the above
        none, alone = fp4.fp4_swiglu(gate, up, dtype=None, format=format)
        assert none is None and torch.equal(alone.codes, m.codes)


def test_swiglu_extremes():
    gate = torch.tensor([[0.0, -0.0, 1e4, -1e4, 90.0, -90.0, 3e38, -3e38] * 4], device="cuda")
    up = torch.full_like(gate, 0.5)
    a, _ = fp4.fp4_swiglu(gate, up)
    assert (a[0, :8].float() == torch.tensor([0.0, -0.0, 5e3, 0, 45.0, 0, 3e38 / 2, 0], device="cuda").to(BF).float()).all()
    gate[0, 3], gate[0, 9] = float("nan"), float("inf")
    a, m = fp4.fp4_swiglu(gate, up, format=NV)
    assert torch.isnan(a[0, 3]) and torch.isinf(a[0, 9]) and torch.isnan(m.row_scale).all()


@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_swiglu_of_gates_whose_exponential_is_near_the_largest_number(dtype):
    """1 + exp(-g) above 2^126: its reciprocal is below the normal numbers, the product with the gate is not."""
    gate = -{BF: torch.arange(73, 89, 0.5), FP: torch.arange(80.75, 88.75, 0.0625), F32: torch.linspace(80, 88.7, 2048)}[dtype]
    gate = gate.to(dtype)[None]
    assert gate.min() >= -88.7 and (gate < -87.5).sum() >= 2
    for size in (1.0, -3.0, 300.0) + ((1e30,) if dtype != FP else ()):
        up = torch.full_like(gate, size)
        want = O.swiglu(f64(gate), f64(up))
        # exp(-g) within 2 + |1.173 g| ulp (of 2^-23 at most), which 1 + exp(-g) takes over; its
        # rounding and two products, half an ulp each; the reciprocal 1 ulp, and where it is
        # subnormal (2^-128 at least, steps of 2^-149) half a step: 2^-22, 2 ulp
        rel = (2 + 1.173 * np.abs(f64(gate)) + 1.5 + 1 + 2) * 2.0 ** -23
        a, m = fp4.fp4_swiglu(gate.cuda(), up.cuda(), format=NV)
        assert (np.abs(f64(a) - want) <= rounded(want, BF, np.abs(want) * rel)).all()
        _, m = fp4.fp4_swiglu(gate.cuda(), up.cuda(), dtype=None, format=MX)
        # (a row's scale of NVFP4 is 2^-126 at least: the smaller products above are below its codes)
        check_fp4(m, want, rel.max())


def test_swiglu_of_subnormal_gates():
    """g / 2 of the smallest numbers, times a large factor: g itself is not rounded on the way."""
    steps = torch.cat([torch.arange(64), -torch.arange(64), 3 * 2 ** torch.arange(22), -(2 ** torch.arange(1, 11)) - 1])
    gate = (steps.double() * 2.0 ** -149).float()[None]
    up = torch.full_like(gate, 2.0 ** 127)
    a, _ = fp4.fp4_swiglu(gate.cuda(), up.cuda())
    # exp(-g) = 1: the quotient is g / 2, off by half a step of 2^-149 and no more
    want = f64(gate) / 2 * 2.0 ** 127
    assert (np.abs(f64(a) - want) <= rounded(want, BF, 2.0 ** -150 * 2.0 ** 127 + np.abs(want) * 2.0 ** -22)).all()


# ---------------------------------------------------------------------------
# Norms around a residual sum
# ---------------------------------------------------------------------------

def run_norm(rows, cols, dtype, block, post, gate, weight=True, scale=0.7, eps=1e-5, seed=0, in_place=False):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + cols)

    def normal(*shape, type=F32, mean=0.0, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std + mean).to(type)

    r = normal(rows, cols + 32, type=dtype, std=3.0)[:, :cols]
    y = None if block is None else normal(rows, cols, type=block, std=2.0)
    shape = {None: None, "channel": (cols,), "token": (rows, 1), "full": (rows, cols)}[gate]
    gt = None if shape is None else normal(*shape, type=block)
    pw = normal(cols, mean=1.0, std=0.2) if post else None
    w = normal(cols, mean=1.0, std=0.2) if weight else None
    want_r, want_h = O.block_norm(f64(r), None if y is None else f64(y), None if pw is None else f64(pw),
                                  None if gt is None else f64(gt), float(np.float32(scale)), None if w is None else f64(w),
                                  float(np.float32(eps)))
    # FP32: a sum of squares of c terms in chains of 32 at most, then two trees of 5
    # steps: 42 roundings, half of that after the root; root, quotient and two products: 4;
    # so a norm is within 26 roundings.  r': the same of its y, two products and a sum.
    rel = 26 * 2.0 ** -24
    part = np.abs(want_r - f64(r))
    slack_r = part * (rel + 3 * 2.0 ** -24) + (np.abs(f64(r)) + part) * 2.0 ** -24
    root = np.sqrt((want_r ** 2).mean(1, keepdims=True) + eps)
    slack_h = (slack_r / root + np.abs(want_h) * np.sqrt((slack_r ** 2).mean(1, keepdims=True)) / root) \
        * (1 if w is None else np.abs(f64(w))) + np.abs(want_h) * rel
    slack_h = slack_h * 2  # second order, and |w| beside h
    args = dict(post_weight=pw, gate=gt, scale=scale, weight=w, eps=eps)
    out_r, h, none = fp4.fp4_block_norm(r, y, dtype=BF, **args)
    assert none is None and (out_r is r if y is None else out_r.dtype == dtype)
    if y is not None:
        assert (np.abs(f64(out_r) - want_r) <= rounded(want_r, dtype, slack_r)).all()
    assert (np.abs(f64(h) - want_h) <= rounded(want_h, BF, slack_h)).all()
    for format in (NV, MX):
        again, h16, m = fp4.fp4_block_norm(r, y, dtype=FP, format=format, **args)
        assert torch.equal(again, out_r)
        assert (np.abs(f64(h16) - want_h) <= rounded(want_h, FP, slack_h)).all()
        check_norm_fp4(m, want_h, slack_h)
        _, none, alone = fp4.fp4_block_norm(r, y, dtype=None, format=format, **args)
        assert none is None and torch.equal(alone.codes, m.codes)
    if y is not None:
        both = r.clone() if not in_place else r
        want = out_r.clone()
        same_r, _, _ = fp4.fp4_block_norm(both, y, r_out=both, **args)
        assert same_r is both and torch.equal(both, want)


def check_norm_fp4(m, want, slack):
    """The matrix against values that are `slack` off: each scale is one that its
    block's range gives, each value within half a gap and the slack."""
    codes, scales, row = parts(m)
    g = O.BLOCK[m.format]
    row = np.ones(m.rows) if row is None else row
    s = O.scale_value(scales, m.format)
    size = np.abs(want).reshape(m.rows, -1, g)
    big, off = size.max(2) / row[:, None], slack.reshape(m.rows, -1, g).max(2) / row[:, None]
    if m.format == NV:
        assert (2688 * row >= (np.abs(want) - slack).max(1)).all() and (1344 * row < (np.abs(want) + slack).max(1)).all()
        lo, hi = O.nearest(np.maximum(big - off, 0) / 6, O.E4M3), O.nearest((big + off) / 6, O.E4M3)
        assert ((scales >= lo) & (scales <= hi)).all()
    else:
        assert (6 * s >= big - off).all() and (3 * s < big + off).all()
    gap = np.repeat(s, g, 1) * row[:, None]
    v = np.abs(O.E2M1[codes])
    half = np.where(v < 2, 0.25, np.where(v < 4, 0.5, 1.0)) * gap
    below = np.where(v == 2, 0.25, np.where(v == 4, 0.5, half / np.where(gap == 0, 1, gap))) * gap
    x = np.abs(want)
    assert (x <= v * gap + half + slack).all() and (x >= v * gap - below - slack).all()


@pytest.mark.parametrize("dtype,block", [(BF, BF), (FP, FP), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2560), (9, 288), (130, 1056), (3, 4128), (2, 16416)])
def test_block_norm(rows, cols, dtype, block):
    run_norm(rows, cols, dtype, block, True, "full")


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
def test_block_norm_forms(gate, post):
    run_norm(21, 640, BF, BF, post, gate, in_place=True)
    run_norm(1, 64, F32, FP, post, gate, weight=False, scale=-2.0)


def test_block_norm_without_a_block():
    run_norm(5, 320, BF, None, False, None)
    run_norm(5, 8192, F32, None, False, None, weight=False)


def test_block_norm_of_zeros_and_of_what_is_not_finite():
    r = torch.zeros(4, 64, device="cuda")
    y = torch.zeros(4, 64, device="cuda")
    r[1, 3], y[2, 5], y[3, 7] = float("inf"), float("nan"), -float("inf")
    ones = torch.ones(64, device="cuda")
    out, h, m = fp4.fp4_block_norm(r, y, post_weight=ones, eps=1e-6, format=NV)
    assert (h[0] == 0).all() and (out[0] == 0).all() and (held(m)[0] == 0).all()
    assert torch.isnan(h[1, 3]) and torch.isnan(h[2:]).any(1).all()
    assert torch.isnan(m.row_scale[1:]).all() and torch.isfinite(m.row_scale[0])
    # eps 0: a row of zeros is 0 / 0
    _, h, _ = fp4.fp4_block_norm(r, eps=0.0)
    assert torch.isnan(h[0]).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    m = fp4.fp4_quantize(x)
    assert m.shape == (0, 64) and fp4.fp4_dequantize(m).shape == (0, 64)
    assert fp4.fp4_swiglu(x, x)[0].shape == (0, 64)
    assert fp4.fp4_block_norm(x, x)[1].shape == (0, 64)


def test_streams_and_a_graph():
    x, y = rows_of(64, 2560, BF, 5), rows_of(64, 2560, BF, 6)
    ones = torch.ones(2560, device="cuda")

    def step(stream=None):
        r, h, m = fp4.fp4_block_norm(x, y, post_weight=ones, weight=ones, format=NV, stream=stream)
        a, am = fp4.fp4_swiglu(h[:, :1280], h[:, 1280:], format=MX, stream=stream)
        # (as values: the scales of rows behind the last are nobody's)
        return [r, h, m.codes, fp4.fp4_dequantize(m, stream=stream), a, am.codes, fp4.fp4_dequantize(am, stream=stream)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        played = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, played):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("rows,cols", [(1, 64), (1, 8224), (5, 640), (2100, 1056), (3, 16416)])
def test_outputs_in_the_place_of_inputs(rows, cols):
    """The same bits, whichever input of the same element size an output of SwiGLU or the norm replaces."""
    def fresh():
        return [rows_of(rows, cols, BF, s, 32) for s in (1, 2, 3)]

    gate, up, _ = fresh()
    want, m = fp4.fp4_swiglu(gate, up, format=NV)
    want_half, _ = fp4.fp4_swiglu(gate, up, dtype=FP)
    for at in (0, 1):
        ops = fresh()
        got, again = fp4.fp4_swiglu(ops[0], ops[1], format=NV, out=ops[at])
        assert got is ops[at] and torch.equal(got, want) and torch.equal(again.codes, m.codes)
        ops = fresh()
        got, _ = fp4.fp4_swiglu(ops[0], ops[1], out=ops[at].view(FP))
        assert torch.equal(got, want_half)
    ones = torch.ones(cols, device="cuda")
    args = dict(post_weight=ones, weight=ones, scale=0.5)
    r, y, g = fresh()
    want_r, want_h, m = fp4.fp4_block_norm(r, y, gate=g, format=MX, **args)
    twice_r, twice_h, _ = fp4.fp4_block_norm(r, r, gate=g, **args)
    for at in range(3):
        for to in range(3):
            ops = fresh()
            if at != to:
                got_r, got_h, again = fp4.fp4_block_norm(ops[0], ops[1], gate=ops[2], format=MX, r_out=ops[at], out=ops[to], **args)
            else:
                got_r, got_h, again = fp4.fp4_block_norm(ops[0], ops[1], gate=ops[2], format=MX, r_out=ops[at], **args)
            assert torch.equal(got_r, want_r) and torch.equal(got_h, want_h) and torch.equal(again.codes, m.codes)
    ops = fresh()
    got_r, got_h, _ = fp4.fp4_block_norm(ops[0], ops[0], gate=ops[2], r_out=ops[0], **args)
    assert torch.equal(got_r, twice_r) and torch.equal(got_h, twice_h)


@pytest.mark.parametrize("rows", [1, 2, 70, 300])
def test_operands_side_by_side_in_one_buffer(rows):
    """gate | up | out, r | y | r_out | h, x | y of a product: rows between one another's."""
    cols = 320
    buf = rows_of(rows, 4 * cols, BF, 4)
    parts = [buf[:, i * cols:(i + 1) * cols] for i in range(4)]
    apart = [p.clone() for p in parts]
    want, _ = fp4.fp4_swiglu(apart[0], apart[1])
    want_r, want_h, _ = fp4.fp4_block_norm(apart[0], apart[1])
    w = fp4.fp4_quantize(torch.randn(cols, cols, device="cuda"))
    want_y = fp4.fp4_linear_rows(apart[0], w)
    got, _ = fp4.fp4_swiglu(parts[0], parts[1], out=parts[2])
    assert torch.equal(got, want)
    got_r, got_h, _ = fp4.fp4_block_norm(parts[0], parts[1], r_out=parts[2], out=parts[3])
    assert torch.equal(got_r, want_r) and torch.equal(got_h, want_h)
    assert torch.equal(fp4.fp4_linear_rows(parts[0], w, out=parts[3]), want_y)
    assert torch.equal(parts[0], apart[0]) and torch.equal(parts[1], apart[1])
    for call in (lambda: fp4.fp4_swiglu(parts[0], parts[1], out=buf[:, 32:32 + cols]),
                 lambda: fp4.fp4_linear_rows(parts[0], w, out=parts[0]),
                 lambda: fp4.fp4_block_norm(parts[0], parts[1], r_out=parts[2], out=buf[:, 3 * cols - 32:4 * cols - 32])):
        with pytest.raises(fp4.MoeError, match="failed: status 1"):
            call()


def test_record_parts_are_matrices():
    """gate | up codes and scales of an expert record are the parts of one matrix."""
    H, I = 256, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    gate, up, down = (torch.randn(*s, generator=g, device="cuda") for s in ((I, H), (I, H), (H, I)))
    for format, block in ((NV, 16), (MX, 32)):
        s = moe.shape(H, I, format)
        record = moe.fp4_pack_expert(gate, up, down, s)
        o = moe.moe_expert_record_offsets(s)
        m = fp4.fp4_matrix(record[o["gate"]:o["down"]].view(2 * I, H // 2), record[o["gate_s"]:o["down_s"]].view(2 * I, H // block), format=format)
        off = (fp4.fp4_dequantize(m, F32) - torch.cat((gate, up))).abs()
        top = torch.cat((gate, up)).unflatten(1, (-1, block)).abs().amax(-1).repeat_interleave(block, 1)
        # half of the widest gap, 2 / 6 of a block's largest that the scale rounds by up
        # to a 16th (NVFP4) or a factor 2 (MXFP4)
        assert (off <= top * (1.0 / 6) * (1 + 1.0 / 16 if format == NV else 2) * 1.0001 + 6 * 2.0 ** -10).all()
