"""fp4_linear and fp4_linear_rows against the oracle, and the operators together."""
import numpy as np
import pytest
import torch

from block_scaled_fp4_softmax_gb300 import fp4, moe
from fp4_helpers import BF, F32, FP, f64, held, random_matrix, rounded
from oracle import fp4 as O

pytestmark = pytest.mark.gpu
NV, MX = fp4.NVFP4, fp4.MXFP4


def slack(x, w, xr, wr, bias, want):
    """FP32 sums of K terms, each cut off or rounded once per addition (2^-23 of what
    has been summed up, at most the sum of magnitudes), the two row scales and the bias."""
    K = x.shape[1]
    size = np.abs(x) @ np.abs(w).T
    size = size * (1 if xr is None else xr[:, None]) * (1 if wr is None else wr)
    return size * (K + 3) * 2.0 ** -23 + (0 if bias is None else np.abs(bias) * 2.0 ** -23)


def check(T, N, K, format, dtype=BF, bias=False, seed=0, row_scale=True, out=None, dev_status=None):
    x, xc, xs, xr = random_matrix(T, K, format, seed + 1, 0.5, row_scale)
    w, wc, ws, wr = random_matrix(N, K, format, seed + 2, 0.5, row_scale)
    b = torch.randn(N, device="cuda") if bias else None
    y = fp4.fp4_linear(x, w, bias=b, dtype=dtype, out=out, dev_status=dev_status)
    torch.cuda.synchronize()
    xv, wv = O.values(xc, xs, None, format), O.values(wc, ws, None, format)
    want = xv @ wv.T
    if row_scale:
        want = want * xr[:, None].astype(np.float64) * wr.astype(np.float64)
    bv = None if b is None else f64(b)
    if bias:
        want = want + bv
    off = np.abs(f64(y) - want)
    most = rounded(want, y.dtype, slack(xv, wv, xr, wr, bv, want))
    ok = (off <= most) | (np.abs(want) > (65504 if y.dtype == FP else np.inf))
    assert ok.all(), (off.max(), np.argwhere(~ok)[:5], int((~ok).sum()))
    return x, w, b, y


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [
    (1, 128, 256), (1, 1, 32), (1, 5, 64), (2, 130, 96), (7, 257, 288), (16, 128, 512), (17, 300, 2560), (32, 64, 160),
    (33, 129, 1056), (64, 1000, 320), (65, 128, 256), (127, 77, 544), (128, 256, 1024), (129, 131, 4128), (300, 640, 2880),
])
def test_linear(T, N, K, format):
    check(T, N, K, format, F32, seed=T + N + K)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_types_and_bias(dtype, format):
    check(5, 200, 640, format, dtype, bias=True)
    check(150, 333, 640, format, dtype, bias=True, row_scale=False)


@pytest.mark.parametrize("format", [NV, MX])
def test_long_rows(format):
    check(3, 140, 32768, format, F32)
    check(200, 40, 16416, format, F32)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [(700, 1500, 512), (513, 2049, 96), (2000, 515, 288), (1025, 1030, 2080)])
def test_many_tiles(T, N, K, format):
    check(T, N, K, format, BF, bias=True)
    check(T, N, K, format, F32)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,N", [(3, 130), (40, 257), (260, 511), (600, 700)])
def test_output_is_a_strided_view(T, N, dtype):
    """Nothing between the rows is written, at any alignment."""
    for pad, off in ((3, 0), (13, 1), (16, 8)):
        big = torch.full((T + 1, N + pad), 7.0, device="cuda", dtype=dtype)
        check(T, N, 320, NV, out=big[:T, off:off + N])
        assert (big[T] == 7).all() and (big[:, :off] == 7).all() and (big[:, off + N:] == 7).all()


def test_every_scale_reaches_its_block():
    """One element of each row and one block scale at a time stand out."""
    for format, block in ((NV, 16), (MX, 32)):
        K, T, N = 512, 140, 300
        xc = np.full((T, K), 2, np.uint8)
        wc = np.full((N, K), 2, np.uint8)
        one = 0x38 if format == NV else 127
        xs, ws = np.full((T, K // block), one, np.uint8), np.full((N, K // block), one, np.uint8)
        up = 8 if format == NV else 1  # twice
        for t in range(T):
            xs[t, t % (K // block)] += up * (1 + t % 3)
        for n in range(N):
            ws[n, (n * 7) % (K // block)] += up * (1 + n % 2)
        x, w = (fp4.fp4_matrix(torch.from_numpy(O.pack(c)).cuda(), torch.from_numpy(s).cuda(), format=format)
                for c, s in ((xc, xs), (wc, ws)))
        want = O.values(xc, xs, None, format) @ O.values(wc, ws, None, format).T
        assert np.array_equal(f64(fp4.fp4_linear(x, w, dtype=F32)), want)
        assert np.array_equal(f64(fp4.fp4_linear(w, x, dtype=F32)), want.T)
        few = fp4.fp4_matrix(torch.from_numpy(O.pack(xc[:9])).cuda(), torch.from_numpy(xs[:9]).cuda(), format=format)
        assert np.array_equal(f64(fp4.fp4_linear(few, w, dtype=F32)), want[:9])


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T", [4, 150, 600])
def test_nan_stays_in_its_row_and_column(format, T):
    N, K = 260, 1056
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF)
    wx = torch.randn(N, K, generator=g, device="cuda")
    clean = fp4.fp4_linear(fp4.fp4_quantize(x, format), fp4.fp4_quantize(wx, format))
    x[T - 2, 40], wx[131, K - 1] = float("nan"), float("inf")
    y = fp4.fp4_linear(fp4.fp4_quantize(x, format), fp4.fp4_quantize(wx, format))
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    bad[T - 2], bad[:, 131] = True, True
    assert torch.isnan(y[bad]).all()
    assert torch.equal(y[~bad], clean[~bad])


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 90, 200, 700])
def test_rows_are_quantised(T, format):
    """fp4_linear_rows is fp4_linear of fp4_quantize, bit by bit, from any type and stride."""
    g = torch.Generator(device="cuda").manual_seed(T)
    w = fp4.fp4_quantize(torch.randn(500, 1120, generator=g, device="cuda"), format)
    bias = torch.randn(500, device="cuda")
    ws = fp4.fp4_linear_rows_workspace(w, 1000)
    for dtype in (BF, FP, F32):
        x = (torch.randn(T, 1200, generator=g, device="cuda") * 3).to(dtype)[:, :1120]
        want = fp4.fp4_linear(fp4.fp4_quantize(x, format), w, bias=bias)
        ws.random_()
        assert torch.equal(fp4.fp4_linear_rows(x, w, bias=bias, workspace=ws), want)
        assert torch.equal(fp4.fp4_linear_rows(x, w, bias=bias), want)


def test_no_rows_and_no_features():
    w = fp4.fp4_quantize(torch.randn(40, 64, device="cuda"))
    none = fp4.fp4_empty(0, 64)
    assert fp4.fp4_linear(none, w).shape == (0, 40)
    assert fp4.fp4_linear(w, none).shape == (40, 0)
    assert fp4.fp4_linear_rows(torch.empty(0, 64, device="cuda"), w).shape == (0, 40)


@pytest.mark.parametrize("T", [1, 20, 300, 1500])
def test_repeats_bit_for_bit(T):
    x, _, _, _ = random_matrix(T, 2560, NV, 1)
    w, _, _, _ = random_matrix(1100, 2560, NV, 2)
    want = fp4.fp4_linear(x, w, dtype=F32)
    for _ in range(5):
        assert torch.equal(fp4.fp4_linear(x, w, dtype=F32).view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("T,K", [(1, 1024), (40, 1024), (100, 1024), (100, 2080), (700, 1024)])
def test_streams_side_by_side_and_a_graph(T, K):
    """Calls that overlap share nothing but their inputs."""
    x = torch.randn(T, K, device="cuda").to(BF)
    w = fp4.fp4_quantize(torch.randn(3000, K, device="cuda"))
    want = fp4.fp4_linear_rows(x, w)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            outs.append(fp4.fp4_linear_rows(x, w, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = fp4.fp4_linear_rows(x, w)
        b = fp4.fp4_linear_rows(a[:, :K], w)
    want_b = fp4.fp4_linear_rows(want[:, :K], w)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want_b)


@pytest.mark.parametrize("T,K", [(1, 2560), (8, 256), (40, 4096), (200, 1024), (200, 4096), (900, 1024)])
def test_a_wait_that_runs_out(T, K):
    """The barrier of the sums expects an arrival that never comes: NaN, the flag, and
    the next call is right."""
    x, _, _, _ = random_matrix(T, K, NV, 1)
    w, _, _, _ = random_matrix(700, K, NV, 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = fp4.fp4_linear(x, w, dev_status=status)
    assert int(status) == 0
    moe.moe_test_set_wait_limit(200_000, 1)
    try:
        y = fp4.fp4_linear(x, w, dev_status=status)
        torch.cuda.synchronize()
    finally:
        moe.moe_test_set_wait_limit(0, 0)
    assert int(status) == fp4.DEV_TIMEOUT and torch.isnan(y).all()
    status.zero_()
    assert torch.equal(fp4.fp4_linear(x, w, dev_status=status), want) and int(status) == 0


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (35, 2560, 640), (300, 512, 288)])
def test_shared_expert_between_two_sums(T, H, I, format):
    """The operators as a layer runs them, each step against the oracle on what the step before handed over."""
    g = torch.Generator(device="cuda").manual_seed(T)
    r = torch.randn(T, H, generator=g, device="cuda")
    y = torch.randn(T, H, generator=g, device="cuda").to(BF)
    w_in = fp4.fp4_quantize(torch.randn(2 * I, H, generator=g, device="cuda") * H ** -0.5, format)
    w_out = fp4.fp4_quantize(torch.randn(H, I, generator=g, device="cuda") * I ** -0.5, format)
    ones = torch.ones(H, device="cuda")
    r1, _, h = fp4.fp4_block_norm(r, y, weight=ones, dtype=None, format=format)
    both = fp4.fp4_linear(h, w_in)
    _, a = fp4.fp4_swiglu(both[:, :I], both[:, I:], dtype=None, format=format)
    down = fp4.fp4_linear(a, w_out)
    r2, h2, _ = fp4.fp4_block_norm(r1, down, weight=ones, r_out=r1)
    assert r2 is r1
    want = held(h) @ held(w_in).T
    size = np.abs(held(h)) @ np.abs(held(w_in)).T
    assert (np.abs(f64(both) - want) <= rounded(want, BF, size * (H + 3) * 2.0 ** -23)).all()
    want = held(a) @ held(w_out).T
    size = np.abs(held(a)) @ np.abs(held(w_out)).T
    assert (np.abs(f64(down) - want) <= rounded(want, BF, size * (I + 3) * 2.0 ** -23)).all()
    # the whole in 64 bits without FP4: what the quantisation costs, no more than its steps.
    # An element in FP4 is off by at most a sixth of its block's largest (NVFP4), or a third.
    full, norm = O.block_norm(f64(r), f64(y), None, None, 1.0, None, 1e-6)
    assert np.abs(held(h) - norm).max() <= np.abs(norm).max() * (1 / 5.6 if format == NV else 1 / 2.9)
    want_r, want_h = O.block_norm(full, f64(down), None, None, 1.0, None, 1e-6)
    assert (np.abs(f64(r2) - want_r) <= rounded(want_r, F32, np.abs(full) * 2.0 ** -22 + np.abs(want_r) * 2.0 ** -22)).all()
    assert (np.abs(f64(h2) - want_h) <= rounded(want_h, BF, (np.abs(want_h) + 1) * 40 * 2.0 ** -24)).all()


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [(300, 192, 256), (257, 577, 1056), (2451, 5760, 320), (2451, 4096, 288), (260, 19000, 96),
                                   (5000, 1000, 64)])
def test_tiles_of_every_width(T, N, K, format):
    """Rounds of tiles that come out best at 256, 192 and 128 columns."""
    check(T, N, K, format, BF, bias=True)
    check(T, N, K, format, F32)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,K", [(1, 32), (1, 2560), (1, 32768), (2, 16384), (3, 96), (5, 1056), (7, 2880), (16, 2048), (16, 2080)])
def test_few_elements_are_quantised_by_the_product(T, K, format):
    """Below and above 32768 elements the same bits as from a matrix: rows of zeros, of
    tiny numbers, with an infinity."""
    g = torch.Generator(device="cuda").manual_seed(K)
    w = fp4.fp4_quantize(torch.randn(700, K, generator=g, device="cuda"), format)
    for dtype in (BF, FP, F32):
        x = torch.randn(T, K + 32, generator=g, device="cuda")
        x[0] *= 1e-3
        if T > 2:
            x[1], x[2, 40 % K] = 0, float("inf")
        if T > 4 and dtype != FP:
            x[3] *= 1e-37
        x = x.to(dtype)[:, :K]
        want = fp4.fp4_linear(fp4.fp4_quantize(x, format), w, dtype=F32)
        got = fp4.fp4_linear_rows(x, w, dtype=F32)
        assert torch.equal(got.view(torch.int32), want.view(torch.int32))


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [(1, 8192, 16384), (1, 9000, 32768), (2, 19300, 8192), (1, 6000, 32768), (16, 10000, 16384)])
def test_few_rows_that_shared_memory_does_not_hold(T, N, K, format):
    """Long rows over many tiles: a CTA's part of them is more than it may keep beside its ring."""
    g = torch.Generator(device="cuda").manual_seed(K)
    w = fp4.fp4_quantize(torch.randn(N, K, generator=g, device="cuda").to(BF), format)
    x = torch.randn(T, K, generator=g, device="cuda").to(BF)
    m = fp4.fp4_quantize(x, format)
    got = fp4.fp4_linear(m, w, dtype=F32)
    assert torch.equal(fp4.fp4_linear_rows(x, w, dtype=F32).view(torch.int32), got.view(torch.int32))
    # (the plain product in 64 bits of what is held)
    a, b = (fp4.fp4_dequantize(t, F32).double() for t in (m, w))
    off = (got.double() - a @ b.T).abs()
    assert (off <= (a.abs() @ b.abs().T) * (K + 3) * 2.0 ** -23).all()


@pytest.mark.parametrize("format", [NV, MX])
def test_many_tiles_of_few_rows(format):
    """More tiles than SMs: each CTA makes several, from one ring and two places of sums."""
    for T, N, K in ((1, 30000, 288), (16, 50257, 64), (17, 40000, 96), (64, 25000, 1056), (100, 20500, 320), (9, 20000, 8224)):
        check(T, N, K, format, BF, seed=T)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [(16, 1920, 4096), (16, 2048, 4096), (60, 2048, 8192), (512, 512, 2080), (16, 4608, 8192),
                                   (16, 4736, 8192), (4, 4736, 4096), (9, 9728, 2592), (5, 300, 1280), (16, 300, 1024)])
def test_numbers_of_clusters(T, N, K, format):
    """As many tiles as there are clusters of 8, 4 or 2 that run at once, and one more; columns too few to share."""
    check(T, N, K, format, F32)
    check(T, N, K, format, BF, bias=True)


# ---------------------------------------------------------------------------
# Sums that FP32 holds: nothing may be missing, and every rounding is known
# ---------------------------------------------------------------------------

def whole(rows, cols, format, seed, scales):
    """Any codes, a 6 in each block, block scales among `scales`: a matrix, its values in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    block = O.BLOCK[format]
    codes = torch.randint(0, 16, (rows, cols), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, ::block] = codes[:, ::block] & 8 | 7
    at = torch.randint(0, len(scales), (rows, cols // block), generator=g, device="cuda")
    bytes_ = torch.tensor([0x38 + 8 * s if format == NV else 127 + s for s in scales], dtype=torch.uint8, device="cuda")[at]
    m = fp4.fp4_matrix(codes[:, ::2] | codes[:, 1::2] << 4, bytes_, torch.ones(rows, device="cuda"), format)
    v = torch.tensor(O.E2M1, device="cuda")[codes.int()]
    return m, (v.unflatten(1, (-1, block)) * torch.tensor([2.0 ** s for s in scales], dtype=torch.float64, device="cuda")[at][..., None]).flatten(1)


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [
    (1, 300, 32768), (2, 300, 16384), (3, 140, 16416), (16, 1000, 32768), (16, 1000, 4128), (9, 20000, 4128), (16, 700, 32736),  # x held
    (5, 9000, 32768), (16, 20000, 16416),                                                                     # x too long for that
    (20, 500, 16416), (64, 500, 32768), (50, 20000, 2592), (100, 300, 32768), (300, 40, 32736), (500, 700, 16416),  # 32 to 128 rows a tile
    (200, 700, 1056), (512, 9728, 2592), (2451, 2880, 4128), (2000, 4096, 16416),                             # pairs of CTAs
])
def test_sums_that_fp32_holds_exactly(T, N, K, format):
    """Multiples of 1 / 4 below 2^22: no order of additions rounds, so a block that is lost, taken twice or
    scaled by its neighbour's scale shows in every element; results are the nearest of their type."""
    x, xv = whole(T, K, format, T + N + K, (0,))
    w, wv = whole(N, K, format, T + N + K + 1, (0, 1))
    bias = torch.randint(-4000, 4000, (N,), device="cuda").float() / 4
    assert float((xv.abs() @ wv.abs().T).max()) + 1000 < 2.0 ** 22
    want = xv @ wv.T
    assert torch.equal(fp4.fp4_linear(x, w, dtype=F32).double(), want)
    want += bias.double()
    assert torch.equal(fp4.fp4_linear(x, w, bias=bias, dtype=F32).double(), want)
    # values of one 6 a block at least are their own quantisation
    rows = xv.to(F32)
    assert torch.equal(fp4.fp4_linear_rows(rows, w, bias=bias, dtype=F32).double(), want)
    # with powers of two as factors of rows and columns: some FP16 results overflow, to an infinity of their sign
    x.row_scale[::2], w.row_scale[1::2] = 64, 8
    want = (want - bias.double()) * x.row_scale.double()[:, None] * w.row_scale.double() + bias.double()
    for dtype in (BF, FP):
        got = fp4.fp4_linear(x, w, bias=bias, dtype=dtype)
        assert torch.equal(got, want.to(dtype))
    assert torch.isinf(got).any() and torch.isfinite(got).any()


@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T,N,K", [(1, 300, 640), (5, 200, 640), (33, 200, 1056), (150, 333, 640), (700, 1500, 512)])
def test_fp16_results_within_their_range(T, N, K, format):
    """Any scales and factors, sized so that no result passes 40000."""
    x, xc, xs, xr = random_matrix(T, K, format, 3 * T, 0.5)
    w, wc, ws, wr = random_matrix(N, K, format, 3 * T + 1, 0.5)
    xv, wv = O.values(xc, xs, None, format), O.values(wc, ws, None, format)
    wide = np.abs(xv @ wv.T * wr).max(1)
    xr = (40000 / wide * np.random.default_rng(T).uniform(0.2, 1, T)).astype(np.float32)
    x.row_scale.copy_(torch.from_numpy(xr))
    b = torch.randn(N, device="cuda")
    y = fp4.fp4_linear(x, w, bias=b, dtype=FP)
    want = xv @ wv.T * xr[:, None].astype(np.float64) * wr.astype(np.float64) + f64(b)
    assert np.abs(want).max() < 45000
    assert (np.abs(f64(y) - want) <= rounded(want, FP, slack(xv, wv, xr, wr, f64(b), want))).all()


# ---------------------------------------------------------------------------
# What was written just before
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("format", [NV, MX])
@pytest.mark.parametrize("T", [1, 2, 3, 9, 16, 17, 40, 64, 90, 300])
def test_weights_written_by_the_call_before(T, format):
    """fp4_linear_rows reads w ahead of its quantisation of x: behind a call that has just written
    w, its scales alone, or x, never before it has."""
    N, K = 8192, 2560
    g = torch.Generator(device="cuda").manual_seed(T)
    sources = [torch.randn(N, K, generator=g, device="cuda") * 0.02 for _ in range(3)]
    inputs = [torch.randn(T, K, generator=g, device="cuda").to(BF) for _ in range(3)]
    made = [fp4.fp4_quantize(s, format) for s in sources]
    plain = [torch.from_numpy(O.untile(m.scales.cpu().numpy(), N, K // O.BLOCK[format]).copy()).cuda() for m in made]
    w, ws, x = fp4.fp4_empty(N, K, format), fp4.fp4_linear_rows_workspace(made[0], T), torch.empty(T, K, device="cuda", dtype=BF)
    want = [[fp4.fp4_linear(fp4.fp4_quantize(i, format), m) for m in made] for i in inputs]
    mixed = [fp4.Fp4Matrix(made[0].codes, m.scales, made[0].row_scale, N, K, format) for m in made]
    want_mixed = [fp4.fp4_linear(fp4.fp4_quantize(inputs[0], format), m) for m in mixed]
    fixed = fp4.Fp4Matrix(made[0].codes, torch.zeros_like(made[0].scales), made[0].row_scale, N, K, format)
    torch.cuda.synchronize()

    def steps(outs):
        for i in range(6):
            fp4.fp4_quantize(sources[i % 3], format, out=w)
            x.copy_(inputs[i % 2])
            outs.append((fp4.fp4_linear_rows(x, w, workspace=ws), want[i % 2][i % 3]))
            fp4.fp4_quantize(sources[(i + 1) % 3], format, out=w)
            outs.append((fp4.fp4_linear_rows(x, w, workspace=ws), want[i % 2][(i + 1) % 3]))
            outs.append((fp4.fp4_linear(fp4.fp4_quantize(x, format), w), want[i % 2][(i + 1) % 3]))
            fp4.fp4_tile_scales(plain[i % 3], K, format, tiled=fixed.scales)
            outs.append((fp4.fp4_linear_rows(inputs[0], fixed, workspace=ws), want_mixed[i % 3]))

    outs = []
    steps(outs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        steps(outs)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)
