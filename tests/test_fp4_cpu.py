"""What include/fp4.h promises and the host can show: names, sizes, the oracle's readings, refusals."""
import copy
import ctypes
import os
import pickle
import re
import subprocess
import types

import numpy as np
import pytest
import torch

from block_scaled_fp4_softmax_gb300 import build, fp4
from oracle import fp4 as O
from oracle import oracle as M

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NV, MX = fp4.NVFP4, fp4.MXFP4
OK, INVALID, ALIGNMENT, UNSUPPORTED, SMALL = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fp4.load()


# ---------------------------------------------------------------------------
# Names and sizes
# ---------------------------------------------------------------------------

def declared():
    text = open(os.path.join(ROOT, "include", "fp4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return {n for n in re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)}


def test_header_binding_and_library_agree(lib):
    assert declared() == set(fp4.EXPORTS) == set(fp4._SIGS)
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert declared() <= exported
    for name in fp4.EXPORTS:
        assert callable(getattr(fp4, name))


def test_argument_counts_of_header_and_binding():
    text = open(os.path.join(ROOT, "include", "fp4.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for name, args in re.findall(r"\b(fp4_[a-z_]+)\s*\(([^)]*)\)", text):
        assert len(args.split(",")) == len(fp4._SIGS[name][1]), name


def test_scale_bytes(lib):
    for rows, cols, format, want in ((1, 32, NV, 512), (1, 64, NV, 512), (1, 96, NV, 1024), (128, 96, NV, 1024),
                                     (129, 96, NV, 2048), (1, 128, MX, 512), (1, 160, MX, 1024), (0, 64, NV, 0),
                                     (1 << 24, 32768, NV, (1 << 17) * 512 * 512)):
        assert fp4.fp4_scale_bytes(rows, cols, format) == fp4._scale_bytes(rows, cols, format) == want
        if rows and rows < 1000:
            assert want == O.tile(np.zeros((rows, cols // O.BLOCK[format]), np.uint8)).size
    for rows, cols, format in ((-1, 64, NV), (1, 48, NV), (1, 0, NV), (1, 32800, NV), ((1 << 24) + 1, 64, NV), (1, 64, 2),
                               (1, 1 << 40, NV), (1 << 40, 64, NV)):
        assert fp4.fp4_scale_bytes(rows, cols, format) == 0


# ---------------------------------------------------------------------------
# The oracle's readings
# ---------------------------------------------------------------------------

def test_tiles_are_where_the_header_says():
    rows, blocks = 300, 7
    scales = (np.arange(rows * blocks) % 251).astype(np.uint8).reshape(rows, blocks)
    tiled, kt = O.tile(scales, fill=7), 2
    for r in range(rows):
        for b in range(blocks):
            assert tiled[((r // 128) * kt + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] == scales[r, b]
        assert tiled[((r // 128) * kt + 1) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + 3] == 0
    assert np.array_equal(O.untile(tiled, rows, blocks), scales)


def test_quantisation_is_the_nearest():
    """Codes and scales by the definition, from all of e2m1 and E4M3."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((6, 64)) * np.exp(rng.standard_normal((6, 1)) * 6)).astype(np.float32)
    for format in (NV, MX):
        codes, scales, row = O.quantize(x, format)
        g = O.BLOCK[format]
        for r in range(6):
            top = np.abs(x[r]).max()
            e = 0 if row is None else int(np.log2(row[r]))
            if row is not None:
                assert 2688 * 2.0 ** e >= top > 2688 * 2.0 ** (e - 1)
            for b in range(64 // g):
                y = x[r, b * g:(b + 1) * g].astype(np.float64) * 2.0 ** -e
                s = O.scale_value(scales[r, b], format)
                if format == NV:
                    want = np.abs(y).max() / 6
                    assert abs(want - s) == np.abs(O.E4M3 - want).min()
                else:
                    assert 6 * s >= np.abs(y).max() > 3 * s
                for v, c in zip(y, codes[r, b * g:(b + 1) * g]):
                    assert abs(O.E2M1[c] * s - v) <= np.abs(O.E2M1 * s - v).min() * (1 + 1e-7)


def test_oracle_agrees_with_the_record_quantiser():
    """Rows whose largest element makes the row's power 1 are quantised as an expert record's."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 64)).astype(np.float32)
    x[:, 0] = 2688
    codes, scales, row = O.quantize(x, NV)
    assert (row == 1).all()
    packed, want = M.quantize_matrix(x, M.FMT_NVFP4)[:2]
    assert np.array_equal(O.pack(codes), packed.reshape(4, -1)) and np.array_equal(scales, want.reshape(4, -1))


def test_packing():
    codes = np.arange(64, dtype=np.uint8).reshape(2, 32) % 16
    assert O.pack(codes)[0, 0] == 0x10 and np.array_equal(O.unpack(O.pack(codes)), codes)


# ---------------------------------------------------------------------------
# Refusals of the C ABI: addresses that no call below reaches
# ---------------------------------------------------------------------------

A = 4096


def matrix(codes=A, scales=A, row_scale=A, rows=3, cols=64, format=NV):
    return ctypes.addressof(keep(fp4._MatrixStruct(codes, scales, row_scale, rows, cols, format)))


KEPT = []


def keep(x):
    KEPT.append(x)
    return x


BAD_MATRICES = [
    (dict(rows=-1), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(codes=A + 8), ALIGNMENT),
    (dict(scales=A + 4), ALIGNMENT), (dict(row_scale=A + 2), ALIGNMENT), (dict(cols=48), UNSUPPORTED),
    (dict(cols=0), UNSUPPORTED), (dict(cols=32800), UNSUPPORTED), (dict(format=2), UNSUPPORTED),
    (dict(rows=(1 << 24) + 1), UNSUPPORTED),
]


@pytest.mark.parametrize("bad,rc", BAD_MATRICES)
def test_matrices_are_checked(lib, bad, rc):
    m, cols = matrix(**bad), bad.get("cols", 64)
    good = matrix(cols=cols if cols % 32 == 0 and 32 <= cols <= 32768 else 64)
    assert lib.fp4_quantize(A, 32768, 0, m, None) == rc
    assert lib.fp4_dequantize(m, A, 32768, 0, None) == rc
    assert lib.fp4_linear(m, good, None, A, 64, 0, None, None) == rc
    assert lib.fp4_linear(good, m, None, A, 1 << 25, 0, None, None) == rc
    assert lib.fp4_linear_rows(A, 32768, 0, 3, m, None, A, 1 << 25, 0, A, 1 << 40, None, None) == rc
    if "rows" not in bad and "cols" not in bad:
        assert lib.fp4_swiglu(A, 64, A, 64, 0, 3, 64, None, 0, 0, m, None) == rc
        assert lib.fp4_block_norm(A, 64, 0, A, 64, 0, None, None, 0, 0, 1.0, None, 1e-6, 3, 64, None, 0, None, 0, 0, m, None) == rc


BAD_ROWS = [  # data, stride, type of 3 x 64 rows
    (None, 64, 0, INVALID), (A + 8, 64, 0, ALIGNMENT), (A, 63, 0, INVALID), (A, 68, 0, ALIGNMENT), (A, 66, 2, ALIGNMENT),
    (A, 64, 3, UNSUPPORTED), (A, 64, -1, UNSUPPORTED), (A, 1 << 38, 0, INVALID), (A, -64, 0, INVALID),
]


@pytest.mark.parametrize("data,stride,kind,rc", BAD_ROWS)
def test_rows_are_checked(lib, data, stride, kind, rc):
    m = matrix()
    assert lib.fp4_quantize(data, stride, kind, m, None) == rc
    assert lib.fp4_dequantize(m, data, stride, kind, None) == rc
    assert lib.fp4_linear_rows(data, stride, kind, 3, m, None, A, 64, 0, A, 1 << 30, None, None) == rc
    out = (A, 64, 0)
    assert lib.fp4_swiglu(data, stride, A, 64, kind, 3, 64, *out, None, None) == rc
    assert lib.fp4_swiglu(A, 64, data, stride, kind, 3, 64, *out, None, None) == rc

    def norm(r=(A, 64, 0), y=(A, 64, 0), gate=(None, 0, 0), to=(A, 64), h=(A, 64, 0)):
        return lib.fp4_block_norm(*r, *y, None, *gate, 1.0, None, 1e-6, 3, 64, *to, *h, None, None)

    assert norm(r=(data, stride, kind)) == rc
    if data:  # (without: there is none)
        assert norm(y=(data, stride, kind)) == rc
        assert norm(h=(data, stride, kind)) == (UNSUPPORTED if kind == 2 else rc)
        assert norm(y=(A, 64, kind), gate=(data, stride, 64)) == rc
        if kind in (0, 2):
            assert norm(r=(A, 64, kind), to=(data, stride)) == rc


def test_outputs_of_products_are_checked(lib):
    m = matrix()
    for y, rc in (((None, 3, 0), INVALID), ((A + 1, 3, 0), ALIGNMENT), ((A + 2, 3, 2), ALIGNMENT), ((A, 2, 0), INVALID),
                  ((A, 3, 3), UNSUPPORTED), ((A, 1 << 38, 0), INVALID)):
        assert lib.fp4_linear(m, m, None, *y, None, None) == rc
        assert lib.fp4_linear_rows(A, 64, 0, 3, m, None, *y, A, 1 << 30, None, None) == rc
    assert lib.fp4_linear(m, m, A + 2, A, 3, 0, None, None) == ALIGNMENT
    assert lib.fp4_linear_rows(A, 64, 0, 3, m, A + 2, A, 3, 0, A, 1 << 30, None, None) == ALIGNMENT
    assert lib.fp4_linear(matrix(cols=96), m, None, A, 3, 0, None, None) == INVALID
    assert lib.fp4_linear(matrix(format=MX), m, None, A, 3, 0, None, None) == INVALID
    assert lib.fp4_linear(None, m, None, A, 3, 0, None, None) == INVALID
    assert lib.fp4_linear(m, None, None, A, 3, 0, None, None) == INVALID


def test_workspace_is_checked(lib):
    m = matrix()
    size = lib.fp4_linear_rows_workspace(m, 40)
    assert size >= 40 * 32 + fp4.fp4_scale_bytes(40, 64, NV) + 160
    assert lib.fp4_linear_rows_workspace(m, 0) > 0
    assert lib.fp4_linear_rows_workspace(m, -1) == 0 and lib.fp4_linear_rows_workspace(m, (1 << 24) + 1) == 0
    assert lib.fp4_linear_rows_workspace(None, 4) == 0 and lib.fp4_linear_rows_workspace(matrix(cols=48), 4) == 0
    call = lambda ws, n: lib.fp4_linear_rows(A, 64, 0, 40, m, None, A, 3, 0, ws, n, None, None)  # noqa: E731
    assert call(None, size) == INVALID and call(A + 4, size) == ALIGNMENT and call(A, 64) == SMALL
    assert lib.fp4_linear_rows(A, 64, 0, -1, m, None, A, 3, 0, A, size, None, None) == INVALID


def test_norm_refusals(lib):
    def norm(y=(A, 64, 0), post=None, gate=(None, 0, 0), scale=1.0, w=None, eps=1e-6, rows=3, cols=64, h=(A, 64, 0), m=None):
        return lib.fp4_block_norm(A, 64, 0, *y, post, *gate, scale, w, eps, rows, cols, None, 0, *h, m, None)

    nan, inf = float("nan"), float("inf")
    assert [norm(eps=e) for e in (-1e-6, nan, inf)] == [INVALID] * 3
    assert [norm(scale=s) for s in (nan, inf, -inf)] == [INVALID] * 3
    assert norm(rows=-1) == INVALID and norm(cols=40) == UNSUPPORTED and norm(h=(None, 0, 0)) == INVALID
    assert norm(y=(None, 0, 0), post=A) == INVALID and norm(y=(None, 0, 0), gate=(A, 64, 64)) == INVALID
    assert norm(post=A + 4) == ALIGNMENT and norm(w=A + 8) == ALIGNMENT
    assert norm(gate=(A, 64, 2)) == INVALID and norm(gate=(A, 0, 0)) == INVALID
    assert norm(gate=(A + 1, 1, 1)) == ALIGNMENT and norm(gate=(A, -1, 1)) == INVALID
    assert norm(m=matrix(rows=4)) == INVALID and norm(m=matrix(cols=96)) == INVALID
    assert norm(m=matrix(row_scale=None)) == INVALID  # NVFP4 needs its rows' scales


def test_swiglu_and_scales_refusals(lib):
    assert lib.fp4_swiglu(A, 64, A, 64, 0, 3, 64, None, 0, 0, None, None) == INVALID
    assert lib.fp4_swiglu(A, 64, A, 64, 0, -1, 64, A, 64, 0, None, None) == INVALID
    assert lib.fp4_swiglu(A, 64, A, 64, 0, 3, 50, A, 64, 0, None, None) == UNSUPPORTED
    assert lib.fp4_swiglu(A, 64, A, 64, 0, 3, 64, A, 64, 2, None, None) == UNSUPPORTED
    assert lib.fp4_tile_scales(None, 3, 64, NV, A, None) == INVALID
    assert lib.fp4_tile_scales(A, 3, 64, NV, None, None) == INVALID
    assert lib.fp4_tile_scales(A, -3, 64, NV, A, None) == INVALID
    assert lib.fp4_tile_scales(A, 3, 65, NV, A, None) == UNSUPPORTED
    assert lib.fp4_tile_scales(A, 3, 64, NV, A + 8, None) == ALIGNMENT
    assert lib.fp4_quantize(A, 64, 0, None, None) == INVALID
    assert lib.fp4_quantize(A, 64, 0, matrix(row_scale=None), None) == INVALID


def test_no_rows_need_nothing(lib):
    none = matrix(None, None, None, rows=0)
    assert lib.fp4_quantize(None, 0, 0, none, None) == OK
    assert lib.fp4_dequantize(none, None, 0, 0, None) == OK
    assert lib.fp4_linear(none, matrix(), None, None, 0, 0, None, None) == OK
    assert lib.fp4_linear(matrix(), none, None, None, 0, 0, None, None) == OK
    assert lib.fp4_linear_rows(None, 0, 0, 0, matrix(), None, None, 0, 0, None, 0, None, None) == OK
    assert lib.fp4_swiglu(None, 0, None, 0, 0, 0, 64, None, 0, 0, None, None) == OK
    assert lib.fp4_block_norm(None, 0, 0, None, 0, 0, None, None, 0, 0, 1.0, None, 1e-6, 0, 64, None, 0, None, 0, 0, None, None) == OK
    assert lib.fp4_tile_scales(None, 0, 64, NV, None, None) == OK


# (3 x 64 BF16 rows are 384 bytes, FP32 768; a 3 x 64 NVFP4 matrix 96 + 512 + 12)
X_AT, Y_AT, CODES, SCALES, FACTORS = 1 << 20, 1 << 21, 1 << 22, 1 << 23, 1 << 24


def placed(codes=CODES, scales=SCALES, factors=FACTORS, **shape):
    return matrix(codes, scales, factors, **shape)


def test_rows_between_one_another_are_apart(tmp_path):
    """csrc/fp4_span.h against sets of bytes by tests/fp4_span_check.cu."""
    exe = tmp_path / "fp4_span_check"
    cmd = [build._nvcc(), "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-I", build.CSRC, "-o", str(exe),
           os.path.join(ROOT, "tests", "fp4_span_check.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and ", 0 failed" in r.stdout, r.stdout[-3000:]


def test_outputs_over_inputs_are_refused_by_the_quantiser(lib):
    for at in (X_AT, X_AT + 16, X_AT + 368, X_AT - 80):
        assert lib.fp4_quantize(X_AT, 64, 0, placed(codes=at), None) == INVALID
        assert lib.fp4_dequantize(placed(codes=at), X_AT, 64, 0, None) == INVALID
    for at in (X_AT, X_AT + 368, X_AT - 496):
        assert lib.fp4_quantize(X_AT, 64, 0, placed(scales=at), None) == INVALID
        assert lib.fp4_dequantize(placed(scales=at), X_AT, 64, 0, None) == INVALID
    for at in (X_AT, X_AT + 380, X_AT - 8):
        assert lib.fp4_quantize(X_AT, 64, 0, placed(factors=at), None) == INVALID
        assert lib.fp4_dequantize(placed(factors=at), X_AT, 64, 0, None) == INVALID
    # a row behind two others that lie 256 bytes apart
    assert lib.fp4_quantize(X_AT, 128, 0, placed(codes=X_AT + 2 * 256 + 112), None) == INVALID
    for parts in (dict(scales=CODES + 80), dict(factors=CODES + 92), dict(factors=SCALES + 508)):
        assert lib.fp4_quantize(X_AT, 64, 0, placed(**parts), None) == INVALID
    for at in (X_AT, X_AT - 496):
        assert lib.fp4_tile_scales(X_AT, 3, 64, NV, at, None) == INVALID


def test_outputs_over_inputs_are_refused_by_swiglu(lib):
    def call(out=(None, 0, 0), m=None, up=(Y_AT, 64), kind=0):
        return lib.fp4_swiglu(X_AT, 64, *up, kind, 3, 64, *out, m, None)

    for at in (X_AT + 16, X_AT - 128, X_AT + 128, X_AT + 256, Y_AT + 128, Y_AT - 256):  # shifted by some elements or rows
        assert call(out=(at, 64, 0)) == INVALID
    assert call(out=(X_AT, 72, 0)) == INVALID  # another stride
    assert call(out=(X_AT, 64, 0), kind=2) == INVALID and call(out=(X_AT, 128, 0), kind=2) == INVALID  # other elements
    for m in (placed(codes=X_AT), placed(scales=Y_AT), placed(factors=X_AT + 4)):
        assert call(m=m) == INVALID
    for m in (placed(codes=Y_AT), placed(scales=Y_AT), placed(factors=Y_AT)):
        assert call(out=(Y_AT, 64, 0), up=(X_AT, 64), m=m) == INVALID  # two outputs


def test_outputs_over_inputs_are_refused_by_the_norm(lib):
    R, H, G, W, V = 1 << 25, 1 << 26, 1 << 27, 1 << 28, 1 << 29

    def call(to=(None, 0), h=(H, 64, 0), m=None, r=(R, 64, 0), y=(Y_AT, 64, 0), gate=(G, 64, 64)):
        return lib.fp4_block_norm(*r, *y, V, *gate, 1.0, W, 1e-6, 3, 64, *to, *h, m, None)

    for at in (R + 128, R - 128, R + 256, R - 256, R + 16, Y_AT + 128, G + 128, G - 256, W, V, W + 240, V - 368, H, H + 128):
        assert call(to=(at, 64)) == INVALID, at
    for at in (R + 128, Y_AT - 128, G + 16, W, V):
        assert call(h=(at, 64, 0)) == INVALID, at
    assert call(to=(R, 72)) == INVALID and call(to=(Y_AT, 72)) == INVALID
    assert call(to=(Y_AT, 64), y=(Y_AT, 64, 2), gate=(None, 0, 0)) == INVALID  # other elements
    assert call(to=(G, 64), gate=(G, 0, 64)) == INVALID      # one row of gates for all rows
    assert call(to=(G, 64), gate=(G + 32, 64, 1)) == INVALID  # a gate for each row
    assert call(h=(G, 64, 0), gate=(G + 256, 0, 1)) == INVALID
    for parts in (dict(codes=R), dict(scales=Y_AT + 128), dict(factors=G + 380), dict(codes=W), dict(scales=V), dict(factors=H)):
        assert call(m=placed(**parts)) == INVALID, parts


def test_outputs_over_inputs_are_refused_by_products(lib):
    X, B, S, WS = 1 << 25, 1 << 26, 1 << 27, 1 << 28
    x, w = matrix(X, X + 4096, X + 8192), placed()

    def call(y, bias=B, status=S):
        return lib.fp4_linear(x, w, bias, y, 3, 2, status, None)

    for at in (X, X + 92, X - 32, X + 4096, X + 4096 + 508, X + 8192, X + 8200, CODES, SCALES - 4, FACTORS + 8, B, B + 8, B - 32, S, S - 32):
        assert call(at) == INVALID, at
    assert call(Y_AT, status=X + 4) == INVALID and call(Y_AT, status=B) == INVALID
    size = lib.fp4_linear_rows_workspace(w, 3)

    def rows(y=Y_AT, ws=WS, bias=B, x=X, status=S):
        return lib.fp4_linear_rows(x, 64, 0, 3, w, bias, y, 3, 2, ws, size, status, None)

    for at in (X, X + 380, X - 32, CODES, SCALES + 508, FACTORS, B, WS, WS + 96, S):
        assert rows(y=at) == INVALID, at
    for at in (X, X - 16, CODES, SCALES, FACTORS, B, Y_AT, Y_AT - 16):
        assert rows(ws=at) == INVALID, at
    assert rows(status=WS + 8) == INVALID


# ---------------------------------------------------------------------------
# Refusals of the binding: tensors that claim a device
# ---------------------------------------------------------------------------

class Claims:
    """A CPU tensor that says it is on a device."""

    def __init__(self, t, index=0):
        self._t, self._index = t, index

    def get_device(self):
        return self._index

    @property
    def is_cuda(self):
        return True

    def __getattr__(self, name):
        return getattr(self._t, name)


@pytest.fixture
def here(monkeypatch):
    """cuda:0 is current, and nothing reaches the library."""
    class Library:
        def __getattr__(self, name):
            def called(*args):
                raise AssertionError(f"{name} called")
            return called

    monkeypatch.setattr(fp4, "_current", lambda: 0)
    monkeypatch.setattr(fp4, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(fp4, "_LIB", Library())


def on(t, index=0):
    return Claims(t, index)


def held(rows=4, cols=64, format=NV, index=0):
    scales = torch.zeros(fp4._scale_bytes(rows, cols, format), dtype=torch.uint8)
    return fp4.Fp4Matrix(on(torch.zeros(rows, cols // 2, dtype=torch.uint8), index), on(scales, index),
                         on(torch.ones(rows), index), rows, cols, format)


X = torch.zeros(4, 64, dtype=torch.bfloat16)
CALLS = {
    "quantize": lambda x, **kw: fp4.fp4_quantize(x, **kw),
    "swiglu": lambda x, **kw: fp4.fp4_swiglu(x, x, **kw),
    "norm": lambda x, **kw: fp4.fp4_block_norm(x, x, **kw),
    "linear_rows": lambda x, **kw: fp4.fp4_linear_rows(x, held(index=x.get_device()), workspace=on(torch.zeros(8, dtype=torch.uint8)),
                                                       out=on(torch.zeros(4, 4)), **kw),
}


@pytest.mark.parametrize("call", CALLS)
def test_another_device_is_refused(call, here):
    with pytest.raises(fp4.MoeError, match="cuda:0 is current"):
        CALLS[call](on(X, 1))
    with pytest.raises(fp4.MoeError, match="the stream on cuda:1"):
        CALLS[call](on(X), stream=types.SimpleNamespace(device_index=1, cuda_stream=7))


def test_operands_of_two_devices_are_refused(here):
    with pytest.raises(fp4.MoeError, match="up must be"):
        fp4.fp4_swiglu(on(X), on(X, 1))
    with pytest.raises(fp4.MoeError, match="cuda:1"):
        fp4.fp4_linear(held(index=1), held())
    with pytest.raises(fp4.MoeError, match="out must be"):
        fp4.fp4_quantize(on(X), out=held(index=1))


@pytest.mark.parametrize("x", [None, 3, [1.0], torch.zeros(4, 64)], ids=["none", "number", "list", "cpu"])
def test_what_is_no_tensor_on_a_device_is_refused(x, here):
    for call in ("quantize", "swiglu", "norm"):
        with pytest.raises(fp4.MoeError, match="must be a CUDA tensor"):
            CALLS[call](x) if x is not None or call != "norm" else fp4.fp4_block_norm(None)
    for call in (lambda: fp4.fp4_linear(held(), x), lambda: fp4.fp4_linear(x, held()), lambda: fp4.fp4_dequantize(x),
                 lambda: fp4.fp4_linear_rows(on(X), x), lambda: fp4.fp4_linear_rows_workspace(x, 3)):
        with pytest.raises(fp4.MoeError, match="must be an FP4 matrix"):
            call()


def test_shapes_strides_and_types_are_refused(here):
    bad = [X.t(), X[:, ::2], X[0], X.double(), X[None], X.to(torch.uint8)]
    for x in bad:
        with pytest.raises(fp4.MoeError, match="x must be"):
            fp4.fp4_quantize(on(x), out=held())
    with pytest.raises(fp4.MoeError, match="up must be"):
        fp4.fp4_swiglu(on(X), on(X[:3]))
    with pytest.raises(fp4.MoeError, match="one type"):
        fp4.fp4_swiglu(on(X), on(X.half()))
    with pytest.raises(fp4.MoeError, match="y must be"):
        fp4.fp4_block_norm(on(X), on(X[:, :32]))
    with pytest.raises(fp4.MoeError, match="r_out must be"):
        fp4.fp4_block_norm(on(X), on(X), r_out=on(X.float()))
    with pytest.raises(fp4.MoeError, match="go with y"):
        fp4.fp4_block_norm(on(X), post_weight=on(torch.ones(64)))
    for gate in (X.half(), X[:, :2], X[:3], X.t(), X[:, 0]):
        with pytest.raises(fp4.MoeError, match="gate must be"):
            fp4.fp4_block_norm(on(X), on(X), gate=on(gate), r_out=on(X))
    for w in (torch.ones(63), torch.ones(64, dtype=torch.bfloat16), torch.ones(128)[::2]):
        with pytest.raises(fp4.MoeError, match="weight must be"):
            fp4.fp4_block_norm(on(X), weight=on(w), out=on(X))
    with pytest.raises(fp4.MoeError, match="neither"):
        fp4.fp4_swiglu(on(X), on(X), dtype=None)
    for dtype in (torch.float32, torch.uint8, "bf16"):
        with pytest.raises(fp4.MoeError, match="dtype must be"):
            fp4.fp4_swiglu(on(X), on(X), dtype=dtype)
    with pytest.raises(fp4.MoeError, match="dtype must be one of"):
        fp4.fp4_linear(held(), held(), dtype=torch.float64)
    with pytest.raises(fp4.MoeError, match="same columns and format"):
        fp4.fp4_linear(held(cols=96), held())
    with pytest.raises(fp4.MoeError, match="same columns and format"):
        fp4.fp4_linear(held(format=MX), held())
    with pytest.raises(fp4.MoeError, match=r"x must be \[tokens, 64\]"):
        fp4.fp4_linear_rows(on(X[:, :32]), held())
    with pytest.raises(fp4.MoeError, match="bias must be"):
        fp4.fp4_linear(held(), held(), bias=on(torch.zeros(5)), out=on(torch.zeros(4, 4)))
    with pytest.raises(fp4.MoeError, match="out must be"):
        fp4.fp4_linear(held(), held(), out=on(torch.zeros(4, 5)))
    for ws in (None, torch.zeros(8), 5):
        if ws is not None:
            with pytest.raises(fp4.MoeError, match="workspace must be"):
                fp4.fp4_linear_rows(on(X), held(), out=on(torch.zeros(4, 4)), workspace=on(ws) if torch.is_tensor(ws) else ws)
    with pytest.raises(fp4.MoeError, match="of format 1"):
        fp4.fp4_quantize(on(X), MX, out=held())
    with pytest.raises(fp4.MoeError, match="matrix must be"):
        fp4.fp4_swiglu(on(X), on(X), dtype=None, matrix=held(rows=5))


def test_shapes_of_matrices_are_refused(here):
    for rows, cols, format in ((4, 48, NV), (4, 0, NV), (4, 32800, NV), (-1, 64, NV), ((1 << 24) + 1, 64, NV), (4, 64, 2), (4, 64, None)):
        with pytest.raises(fp4.MoeError, match="no FP4 matrix"):
            fp4.fp4_empty(rows, cols, format)
    with pytest.raises(fp4.MoeError, match="scales must be"):
        fp4.fp4_matrix(on(torch.zeros(4, 32, dtype=torch.uint8)), on(torch.zeros(4, 2, dtype=torch.uint8)))
    with pytest.raises(fp4.MoeError, match="row_scale must be"):
        fp4.fp4_matrix(on(torch.zeros(4, 32, dtype=torch.uint8)), on(torch.zeros(4, 4, dtype=torch.uint8)), on(torch.zeros(3)))
    with pytest.raises(fp4.MoeError, match="codes must be"):
        fp4.fp4_matrix(on(torch.zeros(4, 32)), on(torch.zeros(4, 4, dtype=torch.uint8)))
    with pytest.raises(fp4.MoeError, match="rows must be"):
        fp4.fp4_linear_rows_workspace(held(), 1 << 25)


def test_a_matrix_is_made_of_its_parts_alone(lib):
    """Parts that do not fit the shape would be read past their ends; a part that is replaced later
    would leave its address behind."""
    codes, scales, row = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.ones(4)
    for parts, wrong in (((codes[:3], scales, row), "codes"), ((codes, scales[:511], row), "scales"),
                         ((codes, scales, row[:3]), "row_scale"), ((codes.float(), scales, row), "codes"),
                         ((codes, scales.view(4, 128), row), "scales"), ((codes, scales, row.double()), "row_scale")):
        with pytest.raises(fp4.MoeError, match=f"{wrong} must be"):
            fp4.Fp4Matrix(*parts, 4, 64, NV)
    with pytest.raises(fp4.MoeError, match="no FP4 matrix"):
        fp4.Fp4Matrix(codes, scales, row, 4, 48, NV)
    m = fp4.Fp4Matrix(codes, scales, row, 4, 64, NV)
    for name in ("codes", "scales", "row_scale"):
        with pytest.raises(AttributeError):
            setattr(m, name, getattr(m, name))


def test_copies_describe_their_own_tensors(lib):
    codes = torch.arange(4 * 32, dtype=torch.uint8).view(4, 32)
    m = fp4.Fp4Matrix(codes, torch.full((512,), 56, dtype=torch.uint8), None, 4, 64, NV)
    for other in (copy.deepcopy(m), pickle.loads(pickle.dumps(m))):
        assert other.struct.codes == other.codes.data_ptr() != codes.data_ptr() and other.struct.scales == other.scales.data_ptr()
        assert other.struct.row_scale is None and other.row_scale is None and other.at == ctypes.addressof(other.struct)
        assert torch.equal(other.codes, codes) and other.shape == (4, 64) and other.format == NV
    assert copy.copy(m).struct.codes == codes.data_ptr()
