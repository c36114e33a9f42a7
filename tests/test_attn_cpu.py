"""The attention operators' C ABI and oracle on the host: exports, refusals
that return before any CUDA call, and the oracle against plain loops."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest

from block_scaled_fp4_softmax_gb300 import attn, build
from oracle import attn as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ONE = 4096  # an aligned address that no call below reaches


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load()


def test_header_and_library_carry_the_binding_names(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(attn_[a-z0-9_]*)\s*\(", text))
    assert names == set(attn.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    assert names <= exported


def cache(**kw):
    c = dict(k=ONE, v=ONE, page_stride=4 * 16 * 128, head_stride=16 * 128, row_stride=128, page_table=ONE, batch=2,
             max_pages=8, pages=16, page_size=16, kv_heads=4, head_dim=128, dtype=attn.BF16)
    c.update(kw)
    return ctypes.byref(attn._CacheStruct(**c))


def tree(lib, c, q=ONE, stride=8 * 128, tokens=3, heads=8, words=None, count=0, out=ONE, ws=ONE, nbytes=1 << 40):
    return lib.attn_tree_decode(q, stride, ONE, ONE, tokens, heads, words, count, 0.1, c, out, ONE, ws, nbytes, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), 1), (dict(page_table=None), 1), (dict(batch=0), 1), (dict(pages=-1), 1), (dict(kv_heads=0), 1),
    (dict(dtype=2), 3), (dict(head_dim=12), 3), (dict(head_dim=264), 3), (dict(head_dim=8), 3),
    (dict(page_size=12), 3), (dict(page_size=0), 3), (dict(page_size=1 << 21), 3),
    (dict(max_pages=1 << 28), 3), (dict(row_stride=64), 3), (dict(head_stride=0), 3), (dict(page_stride=2049), 3),
    (dict(k=ONE + 2), 2), (dict(v=ONE + 8), 2),
])
def test_unsupported_caches_are_refused_by_every_entry(lib, kw, status):
    c = cache(**kw)
    assert tree(lib, c) == status
    assert lib.attn_tree_decode_workspace(c) == 0
    assert lib.attn_cache_evict_workspace(c, 10) == 0
    assert lib.attn_qk_norm_rope(ONE, ONE, ONE, 1024, 512, 512, ONE, ONE, ONE, 3, 8, ONE, ONE, 1e-6, ONE, 128, 0, 1.0,
                                 ONE, None, 0, c, None, None) == status
    assert lib.attn_cache_weights(ONE, 1024, ONE, ONE, ONE, 3, 8, None, 0, 0.1, c, ONE, 1.0, ONE, 128, None, None) == status
    assert lib.attn_cache_evict(c, ONE, ONE, 128, ONE, ONE, 10, 0, 0, ONE + 16, ONE + 16, ONE + 16, ONE, 1 << 40, None,
                                None) == status


def test_strides_of_single_axes_are_of_no_account(lib):
    assert lib.attn_cache_evict_workspace(cache(kv_heads=1, head_stride=0), 10) > 0
    assert lib.attn_cache_evict_workspace(cache(pages=1, page_stride=3), 10) > 0


def test_tree_decode_refusals(lib):
    c = cache()
    assert tree(lib, c, q=None) == 1
    assert tree(lib, c, out=None) == 1
    assert tree(lib, c, ws=None) == 1
    assert tree(lib, c, tokens=-1) == 1
    assert tree(lib, c, words=ONE, count=0) == 1
    assert tree(lib, c, heads=6) == 3            # not a multiple of kv_heads
    assert tree(lib, c, stride=1023) == 3
    assert tree(lib, c, stride=1016) == 3        # tokens would overlap
    assert tree(lib, c, q=ONE + 2) == 2
    assert tree(lib, c, nbytes=0) == 4


def test_rope_refusals(lib):
    def rope(q=ONE, k=ONE, v=ONE, sk=512, sv=512, wq=ONE, wk=ONE, eps=1e-6, freq=ONE, rot=128, out=2 * ONE, sp=None, cap=0,
             sq=1024):
        return lib.attn_qk_norm_rope(q, k, v, sq, sk, sv, ONE, ONE, ONE, 3, 8, wq, wk, eps, freq, rot, 0, 1.0, out, sp, cap,
                                     cache(), None, None)
    assert rope(k=None) == 1 and rope(out=None) == 1 and rope(freq=None) == 1 and rope(wq=None) == 1
    assert rope(eps=-1.0) == 1 and rope(eps=math.nan) == 1 and rope(rot=-2) == 1 and rope(sp=ONE, cap=0) == 1
    assert rope(rot=7) == 3 and rope(rot=130) == 3 and rope(sk=511) == 3 and rope(sv=504) == 3
    assert rope(k=ONE + 4) == 2 and rope(wk=ONE + 2) == 2
    assert rope(out=ONE, sq=2048) == 1           # in place needs packed tokens


def test_weights_and_evict_refusals(lib):
    c = cache()

    def weights(lse=ONE, acc=ONE, out=ONE, cap=128, heads=8):
        return lib.attn_cache_weights(ONE, 1024, lse, ONE, ONE, 3, heads, None, 0, 0.1, c, acc, 1.0, out, cap, None, None)

    def evict(acc=ONE, out=2 * ONE, pout=2 * ONE, budget=10, sinks=0, recent=0, cap=128, ws=ONE, nbytes=1 << 40):
        return lib.attn_cache_evict(c, acc, ONE, cap, ONE, ONE, budget, sinks, recent, out, pout, 2 * ONE, ws, nbytes, None, None)

    assert weights(lse=None) == 1 and weights(acc=None) == 1 and weights(out=None) == 1 and weights(cap=0) == 1
    assert weights(heads=9) == 3
    assert evict(acc=None) == 1 and evict(out=ONE) == 1 and evict(pout=ONE) == 1 and evict(budget=0) == 1
    assert evict(sinks=-1) == 1 and evict(recent=-1) == 1 and evict(cap=0) == 1 and evict(ws=None) == 1
    assert evict(ws=ONE + 4) == 2 and evict(nbytes=8 * 10 * 8) == 4


def test_binding_refuses_tensors_of_the_wrong_kind():
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(attn.MoeError):
        attn.attn_cache(k, k, torch.zeros(1, 4, dtype=torch.int32))  # not on a GPU


# ---------------------------------------------------------------------------
# Oracle pins
# ---------------------------------------------------------------------------

def test_oracle_attention_against_loops():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=6), rng.normal(size=(9, 6)), rng.normal(size=(9, 6))
    mask = np.array([1, 1, 0, 1, 1, 0, 1, 0, 1], dtype=bool)
    out, lse, _ = A.attend(q, k, v, mask, 0.4)
    e = [math.exp(0.4 * sum(q[d] * k[j][d] for d in range(6))) if mask[j] else 0.0 for j in range(9)]
    for d in range(6):
        assert abs(out[d] - sum(e[j] * v[j][d] for j in range(9)) / sum(e)) < 1e-13
    assert abs(lse - math.log(sum(e))) < 1e-13
    w = A.received(q[None], np.array([lse]), k, [mask], 0.4)
    assert abs(w.sum() - 1) < 1e-13 and np.all(w[~mask] == 0)
    assert np.all(A.received(q[None], np.array([-np.inf]), k, [mask], 0.4) == 0)
    zero, none, _ = A.attend(q, k, v, np.zeros(9, dtype=bool), 0.4)
    assert np.all(zero == 0) and none == -np.inf


def test_oracle_rotation_against_complex_numbers():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2, 8))
    freq, pos = np.array([1.0, 0.25, 0.01]), np.array([0, 5, 1000])
    for inter in (False, True):
        y = A.head_rows(x, None, 0.0, pos, freq, inter, 2.0)
        for t in range(3):
            for j in range(3):
                i0, i1 = (2 * j, 2 * j + 1) if inter else (j, j + 3)
                z = complex(x[t, 1, i0], x[t, 1, i1]) * np.exp(1j * pos[t] * freq[j]) * 2.0
                assert abs(complex(y[t, 1, i0], y[t, 1, i1]) - z) < 1e-12
        assert np.array_equal(y[..., 6:], x[..., 6:])


def test_oracle_eviction_by_hand():
    #      slot 0    1    2    3    4    5    6
    acc = [0.1, 0.9, 0.0, 0.9, np.nan, 0.5, 0.0]
    pos = [0, 1, 2, 3, 4, 5, 6]
    take, moves = A.evict(acc, pos, 4, 1, 1, 7)       # 0 and 6 are protected; then 1 and 3
    assert moves == [(6, 2)] and take.tolist() == [0, 1, 6, 3]
    take, moves = A.evict(acc, pos, 3, 0, 0, 7)       # 1, 3, 5
    assert moves == [(3, 0), (5, 2)] and take.tolist() == [3, 1, 5]
    take, moves = A.evict(acc, pos, 6, 0, 0, 7)       # NaN goes first
    assert moves == [(6, 4)] and A.evict(acc, pos, 7, 0, 0, 7)[1] == []
    assert A.evict([0.0, -0.0, 0.0], [0, 1, 2], 2, 0, 0, 3)[1] == []


def test_oracle_tree_rows():
    words = np.array([[0b1, 0], [0b11, 0], [0, 0]], dtype=np.uint64)
    assert A.sees(words, 2, 0, 3).tolist() == [True, True, True, False, False]
    assert A.sees(words, 2, 2, 3).tolist() == [True, True, False, False, False]
    assert A.sees(None, 1, 1, 3).tolist() == [True, True, True, False]


def test_work_division_on_host(tmp_path):
    """csrc/attn_plan.h walked for thousands of batches by tests/attn_plan_check.cu."""
    exe = tmp_path / "attn_plan_check"
    cmd = [build._nvcc(), "-std=c++17", "-O2", "-gencode", "arch=compute_103a,code=sm_103a", "-I", build.CSRC, "-o", str(exe),
           os.path.join(ROOT, "tests", "attn_plan_check.cu")]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and ", 0 failed" in r.stdout, r.stdout[-3000:]
