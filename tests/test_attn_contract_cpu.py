"""What include/attn.h promises and the host can show: the oracle's readings of it, and refusals."""
import ctypes
import types
from fractions import Fraction

import numpy as np
import pytest
import torch

from block_scaled_fp4_softmax_gb300 import attn, build
from oracle import attn as A


def test_oracle_ranks_protected_slots_by_weight():
    acc, pos = [9.0, 1.0, 5.0, 7.0, 3.0], [0, 1, 2, 3, 4]
    assert A.evict(acc, pos, 3, 0, 5, 5)[0].tolist() == [0, 3, 2]
    # two of three protected slots stay: NaN last, and no other slot whatever its weight
    assert A.evict([np.nan, 0.0, 100.0, -1.0], [0, 1, 2, 3], 2, 2, 1, 4)[0].tolist() == [3, 1]
    assert A.evict([np.nan, np.nan, 100.0, -1.0], [0, 1, 2, 3], 2, 2, 1, 4)[0].tolist() == [0, 3]


CALLS = {
    "rope": lambda c, **kw: attn.attn_qk_norm_rope(None, None, None, None, None, None, c, None, **kw),
    "tree": lambda c, **kw: attn.attn_tree_decode(None, None, None, c, **kw),
    "weights": lambda c, **kw: attn.attn_cache_weights(None, None, None, None, c, None, **kw),
    "evict": lambda c, **kw: attn.attn_cache_evict(c, None, None, None, None, 8, **kw),
}


@pytest.mark.parametrize("call", CALLS)
def test_a_cache_of_another_device_is_refused(call, monkeypatch):
    """Nothing is looked at, allocated or launched before."""
    cache = types.SimpleNamespace(index=1, device="cuda:1")
    monkeypatch.setattr(attn, "_current", lambda: 0)
    with pytest.raises(attn.MoeError, match="cuda:0 is current"):
        CALLS[call](cache)
    monkeypatch.setattr(attn, "_current", lambda: 1)
    with pytest.raises(attn.MoeError, match="the stream on cuda:0"):
        CALLS[call](cache, stream=types.SimpleNamespace(device_index=0, cuda_stream=7))


ONE = 4096  # an aligned address that no call below reaches


@pytest.fixture(scope="module")
def lib():
    build.build()
    return attn.load()


def cache(**kw):
    c = dict(k=ONE, v=ONE, page_stride=4 * 16 * 128, head_stride=16 * 128, row_stride=128, page_table=ONE, batch=2,
             max_pages=8, pages=16, page_size=16, kv_heads=4, head_dim=128, dtype=attn.BF16)
    c.update(kw)
    return ctypes.byref(attn._CacheStruct(**c))


def test_trees_without_words_are_refused(lib):
    """They would be taken for a chain, whose tokens see what came before them."""
    def calls(words, count):
        return (lib.attn_tree_decode(ONE, 1024, ONE, ONE, 3, 8, words, count, 0.1, cache(), ONE, ONE, ONE, 1 << 40, None, None),
                lib.attn_cache_weights(ONE, 1024, ONE, ONE, ONE, 3, 8, words, count, 0.1, cache(), ONE, 1.0, ONE, 128, None, None))

    for words, count in ((None, 1), (None, -1), (ONE, 0)):
        assert calls(words, count) == (1, 1)
    here = types.SimpleNamespace(index=-1, device="cpu")  # get_device() of a CPU tensor
    with pytest.raises(attn.MoeError, match="one word or more"):
        attn._tree(torch.zeros(3, 0, dtype=torch.int64), 3, here)
    with pytest.raises(attn.MoeError, match="one word or more"):
        attn._tree(torch.zeros(3, dtype=torch.int64), 3, here)
    rows = torch.zeros(3, 2, dtype=torch.int64)
    assert attn._tree(rows, 3, here) == (rows.data_ptr(), 2)
    # no tokens, no address: not to be taken for an array
    assert attn._tree(torch.zeros(0, 2, dtype=torch.int64), 0, here) == (None, 0)
    assert attn._tree(None, 3, here) == (None, 0)


def test_rows_beyond_an_int_are_refused(lib):
    """2^24 tokens of 128 query heads a KV head: 2^31 rows."""
    c = dict(kv_heads=1, head_dim=16, row_stride=16, head_stride=256, page_stride=256)

    def calls(tokens, heads):
        return (lib.attn_tree_decode(ONE, heads * 16, ONE, ONE, tokens, heads, None, 0, 0.1, cache(**c), None, ONE, ONE, 1 << 40, None, None),
                lib.attn_cache_weights(ONE, heads * 16, None, ONE, ONE, tokens, heads, None, 0, 0.1, cache(**c), ONE, 1.0, ONE, 128, None, None))

    assert calls(1 << 24, 128) == (3, 3)
    assert calls((1 << 24) - 16, 128) == (3, 3)       # 2^31 - 2048
    assert calls((1 << 24) - 17, 128) == (1, 1)       # fits: what is missing is found next
    assert calls(1 << 24, 127) == (1, 1)


@pytest.mark.parametrize("name", ["budget", "sinks", "recent"])
@pytest.mark.parametrize("value", [1 << 31, 1 << 32, (1 << 32) + 5, -1, -(1 << 32)])
def test_numbers_beyond_32_bits_are_refused(name, value, monkeypatch):
    """2^32 protected positions are not none."""
    def library():
        raise AssertionError("called")

    monkeypatch.setattr(attn, "_current", lambda: 0)
    monkeypatch.setattr(attn, "_raw_stream", lambda i: 0)
    monkeypatch.setattr(attn, "load", library)
    monkeypatch.setattr(attn, "_LIB", None)
    here = types.SimpleNamespace(index=0, device="cuda:0", batch=1, kv_heads=1, lens_shape=(1,), ref=None)
    acc = torch.zeros(1, 1, 8)
    args = dict(budget=4, sinks=0, recent=0) | {name: value}
    with pytest.raises(attn.MoeError, match=f"{name} must be"):
        attn.attn_cache_evict(here, acc, acc, acc, acc, workspace=acc, acc_out=acc, pos_out=acc, lens_out=acc, **args)
    if name == "budget":
        with pytest.raises(attn.MoeError, match="budget must be"):
            attn.attn_cache_evict_workspace(here, value)
    far = torch.empty(0, 1, 1 << 31)
    with pytest.raises(attn.MoeError, match="slot_cap must be"):
        attn.attn_cache_evict(here, far, acc, acc, acc, 4)


@pytest.mark.parametrize("what", [None, [1.0], 3, torch.zeros(())], ids=["none", "list", "number", "scalar"])
def test_what_has_no_shape_is_refused(what, monkeypatch):
    monkeypatch.setattr(attn, "_current", lambda: -1)
    monkeypatch.setattr(attn, "_raw_stream", lambda i: 0)
    here = types.SimpleNamespace(index=-1, device="cpu", dtype=torch.bfloat16, batch=1, kv_heads=2, head_dim=16,
                                 cu_shape=(2,), lens_shape=(1,), ref=None)  # index: get_device() of a CPU tensor
    x = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    ints, acc = torch.zeros(2, dtype=torch.int32), torch.zeros(1, 2, 8)
    lse, freq = torch.zeros(3, 2), torch.zeros(8, dtype=torch.float64)
    with pytest.raises(attn.MoeError, match="inv_freq"):
        attn.attn_qk_norm_rope(x, x, x, ints, ints, ints, here, what)
    if what is not None:
        with pytest.raises(attn.MoeError, match="slot_pos"):
            attn.attn_qk_norm_rope(x, x, x, ints, ints, ints, here, freq, slot_pos=what)
        with pytest.raises(attn.MoeError, match="tree"):
            attn.attn_tree_decode(x, ints, ints, here, tree=what)
        with pytest.raises(attn.MoeError, match="workspace"):
            attn.attn_tree_decode(x, ints, ints, here, out=x, lse=lse, workspace=what)
        with pytest.raises(attn.MoeError, match="workspace"):
            attn.attn_cache_evict(here, acc, acc, ints, ints, 4, acc_out=acc, pos_out=acc, lens_out=ints, workspace=what)
    with pytest.raises(attn.MoeError, match="acc"):
        attn.attn_cache_weights(x, lse, ints, ints, here, what)
    with pytest.raises(attn.MoeError, match="acc"):
        attn.attn_cache_evict(here, what, acc, ints, ints, 4)


def test_eviction_outputs_that_lie_in_inputs_are_refused(lib):
    """lens_out is written while other CTAs of the batch still read next_pos."""
    rows = 2 * 4 * 128 * 4

    def evict(acc=ONE, pos=ONE, lens=ONE, nxt=ONE, acc_out=16 * ONE, pos_out=16 * ONE, lens_out=16 * ONE):
        # the workspace is too small: the next thing to be found
        return lib.attn_cache_evict(cache(), acc, pos, 128, lens, nxt, 10, 0, 0, acc_out, pos_out, lens_out, ONE, 0, None, None)

    assert evict() == 4
    assert evict(lens_out=ONE) == 1 and evict(nxt=16 * ONE) == 1 and evict(lens=16 * ONE) == 1
    assert evict(lens_out=ONE + 4) == 1 and evict(lens_out=ONE + 8) == 4 and evict(lens_out=ONE - 8) == 4
    for name in ("acc", "pos"):
        for at in (4 * ONE, 4 * ONE + rows - 4, 4 * ONE - rows + 4):
            assert evict(**{name: 4 * ONE, name + "_out": at}) == 1
        for at in (4 * ONE + rows, 4 * ONE - rows):
            assert evict(**{name: 4 * ONE, name + "_out": at}) == 4


def test_angles_are_as_near_as_the_header_says():
    """The rotation's reduction, operation by operation, against pi to 60 digits."""
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)

    def turns(inv_freq, pos):
        t = np.float64(inv_freq) * np.float64(0.15915494309189533577)
        f = t - np.floor(t)
        u = int(f * np.float64(2.0 ** 64)) * pos % 2 ** 64
        top = u >> 32
        return Fraction(float(np.float32(top - 2 ** 32 if top >> 31 else top))) / 2 ** 32  # half turns / 2

    rng = np.random.default_rng(0)
    worst = 0
    for inv_freq in [1.0, 5.75, *rng.uniform(2.0 ** -9, 1.0, 200), *(10000.0 ** -rng.uniform(0.7, 1.0, 100) / 64)]:
        for pos in [0, 1, 2 ** 31 - 1, -2 ** 31, *map(int, rng.integers(-2 ** 31, 2 ** 31, 20))]:
            want = Fraction(float(inv_freq)) * pos / (2 * pi)
            off = turns(inv_freq, pos) - want
            off -= round(off)
            first = abs(pos) * (Fraction(float(inv_freq)) / 2 ** 54 if inv_freq >= 2.0 ** -9 else Fraction(1, 2 ** 63))
            bound = first + Fraction(1, 2 ** 26)
            assert abs(off) <= bound, (inv_freq, pos, float(off), float(bound))
            worst = max(worst, abs(off) / bound)
    assert worst > Fraction(1, 4)  # nor is the bound out of all proportion
