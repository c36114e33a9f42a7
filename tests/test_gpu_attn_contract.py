"""The attention operators where include/attn.h promises something that random
inputs do not show: infinite keys, rows that add nothing, slots without a position, more
protected slots than stay, infinite values, chains of a prompt's length."""
import numpy as np
import pytest
import torch

from attn_helpers import Batch, f64, trees
from block_scaled_fp4_softmax_gb300 import attn
from test_gpu_attn import BF, FP, attend, run_evict
from test_gpu_attn_long import CASES, test_long_caches as check_long

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim,lens,new", [
    (BF, 128, [300, 77], [2, 1]), (FP, 64, [300, 5000], [40, 3]), (BF, 256, [200, 7000], [20, 33]),
    (FP, 72, [30000], [1]),
])
def test_infinite_committed_values(dtype, dim, lens, new):
    """Every token sees them with a weight above 0: what they make of their own column, and
    nothing of the others."""
    bt = Batch(dtype, lens, new, 2, 4, dim, 16, True, trees(new, 5), seed=dim, sharp=0.3)
    want, want_lse = attend(bt)
    inf = float("inf")
    for b, n in enumerate(lens):
        page, row = bt.rows(b)
        for slot, d, x in ((0, 1, inf), (n - 1, 1, inf), (n // 2, 9, -inf), (3, dim - 1, inf), (n - 2, dim - 1, -inf),
                           (7, dim - 2, float("nan"))):
            bt.v[page[slot], 1, row[slot], d] = x
    out, lse = attend(bt)
    assert int(bt.status) == 0 and torch.equal(lse, want_lse)
    assert torch.equal(out[:, :4].view(torch.int16), want[:, :4].view(torch.int16))
    assert (out[:, 4:, 1] == inf).all() and (out[:, 4:, 9] == -inf).all() and torch.isnan(out[:, 4:, dim - 2:]).all()
    rest = [d for d in range(dim) if d not in (1, 9, dim - 2, dim - 1)]
    assert torch.equal(out[:, 4:, rest].view(torch.int16), want[:, 4:, rest].view(torch.int16))


@pytest.mark.parametrize("batch", [2, 64], ids=["divided", "whole"])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64), (BF, 256)])
def test_weights_of_zero_meet_infinite_values(dtype, dim, batch):
    """A seen key of score -inf has weight 0, and 0 * inf is NaN, however the work is divided: also
    where a piece, or one of its two streams, holds no other key that the row sees."""
    new = [3] * batch
    bt = Batch(dtype, [129] * batch, new, 8, 2, dim, 16, True, trees(new, 4, blind=(0, 1, 2)), seed=dim)
    bt.q[:, :, 5] = -1.0
    for b in range(batch):
        page, row = bt.rows(b)
        bt.k[page[128], :, row[128], 5] = float("inf")
    want, want_lse = attend(bt)
    assert torch.isfinite(want).all() and torch.isfinite(want_lse).all()
    for b in range(batch):
        page, row = bt.rows(b)
        bt.v[page[128], :, row[128], 3] = float("inf")
    out, lse = attend(bt)
    assert torch.isnan(out[:, :, 3]).all() and torch.equal(lse, want_lse)
    rest = [d for d in range(dim) if d != 3]
    assert torch.equal(out[:, :, rest].view(torch.int16), want[:, :, rest].view(torch.int16))


@pytest.mark.parametrize("case", [
    (BF, [0], [2451], 2, 4, 128, 64, False),           # a prompt into an empty cache
    (FP, [4096, 0], [256, 1031], 1, 8, 64, 16, False),  # a later part of one, beside another
    (BF, [130], [1300], 1, 3, 256, 24, False),
])
def test_chains_of_a_prompts_length(case, monkeypatch):
    """Attention and weights of thousands of tokens in flight, as for long caches."""
    monkeypatch.setitem(CASES, "chain", case)
    check_long("chain")


# ---------------------------------------------------------------------------
# Weights
# ---------------------------------------------------------------------------

def weights_near(bt, lse, acc, got, bound):
    """As for other weights: a score off by d changes its weight by a factor exp(d); FP32 sums of n rows."""
    want = bt.expected_weights(f64(lse), f64(acc), 0.875)
    got, there = f64(got), ~np.isnan(want)
    assert np.isfinite(got[there]).all(), np.argwhere(~np.isfinite(got) & there)[:4].tolist()
    d = bt.dim * 2.0 ** -23 * bound + 2.0 ** -18
    n = max(1, max(bt.new_list)) * bt.group
    tol = (4 * d + n * 2.0 ** -24) * np.abs(want) + 2.0 ** -40
    assert np.all(np.abs(got - want)[there] <= tol[there]), float(np.abs(got - want)[there].max())


@pytest.mark.parametrize("dtype,dim,group,new,tree", [
    (BF, 128, 3, [1, 1], False),     # few rows
    (FP, 64, 8, [4, 4], False),      # rows that fill groups of 32
    (BF, 72, 7, [7, 1], True),
    (FP, 128, 8, [63, 20], True),    # several chunks, the last one not full
    (BF, 256, 5, [60, 3], True),     # several passes
])
def test_a_key_at_minus_infinity_receives_nothing(dtype, dim, group, new, tree):
    """Every row's score of an infinite key is -inf: its weight is 0, for committed keys
    among others, next to the drafts, and for a draft."""
    bt = Batch(dtype, [300, 77], new, 2, group, dim, 16, True, trees(new, 5) if tree else None, seed=dim + group)
    bound = bt.dot_bound()
    bt.q[:, :, 5] = -1.0
    for b, slots in enumerate(([0, 130, 299, 300], [0, 31, 40, 76])):
        page, row = bt.rows(b)
        for s in slots:
            bt.k[page[s], :, row[s], 5] = float("inf")
    out, lse = attend(bt)
    assert int(bt.status) == 0
    # a token whose one draft is infinite still sees the committed keys
    assert torch.isfinite(lse).all() and torch.isfinite(out).all()
    acc = torch.rand(2, 2, bt.cap, device="cuda")
    got = attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, tree=bt.tree, decay=0.875,
                                  dev_status=bt.status)
    assert int(bt.status) == 0
    with np.errstate(invalid="ignore"):
        weights_near(bt, lse, acc, got, bound)
    for b, slots in enumerate(([0, 130, 299], [0, 31, 40, 76])):
        assert torch.equal(got[b, :, slots], 0.875 * acc[b, :, slots])


@pytest.mark.parametrize("dtype,dim,group,new", [(BF, 128, 4, [9, 3]), (FP, 64, 8, [40, 12]), (BF, 256, 3, [50, 90])])
def test_rows_without_weight_add_nothing(dtype, dim, group, new):
    """lse = -inf takes a row out whatever its query holds."""
    bt = Batch(dtype, [200, 500], new, 2, group, dim, 16, True, trees(new, 6), seed=dim)
    _, lse = attend(bt)
    bound = bt.dot_bound()
    t = new[0] - 2
    lse[t], lse[-1, 1], lse[0, 0] = -float("inf"), -float("inf"), -float("inf")
    bt.q[t], bt.q[-1, 1], bt.q[0, 0] = float("nan"), float("inf"), -float("inf")
    acc = torch.rand(2, 2, bt.cap, device="cuda")
    got = attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, tree=bt.tree, decay=0.875)
    weights_near(bt, lse, acc, got, bound)


# ---------------------------------------------------------------------------
# Norm, rotation, append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("cap,fits", [(42, 2), (40, 0), (44, 4)])
def test_a_slot_that_has_no_position_is_not_appended(cap, fits):
    """Tokens whose slots `slot_pos` does not hold: no row, no position, but the rotated q."""
    bt = Batch(BF, [40, 5], [4, 2], 2, 3, 64, 16, seed=3)
    pos = torch.tensor([40, 41, 42, 43, 5, 6], dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).cuda()
    k0, v0 = bt.k.clone(), bt.v.clone()
    want_q = attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq)
    k1, v1 = bt.k.clone(), bt.v.clone()
    bt.k.copy_(k0), bt.v.copy_(v0)
    slot_pos = torch.full((2, 2, cap), -9, dtype=torch.int32, device="cuda")
    q = attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq, slot_pos=slot_pos,
                               dev_status=bt.status)
    assert int(bt.status) == (0 if fits == 4 else attn.DEV_BAD_LENGTH)
    assert torch.equal(q, want_q)
    page, row = bt.rows(0)
    for s in range(40 + fits, 44):
        k1[page[s], :, row[s]], v1[page[s], :, row[s]] = k0[page[s], :, row[s]], v0[page[s], :, row[s]]
    assert torch.equal(bt.k.view(torch.int16), k1.view(torch.int16)) and torch.equal(bt.v.view(torch.int16), v1.view(torch.int16))
    want = torch.full_like(slot_pos, -9)
    want[0, :, 40:40 + fits] = pos[:fits]
    want[1, :, 5:7] = pos[4:]
    assert torch.equal(slot_pos, want)


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------

def test_protected_slots_are_ranked_by_weight():
    bt = Batch(BF, [5], [0], 1, 1, 64, 16, seed=1)
    acc, pos = torch.zeros(1, 1, 8, device="cuda"), torch.arange(8, dtype=torch.int32, device="cuda").view(1, 1, 8)
    acc[0, 0, :5] = torch.tensor([9.0, 1.0, 5.0, 7.0, 3.0])
    _, acc_out, pos_out = attn.attn_cache_evict(bt.cache, acc, pos, bt.lens, bt.lens, 3, recent=5)
    assert pos_out[0, 0, :3].tolist() == [0, 3, 2] and acc_out[0, 0, :3].tolist() == [9.0, 7.0, 5.0]


@pytest.mark.parametrize("lens,hk,page,budget,over", [
    ([900, 40, 700], 2, 16, 500, 37),           # one CTA, beside sequences that have room
    ([5000, 4001], 2, 64, 1000, 1),             # clusters of two and four
    ([900, 2000], 1, 16, 800, 0),               # exactly as many as stay
    ([70001], 1, 1024, 30001, 20011),           # 16 CTAs, rows not on 16 bytes
    ([420000], 1, 4096, 200001, 777),           # the same, aligned
    ([46001, 50, 45999] + [7] * 17, 8, 1024, 20011, 5000),  # keys that shared memory does not hold
])
@pytest.mark.parametrize("kind", ["ties", "special"])
def test_more_protected_slots_than_the_budget(lens, hk, page, budget, over, kind):
    """`over` protected slots too many: by weight, then by slot, NaN last."""
    bt = Batch(BF, lens, [0] * len(lens), hk, 1, 16, page, seed=budget + over)
    g = torch.Generator(device="cuda").manual_seed(over)
    if kind == "ties":
        acc = torch.rand(bt.B, hk, bt.cap, generator=g, device="cuda").mul_(300).round_()
    else:
        vals = torch.tensor([0.0, -0.0, float("nan"), float("inf"), -float("inf"), 1e-42, -1.0, 3.0, -float("nan")], device="cuda")
        acc = vals[torch.randint(0, len(vals), (bt.B, hk, bt.cap), generator=g, device="cuda")]
    # each sequence's positions are a permutation of 0 .. n - 1, in random order
    pos = torch.full((bt.B, hk, bt.cap), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        pos[b, :, :n] = torch.rand(hk, n, generator=g, device="cuda").argsort(dim=-1).to(torch.int32)
    sinks = 4
    run_evict(bt, acc, pos, lens, torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, sinks, budget + over - sinks)
