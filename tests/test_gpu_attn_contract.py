"""The attention operators where include/attn.h promises something that random
inputs do not show: infinite keys, rows that add nothing, slots without a position."""
import numpy as np
import pytest
import torch

from attn_helpers import Batch, f64, trees
from block_scaled_fp4_softmax_gb300 import attn
from test_gpu_attn import BF, FP, attend

pytestmark = pytest.mark.gpu


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
