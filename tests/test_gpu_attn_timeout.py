"""The bounded waits of the attention kernels run out cleanly.

A test hook shortens every wait to 200 us and makes one barrier of each kernel expect an
arrival that never comes (the one that announces a tile's weights, the one that frees a
buffer of scores), with products and copies in flight behind and before it.  Each role of a
CTA then gives up, the launch ends by itself, sets MOE_DEV_TIMEOUT and writes NaN, and the
next call is right.  Nothing here traps, faults or waits without a limit."""
import pytest
import torch

from attn_helpers import Batch, trees
from block_scaled_fp4_softmax_gb300 import attn, moe
from test_gpu_attn import BF, FP, attend

pytestmark = pytest.mark.gpu


def timed_out(call):
    moe.moe_test_set_wait_limit(200_000, 1)
    try:
        out = call()
        torch.cuda.synchronize()
    finally:
        moe.moe_test_set_wait_limit(0, 0)
    return out


@pytest.mark.parametrize("dtype,dim,group,lens,new,tree", [
    (BF, 128, 4, [40], [1], False),               # one tile
    (BF, 128, 4, [9000, 300], [2, 1], False),     # divided units, two streams of keys
    (FP, 64, 8, [4000, 70, 0], [30, 40, 5], True),  # two streams of rows
    (BF, 256, 8, [3000, 5], [20, 1], True),       # one stream
])
def test_tree_decode(dtype, dim, group, lens, new, tree):
    bt = Batch(dtype, lens, new, 2, group, dim, 16, True, trees(new, 5) if tree else None, seed=dim)
    want, want_lse = attend(bt)
    assert int(bt.status) == 0
    out, lse = timed_out(lambda: attend(bt))
    assert int(bt.status) == attn.DEV_TIMEOUT
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    bt.status.zero_()
    out, lse = attend(bt)
    assert int(bt.status) == 0
    assert torch.equal(out.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("dtype,dim,group,lens,new", [
    (BF, 64, 8, [3000, 40], [64, 40]),
    (FP, 128, 16, [200, 900, 0], [20, 30, 17]),
    (BF, 256, 8, [1500], [40]),
])
def test_cache_weights(dtype, dim, group, lens, new):
    """More than 256 rows, or passes of several tiles: every CTA comes to use a buffer again."""
    bt = Batch(dtype, lens, new, 2, group, dim, 16, True, trees(new, 5), seed=dim)
    _, lse = attend(bt)
    acc = torch.rand(bt.B, 2, bt.cap, device="cuda")

    def weigh():
        return attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, tree=bt.tree, dev_status=bt.status)

    want = weigh()
    assert int(bt.status) == 0
    out = timed_out(weigh)
    assert int(bt.status) == attn.DEV_TIMEOUT
    for b in range(bt.B):
        n = lens[b] + new[b]
        assert torch.isnan(out[b, :, :n]).all() and torch.equal(out[b, :, n:], want[b, :, n:])
    bt.status.zero_()
    assert torch.equal(weigh(), want) and int(bt.status) == 0
