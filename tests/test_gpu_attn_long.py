"""The attention operators over long caches: pieces of many tiles, units of several
row groups, slices that shared memory does not hold."""
import pytest
import torch

from attn_helpers import Batch, trees
from block_scaled_fp4_softmax_gb300 import attn
from test_gpu_attn import BF, FP, attend, half_step, run_evict

pytestmark = pytest.mark.gpu


def heads(bt):
    """Sequence, KV head, its rows (tokens, query heads), keys, values and what each row
    sees, in float64 on the device."""
    q, words = bt.q.double(), bt.tree_np
    for b in range(bt.B):
        n, m, lo = bt.len_list[b], bt.new_list[b], bt.cu_list[b]
        slots = torch.arange(n + m, device="cuda")
        page, row = bt.table[b].long()[slots // bt.page], slots % bt.page
        see = torch.ones(m, n + m, dtype=torch.bool)
        for i in range(m):
            for j in range(m):
                see[i, n + j] = j <= i if words is None else bool((int(words[lo + i, j // 64]) >> (j % 64)) & 1)
        see = see.cuda()[:, None].expand(m, bt.group, n + m).reshape(m * bt.group, n + m)
        for h in range(bt.kv_heads):
            hs = slice(h * bt.group, (h + 1) * bt.group)
            yield (b, h, slice(lo, lo + m), hs, q[lo:lo + m, hs].reshape(m * bt.group, bt.dim), bt.k[page, h, row].double(),
                   bt.v[page, h, row].double(), see)


CASES = {
    # both streams on the same rows; some 17 tiles a part
    "single": (BF, [20011], [1], 16, 8, 128, 64, False),
    "single_64": (FP, [30000, 777], [3, 1], 8, 4, 64, 48, False),
    # the streams are the halves of the rows
    "halves": (BF, [12345], [25], 12, 8, 128, 32, True),
    "halves_64": (FP, [9999, 0, 4000], [40, 50, 0], 8, 4, 64, 16, False),
    # two and three row groups, beside sequences of one
    "groups": (BF, [3000, 9000, 127, 500], [33, 70, 1, 20], 4, 8, 128, 128, True),
    "groups_wide": (FP, [7001, 100], [40, 9], 3, 8, 256, 64, True),
    "groups_160": (BF, [5000], [50], 2, 5, 160, 24, False),
    # more rows than the weights' kernel holds at once
    "passes": (FP, [2500, 300], [150, 3], 2, 8, 64, 16, True),
    "passes_wide": (BF, [2222], [90], 1, 7, 232, 40, False),
}


@pytest.mark.parametrize("name", CASES)
def test_long_caches(name):
    """As for short ones; on top, the FP32 sums of n keys: the tensor core adds 16 at a
    time, each addition off by at most 2^-23, and l is a sum of n / 64 terms a thread at
    least, each off by 2^-24."""
    dtype, lens, new, hk, g, dim, page, tree = CASES[name]
    bt = Batch(dtype, lens, new, hk, g, dim, page, True, trees(new, 5) if tree else None, seed=dim + len(name))
    out, lse = attend(bt)
    acc = torch.rand(bt.B, hk, bt.cap, device="cuda")
    weights = torch.full_like(acc, 5.0)
    attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, tree=bt.tree, decay=0.875, acc_out=weights,
                            dev_status=bt.status)
    assert int(bt.status) == 0
    q = bt.q.double().abs().amax((0, 1))
    k = torch.where(torch.isfinite(bt.k), bt.k, 0).abs().amax((0, 1, 2)).double()
    d = bt.dim * 2.0 ** -23 * float(q @ k) * bt.scale + 2.0 ** -18
    u = half_step(dtype)
    for b, h, ts, hs, qq, kk, vv, see in heads(bt):
        if not len(qq):
            continue
        n = kk.shape[0]
        sums = n / 16 * 2.0 ** -23 + n / 64 * 2.0 ** -24
        s = (qq @ kk.T * bt.scale).masked_fill(~see, -float("inf"))
        want_lse = torch.logsumexp(s, -1)
        p = torch.exp(s - want_lse[:, None])
        want, mag = p @ vv, p @ vv.abs()
        got = out[ts, hs].double().reshape(want.shape)
        tol = u * want.abs() + (u + 4 * d + sums) * mag + torch.finfo(dtype).tiny
        assert ((got - want).abs() <= tol).all(), (b, h, float((got - want).abs().max()))
        got_lse = lse[ts, hs].double().reshape(-1)
        assert ((got_lse - want_lse).abs() <= d + sums + 2.0 ** -22 * want_lse.abs()).all(), (b, h)
        # from the lse that the kernel was given
        received = torch.exp(s - got_lse[:, None]).sum(0)
        received[:lens[b]] += 0.875 * acc[b, h, :lens[b]].double()
        got_w = weights[b, h, :n].double()
        tol = (4 * d + len(qq) * 2.0 ** -24) * received + 2.0 ** -40
        assert ((got_w - received).abs() <= tol).all(), (b, h, float((got_w - received).abs().max()))
        assert (weights[b, h, n:] == 5.0).all()
    again, lse2 = attend(bt)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("long", [46000, 46001])
def test_evict_many_heads_whose_keys_do_not_fit(long):
    """More (sequence, head) pairs than SMs, each with a CTA of its own, and more slots
    than its shared memory holds; rows of acc and slot_pos on 16 bytes, or not."""
    lens = [long, 50, 45999] + [7] * 17
    bt = Batch(BF, lens, [0] * 20, 8, 1, 16, 1024, seed=long)
    assert bt.cap == long
    g = torch.Generator(device="cuda").manual_seed(long)
    acc = torch.rand(20, 8, bt.cap, generator=g, device="cuda").mul_(300).round_()
    pos = torch.arange(bt.cap, dtype=torch.int32, device="cuda").expand(20, 8, -1).contiguous()
    run_evict(bt, acc, pos, lens, torch.tensor(lens, dtype=torch.int32, device="cuda"), 20011, 4, 77)


def test_evict_a_cluster_whose_keys_do_not_fit():
    n = 725003
    bt = Batch(FP, [n], [0], 1, 1, 16, 4096, seed=2)
    acc = torch.rand(1, 1, bt.cap, device="cuda").mul_(1000).round_()
    pos = torch.arange(bt.cap, dtype=torch.int32, device="cuda").expand(1, 1, -1).contiguous()
    run_evict(bt, acc, pos, [n], torch.tensor([n], dtype=torch.int32, device="cuda"), 400001, 4, 77)
