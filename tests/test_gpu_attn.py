"""The attention operators over a paged cache against the float64 oracle."""
import numpy as np
import pytest
import torch

from attn_helpers import Batch, f64, trees
from block_scaled_fp4_softmax_gb300 import attn
from oracle import attn as A

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def check_attention(bt, out, lse):
    """Every element within: one rounding of the result, one rounding of each
    weight (relative, so at most half a step of sum p |v|), and FP32 sums: a
    score off by d changes its weight by a factor exp(d)."""
    want, want_lse, mag = bt.expected_attention()
    got, got_lse = f64(out), f64(lse)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), empty)
    assert np.all(got[empty] == 0)
    u = half_step(bt.dtype)
    d = bt.dim * 2.0 ** -23 * bt.dot_bound() + 2.0 ** -20
    tol = u * np.abs(want) + (u + 4 * d) * mag + torch.finfo(bt.dtype).tiny
    bad = np.abs(got - want) > tol
    assert not bad.any(), (int(bad.sum()), float(np.abs(got - want).max()), np.argwhere(bad)[:4].tolist())
    diff = np.abs(got_lse[~empty] - want_lse[~empty])
    assert np.all(diff <= d + 2.0 ** -22 * np.abs(want_lse[~empty])), float(diff.max())


def attend(bt, **kw):
    out = torch.full((bt.T, bt.q_heads, bt.dim), 7.0, dtype=bt.dtype, device="cuda")
    lse = torch.full((bt.T, bt.q_heads), 7.0, device="cuda")
    attn.attn_tree_decode(bt.q, bt.cu, bt.lens, bt.cache, tree=bt.tree, out=out, lse=lse, dev_status=bt.status, **kw)
    torch.cuda.synchronize()
    return out, lse


# lengths around a tile of keys, groups that fill rows unevenly, pages that end
# inside a tile or span several, every class of head dim
TREE_CASES = [
    # dtype, lens, new, kv_heads, group, dim, page, heads_first, tree, pad
    (BF, [0], [1], 1, 1, 128, 16, True, False, 0),
    (BF, [1], [1], 2, 4, 128, 16, True, False, 0),
    (FP, [126, 127, 128, 129, 0], [1, 1, 1, 1, 1], 2, 5, 128, 16, False, False, 0),
    (BF, [255, 64, 63, 65], [1, 2, 0, 3], 1, 16, 64, 64, True, False, 0),
    (BF, [300, 0, 17], [33, 7, 64], 2, 3, 128, 32, False, True, 0),
    (FP, [511, 512, 513], [5, 63, 1], 1, 8, 96, 24, True, True, 8),
    (BF, [40], [200], 1, 3, 80, 8, True, True, 0),
    (BF, [0, 5], [130, 65], 2, 2, 72, 16, True, False, 0),
    (FP, [700, 64], [17, 2], 2, 8, 256, 128, True, True, 0),
    (BF, [1000, 3], [1, 70], 1, 7, 160, 256, False, False, 0),
    (BF, [90], [4], 1, 2, 16, 40, True, True, 0),
    (FP, [333], [40], 3, 20, 64, 48, True, True, 0),
    (FP, [2000], [1], 1, 1, 248, 2048, True, False, 0),
]


@pytest.mark.parametrize("case", TREE_CASES, ids=[str(i) for i in range(len(TREE_CASES))])
def test_tree_decode(case):
    dtype, lens, new, hk, g, dim, page, hf, tree, pad = case
    bt = Batch(dtype, lens, new, hk, g, dim, page, hf, trees(new, 5) if tree else None, seed=len(lens) + dim, pad=pad)
    out, lse = attend(bt)
    assert int(bt.status) == 0
    check_attention(bt, out, lse)


def test_tree_decode_many_splits():
    """One long sequence spread over the whole GPU, next to many short ones."""
    bt = Batch(BF, [30000] + [3] * 40, [1] + [2] * 40, 2, 4, 128, 64, seed=3)
    out, lse = attend(bt)
    check_attention(bt, out, lse)
    again, lse2 = attend(bt)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_tree_rows_that_see_nothing(dtype):
    """Blind drafts see the committed slots only, and nothing at all where there are none."""
    new = [6, 5, 1]
    bt = Batch(dtype, [0, 130, 0], new, 2, 4, 128, 16, True, trees(new, 2, blind=(0, 4)), seed=9)
    out, lse = attend(bt)
    check_attention(bt, out, lse)
    assert torch.isneginf(lse[0]).all() and torch.isneginf(lse[11]).all()


def test_tree_words_narrower_than_the_drafts():
    """Missing words of a tree row are zero."""
    new = [100]
    full = trees(new, 4)
    bt = Batch(BF, [50], new, 1, 2, 64, 16, True, np.ascontiguousarray(full[:, :1]), seed=4)
    out, lse = attend(bt)
    check_attention(bt, out, lse)


@pytest.mark.parametrize("dim,dtype", [(128, BF), (64, FP), (256, BF)])
def test_unseen_drafts_do_not_leak(dim, dtype):
    """NaN and infinities in keys and values of drafts reach exactly the tokens that see them."""
    new = [20, 9]
    clean = Batch(dtype, [117, 128], new, 2, 4, dim, 16, True, trees(new, 8), seed=6)
    want, want_lse = attend(clean)
    dirty = Batch(dtype, [117, 128], new, 2, 4, dim, 16, True, trees(new, 8), seed=6)
    page, row = dirty.rows(0)
    bad_v, bad_k = 7, 12
    dirty.v[page[117 + bad_v], 0, row[117 + bad_v]] = float("inf")
    dirty.v[page[117 + bad_v], 0, row[117 + bad_v], 3] = float("nan")
    dirty.k[page[117 + bad_k], 1, row[117 + bad_k]] = float("nan")
    out, lse = attend(dirty)
    assert int(dirty.status) == 0
    masks = dirty.masks(0)
    for i in range(20):
        sees_v, sees_k = masks[i][117 + bad_v], masks[i][117 + bad_k]
        o, w = out[i].float(), want[i].float()
        if sees_v:
            assert torch.isinf(o[:4, :3]).all() and torch.isnan(o[:4, 3]).all()
        else:
            assert torch.equal(o[:4], w[:4])
        assert torch.equal(lse[i, :4], want_lse[i, :4])
        if sees_k:
            assert torch.isnan(o[4:]).all() and torch.isnan(lse[i, 4:]).all()
        else:
            assert torch.equal(o[4:], w[4:]) and torch.equal(lse[i, 4:], want_lse[i, 4:])
    assert torch.equal(out[20:].view(torch.int16), want[20:].view(torch.int16))


@pytest.mark.parametrize("dim,scale", [(128, -0.11), (64, -1e-3), (256, 0.5)])
def test_other_scales(dim, scale):
    bt = Batch(BF, [300, 5], [3, 40], 2, 4, dim, 16, seed=17, sharp=0.7)
    bt.scale = scale
    out, lse = attend(bt, scale=scale)
    bt.scale = abs(scale)  # the bound of a score is that of its size
    bound = bt.dot_bound()
    bt.scale, bt.dot_bound = scale, lambda: bound
    check_attention(bt, out, lse)
    acc = torch.zeros(2, 2, bt.cap, device="cuda")
    got = f64(attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, scale=scale))
    want = bt.expected_weights(f64(lse), f64(acc), 1.0)
    there = ~np.isnan(want)
    tol = (4 * (dim * 2.0 ** -23 * bound + 2.0 ** -18) + 160 * 2.0 ** -24) * want + 2.0 ** -40
    assert np.all(np.abs(got - want)[there] <= tol[there])


def test_cache_with_heads_outermost():
    """[kv_heads, pages, page_size, D]: the pages lie closer together than the heads."""
    bt = Batch(FP, [130, 33], [2, 5], 3, 2, 64, 16, seed=18)
    want = attend(bt)
    k, v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (bt.k, bt.v))
    assert k.stride(0) < k.stride(1)
    cache = attn.attn_cache(k, v, bt.table)
    got = attn.attn_tree_decode(bt.q, bt.cu, bt.lens, cache)
    assert torch.equal(want[0].view(torch.int16), got[0].view(torch.int16)) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_large_scores(dtype):
    """Scores in the hundreds, and rows whose later keys are far above the first ones."""
    bt = Batch(dtype, [400], [3], 1, 4, 64, 16, seed=12, sharp=40.0)
    bt.k[:] = bt.k * torch.linspace(0.2, 3.0, bt.page, device="cuda").to(dtype)[:, None]
    out, lse = attend(bt)
    want, want_lse, mag = bt.expected_attention()
    d = bt.dim * 2.0 ** -23 * bt.dot_bound() + 2.0 ** -18
    assert np.all(np.abs(f64(out) - want) <= half_step(dtype) * (np.abs(want) + mag) + 4 * d * mag)
    assert np.all(np.abs(f64(lse) - want_lse) <= d + 2.0 ** -22 * np.abs(want_lse))


def test_rare_weights_of_half_precision_count():
    """One key far above 4000 equal ones: their small weights add up to a visible share."""
    bt = Batch(FP, [4001], [1], 1, 1, 64, 32, seed=13)
    bt.q[:] = 1.0
    bt.k[:] = 0.0
    page, row = bt.rows(0)
    bt.k[page[5], 0, row[5]] = 1.5  # score 12: the others weigh e^-12 each
    bt.v[:] = 1.0
    bt.v[page[5], 0, row[5]] = 0.0
    out, lse = attend(bt)
    check_attention(bt, out, lse)
    assert 0.015 < float(out[0, 0, 0]) < 0.03


def test_far_page_offsets():
    """Pages whose element offsets pass 32 bits."""
    pages, page, hk, dim = 132000, 64, 4, 64  # 2.16e9 elements per tensor
    k = torch.empty(pages, hk, page, dim, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    bt = Batch(BF, [150, 70], [3, 1], hk, 2, dim, page, seed=15)
    far = np.array([[pages - 1, 131100, pages - 2], [131072, 5, 0]], dtype=np.int32)
    table = torch.from_numpy(far).cuda()
    for b in range(2):
        for p in range(-(-(bt.len_list[b] + bt.new_list[b]) // page)):
            k[far[b, p]], v[far[b, p]] = bt.k[bt.table_np[b, p]], bt.v[bt.table_np[b, p]]
    want = attend(bt)
    cache = attn.attn_cache(k, v, table)
    got = attn.attn_tree_decode(bt.q, bt.cu, bt.lens, cache)
    assert torch.equal(want[0].view(torch.int16), got[0].view(torch.int16)) and torch.equal(want[1], got[1])
    acc = torch.rand(2, hk, 160, device="cuda")
    w1 = attn.attn_cache_weights(bt.q, want[1], bt.cu, bt.lens, bt.cache, acc)
    w2 = attn.attn_cache_weights(bt.q, want[1], bt.cu, bt.lens, cache, acc)
    assert torch.equal(w1, w2)
    pos = torch.arange(160, device="cuda", dtype=torch.int32).expand(2, hk, 160).contiguous()
    freq = torch.ones(8, dtype=torch.float64, device="cuda")
    tp = torch.arange(4, dtype=torch.int32, device="cuda")
    for c in (bt.cache, cache):
        attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, tp, bt.cu, bt.lens, c, freq)
    total = bt.lens + (bt.cu[1:] - bt.cu[:-1])
    for c in (bt.cache, cache):
        attn.attn_cache_evict(c, acc, pos, total, total, 64, sinks=2, recent=5)
    for b in range(2):
        for p in range(-(-(bt.len_list[b] + bt.new_list[b]) // page)):
            n = min(page, bt.len_list[b] + bt.new_list[b] - p * page)
            assert torch.equal(k[far[b, p], :, :n], bt.k[bt.table_np[b, p], :, :n])
            assert torch.equal(v[far[b, p], :, :n], bt.v[bt.table_np[b, p], :, :n])


# ---------------------------------------------------------------------------
# Weights
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("case", TREE_CASES, ids=[str(i) for i in range(len(TREE_CASES))])
def test_cache_weights(case):
    dtype, lens, new, hk, g, dim, page, hf, tree, pad = case
    bt = Batch(dtype, lens, new, hk, g, dim, page, hf, trees(new, 5, blind=(2,)) if tree else None,
               seed=len(lens) + dim, pad=pad)
    _, lse = attend(bt)
    acc = torch.rand(bt.B, hk, bt.cap, device="cuda")
    out = torch.full_like(acc, 5.0)
    attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, tree=bt.tree, decay=0.875, acc_out=out,
                            dev_status=bt.status)
    assert int(bt.status) == 0
    want = bt.expected_weights(f64(lse), f64(acc), 0.875)
    got = f64(out)
    beyond = np.isnan(want)
    assert np.all(got[beyond] == 5.0)
    # a score off by d changes its weight by a factor exp(d); FP32 sums of n rows
    d = bt.dim * 2.0 ** -23 * bt.dot_bound() + 2.0 ** -18
    n = max(1, max(new)) * g
    tol = (4 * d + n * 2.0 ** -24) * np.abs(want) + 2.0 ** -40
    assert np.all(np.abs(got - want)[~beyond] <= tol[~beyond]), float(np.nanmax(np.abs(got - want)))
    same = acc.clone()
    attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, same, tree=bt.tree, decay=0.875, acc_out=same)
    assert np.array_equal(f64(same)[~beyond], got[~beyond])


def test_cache_weights_without_tokens():
    bt = Batch(BF, [37, 5], [0, 0], 2, 2, 64, 16)
    acc = torch.rand(2, 2, bt.cap, device="cuda")
    out = attn.attn_cache_weights(bt.q, torch.empty(0, 4, device="cuda"), bt.cu, bt.lens, bt.cache, acc, decay=0.5)
    assert torch.equal(out[0, :, :37], acc[0, :, :37] * 0.5) and torch.equal(out[1, :, :5], acc[1, :, :5] * 0.5)
    assert torch.count_nonzero(out[1, :, 5:]) == 0
    o, lse = attn.attn_tree_decode(bt.q, bt.cu, bt.lens, bt.cache)
    assert o.shape[0] == 0 and lse.shape[0] == 0


def test_weights_of_a_token_sum_to_one_per_query_head():
    bt = Batch(FP, [777, 1], [1, 1], 2, 6, 128, 32, seed=21)
    _, lse = attend(bt)
    acc = torch.zeros(2, 2, bt.cap, device="cuda")
    out = attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc)
    assert np.allclose(f64(out).sum(-1), 6.0, rtol=2.0 ** -14)


# ---------------------------------------------------------------------------
# Norm, rotation, append
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim,rot,inter,norm,hk,g,page,hf", [
    (BF, 128, 128, False, True, 4, 4, 16, True),
    (FP, 128, 64, True, True, 2, 5, 24, False),
    (BF, 72, 72, False, True, 1, 3, 8, True),      # pairs 36 apart: not a multiple of 8
    (FP, 96, 24, False, False, 3, 1, 16, True),    # pairs 12 apart
    (BF, 256, 0, False, True, 2, 2, 64, True),
    (FP, 16, 16, True, True, 2, 1, 16, False),
    (BF, 24, 6, False, True, 1, 17, 16, True),
    (BF, 160, 80, False, True, 2, 3, 16, True),
    (FP, 256, 256, True, False, 1, 1, 16, True),
])
def test_qk_norm_rope(dtype, dim, rot, inter, norm, hk, g, page, hf):
    lens, new = [40, 0, 3, 7], [3, 5, 0, 1]
    bt = Batch(dtype, lens, new, hk, g, dim, page, hf, seed=rot + dim)
    gen = torch.Generator(device="cuda").manual_seed(1)
    wq, wk = (torch.randn(dim, generator=gen, device="cuda").to(dtype) for _ in range(2))
    pos = torch.tensor([40, 41, 41, 0, 1, 2, 2, 3, 1999999999], dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).cuda()
    slot_pos = torch.full((4, hk, bt.cap), -1, dtype=torch.int32, device="cuda")
    k0, v0 = f64(bt.k), f64(bt.v)
    mag = 1.25
    q = attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq,
                               q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-5,
                               interleaved=inter, magnitude=mag, slot_pos=slot_pos, dev_status=bt.status)
    torch.cuda.synchronize()
    assert int(bt.status) == 0
    u = half_step(dtype)

    def near(got, x, w):
        want = A.head_rows(f64(x), f64(w) if norm else None, 1e-5, pos.cpu().numpy(), freq.cpu().numpy(), inter, mag)
        # one rounding, and FP32 arithmetic on the two channels of a pair: each within the row's largest value
        big = np.abs(want).max(-1, keepdims=True) * 2
        tol = u * np.abs(want) + 2.0 ** -18 * big + torch.finfo(dtype).tiny
        assert np.all(np.abs(got - want) <= tol), float(np.abs(got - want).max())

    near(f64(q), bt.q, wq)
    k1, v1 = f64(bt.k), f64(bt.v)
    got_k = np.zeros((bt.T, hk, dim))
    for b in range(4):
        page_i, row_i = bt.rows(b)
        for i in range(new[b]):
            t, s = bt.cu_list[b] + i, lens[b] + i
            got_k[t] = k1[page_i[s], :, row_i[s]]
            assert np.array_equal(v1[page_i[s], :, row_i[s]], f64(bt.v_new)[t])
            assert (slot_pos[b, :, s] == pos[t]).all()
            k1[page_i[s], :, row_i[s]], v1[page_i[s], :, row_i[s]] = k0[page_i[s], :, row_i[s]], v0[page_i[s], :, row_i[s]]
    near(got_k, bt.k_new, wk)
    assert np.array_equal(k0, k1, equal_nan=True) and np.array_equal(v0, v1, equal_nan=True)
    assert int((slot_pos >= 0).sum()) == bt.T * hk


def test_rope_in_place_and_negative_positions():
    bt = Batch(BF, [4], [6], 1, 2, 64, 16, seed=31)
    pos = torch.tensor([-5, -1, 0, 1, 5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).cuda()
    q = bt.q.contiguous()
    want = attn.attn_qk_norm_rope(q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq)
    ref = A.head_rows(f64(q), None, 0.0, pos.cpu().numpy(), freq.cpu().numpy(), False, 1.0)
    assert np.all(np.abs(f64(want) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -18 * np.abs(ref).max() * 2)
    attn.attn_qk_norm_rope(q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq, q_out=q)
    assert torch.equal(q, want)


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------

def run_evict(bt, acc, pos, lens, nxt, budget, sinks, recent):
    k0, v0 = f64(bt.k), f64(bt.v)
    a, p = acc.cpu().numpy(), pos.cpu().numpy()
    acc_out, pos_out = torch.full_like(acc, -3.0), torch.full_like(pos, -3)
    lens_out, _, _ = attn.attn_cache_evict(bt.cache, acc, pos, bt.lens, nxt, budget, sinks, recent, acc_out=acc_out,
                                           pos_out=pos_out, dev_status=bt.status)
    torch.cuda.synchronize()
    assert int(bt.status) == 0
    assert lens_out.tolist() == [min(n, budget) for n in lens]
    want_k, want_v = k0.copy(), v0.copy()
    want_a, want_p = np.full(a.shape, -3.0, np.float32), np.full(p.shape, -3, np.int32)
    for b, n in enumerate(lens):
        page, row = bt.rows(b)
        for h in range(bt.kv_heads):
            take, moves = A.evict(a[b, h, :n], p[b, h, :n], budget, sinks, recent, int(nxt[b]))
            m = len(take)
            want_a[b, h, :m], want_p[b, h, :m] = a[b, h, take], p[b, h, take]
            for s, d in moves:
                want_k[page[d], h, row[d]], want_v[page[d], h, row[d]] = k0[page[s], h, row[s]], v0[page[s], h, row[s]]
    assert np.array_equal(acc_out.cpu().numpy(), want_a, equal_nan=True)
    assert np.array_equal(pos_out.cpu().numpy(), want_p)
    assert np.array_equal(f64(bt.k), want_k, equal_nan=True) and np.array_equal(f64(bt.v), want_v, equal_nan=True)


@pytest.mark.parametrize("lens,hk,dim,page,hf,budget,sinks,recent,dtype", [
    ([100, 64, 65, 0, 1], 2, 64, 16, True, 64, 0, 0, BF),
    ([3000, 2049, 5000], 3, 128, 24, False, 2048, 4, 100, FP),
    ([33], 1, 16, 8, True, 1, 0, 0, BF),
    ([40], 1, 24, 8, True, 39, 0, 0, BF),
    ([1500], 2, 256, 64, True, 700, 50, 900, BF),   # more protected slots than the budget holds
    ([20000], 1, 72, 256, True, 9999, 4, 4000, FP),
    ([70000], 1, 16, 1024, True, 30001, 4, 100, FP),
])
def test_evict(lens, hk, dim, page, hf, budget, sinks, recent, dtype):
    bt = Batch(dtype, lens, [0] * len(lens), hk, 1, dim, page, hf, seed=budget)
    g = torch.Generator(device="cuda").manual_seed(budget)
    acc = torch.randn(bt.B, hk, bt.cap, generator=g, device="cuda").exp()
    acc[acc < 0.6] = 0.0                                  # many ties
    pos = torch.rand(bt.B, hk, bt.cap, generator=g, device="cuda").argsort(dim=-1).to(torch.int32)
    run_evict(bt, acc, pos, lens, torch.tensor([bt.cap] * bt.B, dtype=torch.int32, device="cuda"), budget, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "special"])
def test_evict_ties_and_special_weights(kind):
    n = 4100
    bt = Batch(BF, [n], [0], 2, 1, 32, 16, seed=40)
    acc = torch.full((1, 2, bt.cap), 0.25, device="cuda")
    if kind == "special":
        vals = torch.tensor([0.0, -0.0, float("nan"), float("inf"), -float("inf"), 1e-42, -1.0, 3.0, -float("nan")], device="cuda")
        acc = vals[torch.randint(0, len(vals), acc.shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")]
    pos = torch.arange(bt.cap, dtype=torch.int32, device="cuda").flip(0).expand(1, 2, -1).contiguous()
    run_evict(bt, acc, pos, [n], torch.tensor([n], dtype=torch.int32, device="cuda"), 2500, 3, 10)


def test_evict_more_keys_than_shared_memory_holds():
    n = 420000
    bt = Batch(BF, [n], [0], 1, 1, 16, 4096, seed=41)
    acc = torch.rand(1, 1, bt.cap, device="cuda").mul_(1000).round_()
    pos = torch.arange(bt.cap, dtype=torch.int32, device="cuda").expand(1, 1, -1).contiguous()
    run_evict(bt, acc, pos, [n], torch.tensor([n], dtype=torch.int32, device="cuda"), 200001, 4, 77)


# ---------------------------------------------------------------------------
# Errors that only the device can see
# ---------------------------------------------------------------------------

def test_bad_page_is_flagged_and_poisons_its_sequence():
    bt = Batch(BF, [200, 90], [2, 2], 2, 3, 128, 16, seed=50)
    want, _ = attend(bt)
    lse = torch.zeros(bt.T, bt.q_heads, device="cuda")
    acc = torch.rand(2, 2, bt.cap, device="cuda")
    good = attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc)
    for number in (-1, bt.k.shape[0], 2 ** 31 - 1):
        bt.status.zero_()
        bt.table[0, 3] = number
        out, got_lse = attend(bt)
        assert int(bt.status) == attn.DEV_BAD_PAGE
        assert torch.isnan(out[:2]).all() and torch.isnan(got_lse[:2]).all()
        assert torch.equal(out[2:], want[2:])
        bt.status.zero_()
        w = attn.attn_cache_weights(bt.q, lse, bt.cu, bt.lens, bt.cache, acc, dev_status=bt.status)
        assert int(bt.status) == attn.DEV_BAD_PAGE
        assert torch.isnan(w[0, :, 48:64]).all() and torch.equal(w[0, :, :48], good[0, :, :48])
        assert torch.equal(w[0, :, 64:], good[0, :, 64:]) and torch.equal(w[1], good[1])
    bt.table[0, 12] = -1  # the page of the tokens in flight
    bt.table[0, 3] = bt.table_np[0, 3]
    bt.status.zero_()
    k0 = bt.k.clone()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    freq = torch.ones(64, dtype=torch.float64, device="cuda")
    attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq, dev_status=bt.status)
    assert int(bt.status) == attn.DEV_BAD_PAGE
    page, row = bt.rows(1)
    for i in (90, 91):
        k0[page[i], :, row[i]] = bt.k[page[i], :, row[i]]
    assert torch.equal(k0.nan_to_num(), bt.k.nan_to_num())
    bt.status.zero_()
    k0 = bt.k.clone()
    slot_pos = torch.zeros(2, 2, bt.cap, dtype=torch.int32, device="cuda")
    acc = torch.zeros(2, 2, bt.cap, device="cuda")
    acc[0, :, 192:] = 1.0  # the bad page's rows are the ones to move
    lens_out, acc_out, _ = attn.attn_cache_evict(bt.cache, acc, slot_pos, bt.lens, bt.lens, 100, 0, 0, dev_status=bt.status)
    assert int(bt.status) == attn.DEV_BAD_PAGE
    assert int(torch.isnan(acc_out).sum()) == 16 and torch.equal(k0.nan_to_num(), bt.k.nan_to_num())


@pytest.mark.parametrize("what", ["negative", "too_long", "descending", "beyond"])
def test_bad_lengths_are_flagged(what):
    bt = Batch(BF, [200, 90], [2, 2], 2, 3, 128, 16, seed=51)
    lens, cu = bt.lens.clone(), bt.cu.clone()
    if what == "negative":
        lens[1] = -1
    elif what == "too_long":
        lens[1] = bt.table.shape[1] * bt.page - 1
    elif what == "descending":
        cu[1] = 5
    else:
        cu[2] = 99
    k0, v0 = bt.k.clone(), bt.v.clone()
    out, lse = attn.attn_tree_decode(bt.q, cu, lens, bt.cache, dev_status=bt.status)
    assert int(bt.status) == attn.DEV_BAD_LENGTH and torch.isnan(out[2:]).all() and torch.isnan(lse[2:]).all()
    bt.status.zero_()
    acc = torch.rand(2, 2, bt.cap, device="cuda")
    w = attn.attn_cache_weights(bt.q, torch.zeros_like(lse), cu, lens, bt.cache, acc, dev_status=bt.status)
    assert int(bt.status) == attn.DEV_BAD_LENGTH and torch.isnan(w[1]).all()
    bt.status.zero_()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    q = attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, pos, cu, lens, bt.cache,
                               torch.ones(64, dtype=torch.float64, device="cuda"), dev_status=bt.status)
    assert int(bt.status) == attn.DEV_BAD_LENGTH and torch.isnan(q[2:]).all()
    page, row = bt.rows(0)
    for i in (200, 201):
        bt.k[page[i], :, row[i]], bt.v[page[i], :, row[i]] = k0[page[i], :, row[i]], v0[page[i], :, row[i]]
    assert torch.equal(k0.nan_to_num(), bt.k.nan_to_num()) and torch.equal(v0.nan_to_num(), bt.v.nan_to_num())
    bt.status.zero_()
    if what in ("negative", "too_long"):
        slot_pos = torch.zeros(2, 2, bt.cap, dtype=torch.int32, device="cuda")
        lens_out, a, _ = attn.attn_cache_evict(bt.cache, acc, slot_pos, lens, lens, 50, dev_status=bt.status)
        assert int(bt.status) == attn.DEV_BAD_LENGTH
        assert what == "negative" or torch.isnan(a[1, :, :50]).all()
        assert int(lens_out[1]) == (0 if what == "negative" else 50)


# ---------------------------------------------------------------------------
# Streams, graphs, the step as a whole
# ---------------------------------------------------------------------------

def step(bt, pos, freq, slot_pos, acc, stream=None):
    q = attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, pos, bt.cu, bt.lens, bt.cache, freq, slot_pos=slot_pos,
                               stream=stream)
    out, lse = attn.attn_tree_decode(q, bt.cu, bt.lens, bt.cache, tree=bt.tree, stream=stream)
    acc1 = attn.attn_cache_weights(q, lse, bt.cu, bt.lens, bt.cache, acc, tree=bt.tree, stream=stream)
    total = bt.lens + (bt.cu[1:] - bt.cu[:-1]) if stream is None else bt.total
    return (out, lse, acc1) + attn.attn_cache_evict(bt.cache, acc1, slot_pos, total, total, 150, 4, 20, stream=stream)


def test_other_stream_and_graph_replay():
    def fresh():
        new = [9, 4, 1]
        bt = Batch(BF, [300, 120, 149], new, 2, 4, 128, 16, True, trees(new, 3), seed=60)
        bt.total = bt.lens + (bt.cu[1:] - bt.cu[:-1])
        pos = torch.arange(14, dtype=torch.int32, device="cuda") + 300
        freq = (10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128)).cuda()
        g = torch.Generator(device="cuda").manual_seed(2)
        acc = torch.rand(3, 2, bt.cap, generator=g, device="cuda")
        slot_pos = torch.arange(bt.cap, dtype=torch.int32, device="cuda").expand(3, 2, -1).contiguous()
        torch.cuda.synchronize()
        return bt, (bt, pos, freq, slot_pos, acc)

    bt, args = fresh()
    want = [t.clone() for t in step(*args)] + [bt.k.clone(), bt.v.clone()]
    bt, args = fresh()
    s = torch.cuda.Stream()
    got = step(*args, stream=s)
    s.synchronize()
    for w, x in zip(want, list(got) + [bt.k, bt.v]):
        assert torch.equal(w.nan_to_num(), x.nan_to_num())
    bt, args = fresh()
    k0, v0 = bt.k.clone(), bt.v.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*args)
    for _ in range(2):
        bt.k.copy_(k0)
        bt.v.copy_(v0)
        g.replay()
        torch.cuda.synchronize()
        for w, x in zip(want, list(got) + [bt.k, bt.v]):
            assert torch.equal(w.nan_to_num(), x.nan_to_num())


def test_attention_does_not_depend_on_slot_order_after_eviction():
    """A decode over the evicted cache equals attention over exactly the kept keys."""
    bt = Batch(FP, [500], [1], 1, 4, 128, 16, seed=70)
    acc = torch.rand(1, 1, bt.cap, device="cuda")
    pos = torch.arange(bt.cap, dtype=torch.int32, device="cuda").expand(1, 1, -1).contiguous()
    k0, v0 = f64(bt.k), f64(bt.v)
    page, row = bt.rows(0)
    take, _ = A.evict(acc[0, 0, :500].cpu().numpy(), pos[0, 0, :500].cpu().numpy(), 200, 4, 32, 500)
    lens, _, pos1 = attn.attn_cache_evict(bt.cache, acc, pos, bt.lens, bt.lens, 200, 4, 32)
    assert sorted(pos1[0, 0, :200].tolist()) == sorted(take.tolist())
    freq = torch.zeros(0, dtype=torch.float64, device="cuda")
    attn.attn_qk_norm_rope(bt.q, bt.k_new, bt.v_new, torch.tensor([500], dtype=torch.int32, device="cuda"), bt.cu, lens,
                           bt.cache, freq)
    out, _ = attn.attn_tree_decode(bt.q, bt.cu, lens, bt.cache)
    kk = np.concatenate([k0[page[take], 0, row[take]], f64(bt.k_new)[:, 0]])
    vv = np.concatenate([v0[page[take], 0, row[take]], f64(bt.v_new)[:, 0]])
    for h in range(4):
        want, _, mag = A.attend(f64(bt.q)[0, h], kk, vv, np.ones(201, dtype=bool), bt.scale)
        assert np.all(np.abs(f64(out)[0, h] - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -10 * mag)
