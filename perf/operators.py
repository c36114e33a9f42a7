"""Performance cases of the attention operators over a paged cache.

Four operators make up the attention step of a speculative decode:

  rope     attn_qk_norm_rope   head norms and position rotation, append to the cache
  tree     attn_tree_decode    attention of the tokens in flight over the cache
  weights  attn_cache_weights  accumulates the softmax weight every cached slot received
  evict    attn_cache_evict    keeps the slots with the most weight, moves rows into the holes

A case is a dict of plain values.  ``run`` computes it with elementary torch
operations in FP32 (FP64 for rotation angles), or, when ``own`` is set, with
one call of the library, as a serving loop makes it.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one sequence: the latency of a plain decode step
        dict(name="rope_token", op="rope", type="bf16", batch=1, drafts=1, length=700, ragged=False, q_heads=16,
             kv_heads=4, dim=128, page=16, heads_first=True, rot=128, interleaved=False, stretch=1.0),
        # trees of a batch, part of the head rotated, positions far beyond FP32's reach
        dict(name="rope_drafts", op="rope", type="fp16", batch=24, drafts=33, length=900, ragged=True, q_heads=20,
             kv_heads=4, dim=96, page=24, heads_first=False, rot=48, interleaved=True, stretch=8.0),
        # prompts entering the cache
        dict(name="rope_prompt", op="rope", type="bf16", batch=5, drafts=2451, length=0, ragged=False, q_heads=32,
             kv_heads=8, dim=128, page=64, heads_first=True, rot=128, interleaved=False, stretch=4.0),
        # one token over a short cache: latency
        dict(name="tree_token", op="tree", type="bf16", batch=1, drafts=1, length=1000, ragged=False, q_heads=16,
             kv_heads=4, dim=128, page=16, heads_first=True, tree=False),
        # single tokens of a ragged batch: the cache's bytes are the time
        dict(name="tree_batch", op="tree", type="bf16", batch=32, drafts=1, length=8192, ragged=True, q_heads=32,
             kv_heads=4, dim=128, page=64, heads_first=True, tree=False),
        # trees of 63 drafts: as much matrix work as bytes
        dict(name="tree_drafts", op="tree", type="bf16", batch=8, drafts=63, length=16384, ragged=False, q_heads=32,
             kv_heads=4, dim=128, page=32, heads_first=False, tree=True),
        # one sequence with a very long cache and wide heads
        dict(name="tree_long", op="tree", type="fp16", batch=1, drafts=17, length=300001, ragged=False, q_heads=16,
             kv_heads=2, dim=256, page=128, heads_first=True, tree=True),
        # the weights of one token's step over short caches: latency
        dict(name="weights_token", op="weights", type="fp16", batch=2, drafts=1, length=1500, ragged=True, q_heads=20,
             kv_heads=4, dim=80, page=16, heads_first=False, tree=False),
        # the weights of a batch of trees
        dict(name="weights_drafts", op="weights", type="bf16", batch=8, drafts=63, length=16384, ragged=False,
             q_heads=32, kv_heads=4, dim=128, page=32, heads_first=False, tree=True),
        # one sequence a little over its budget: latency
        dict(name="evict_one", op="evict", type="bf16", batch=1, length=2500, ragged=False, kv_heads=4, dim=128,
             page=16, heads_first=True, budget=2048),
        # a batch cut to half its length
        dict(name="evict_batch", op="evict", type="bf16", batch=16, length=16384, ragged=True, kv_heads=8, dim=128,
             page=64, heads_first=True, budget=6144),
        # few sequences, very long: little parallelism across heads
        dict(name="evict_long", op="evict", type="fp16", batch=2, length=200003, ragged=False, kv_heads=2, dim=64,
             page=128, heads_first=False, budget=131072),
    ]


def _spread(rng, low, high):
    """An integer from low to high, even in its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    def one(op):
        c = dict(op=op, type=rng.choice(["bf16", "fp16"]), ragged=rng.random() < 0.6, kv_heads=_spread(rng, 1, 8),
                 dim=rng.choice([64, 72, 80, 96, 128, 128, 160, 256]), page=rng.choice([8, 16, 24, 32, 64, 128, 256]),
                 heads_first=rng.random() < 0.5)
        if op == "evict":
            c.update(batch=_spread(rng, 1, 32), length=_spread(rng, 40, 200000))
            c["budget"] = max(1, int(c["length"] * rng.uniform(0.3, 0.95)))
            return c
        c["q_heads"] = c["kv_heads"] * _spread(rng, 1, 16)
        if op == "rope":
            c.update(batch=_spread(rng, 1, 32), drafts=_spread(rng, 1, 2500), length=_spread(rng, 1, 1000),
                     rot=c["dim"] // rng.choice([1, 2, 4]) // 2 * 2, interleaved=rng.random() < 0.5,
                     stretch=rng.choice([1.0, 4.0, 8.0]))
        else:
            c.update(batch=_spread(rng, 1, 64), drafts=_spread(rng, 1, 100), length=_spread(rng, 1, 300000),
                     tree=rng.random() < 0.6)
        return c

    def fits(c):
        top = [work(k) for k in listed() if k["op"] == c["op"]]
        w = work(c)
        slots = c["batch"] * (c["length"] + c.get("drafts", 0))
        plain = 4 * slots * (c["kv_heads"] * c["dim"] * 2 + c.get("q_heads", 0) * (c["drafts"] if "tree" in c else 0))
        return (w["bytes"] <= max(t["bytes"] for t in top) and w["flops"] <= max(t["flops"] for t in top)
                and plain <= 6e9)

    op = rng.choice(["rope", "tree", "tree", "weights", "evict"])
    c = one(op)
    while not fits(c):
        c = one(op)
    return c


def _sizes(case):
    """Committed length and tokens in flight of each sequence, from the case alone."""
    B, L, N = case["batch"], case["length"], case.get("drafts", 0)
    if not case["ragged"]:
        return [L] * B, [N] * B
    rng = random.Random(1000003 * B + 1009 * L + N)
    lens = [rng.randint(L // 8, L) for _ in range(B)]
    new = [rng.randint((N + 3) // 4, N) for _ in range(B)]
    if B > 2:  # a sequence that starts empty, and one with nothing in flight
        lens[1], new[2] = 0, 0
    return lens, new


def work(case):
    lens, new = _sizes(case)
    hk, d, e = case["kv_heads"], case["dim"], 2
    if case["op"] == "evict":
        k = case["budget"]
        moved = sum(k * (n - k) / n for n in lens if n > k)
        kept = sum(min(k, n) for n in lens)
        return {"bytes": hk * (8 * sum(lens) + 8 * kept + moved * 4 * d * e), "flops": 0}
    hq, t = case["q_heads"], sum(new)
    if case["op"] == "rope":
        row = (hq + 2 * hk) * d * e
        return {"bytes": 2 * t * row + 4 * t * (1 + hk), "flops": 8 * t * (hq + hk) * d}
    slots = sum(n + m for n, m in zip(lens, new) if m)
    pairs = sum((n + m) * m for n, m in zip(lens, new))
    if case["op"] == "tree":
        return {"bytes": 2 * slots * hk * d * e + 2 * t * hq * d * e + 4 * t * hq, "flops": 4 * pairs * hq * d}
    return {"bytes": slots * hk * (d * e + 8) + t * hq * (d * e + 4), "flops": 2 * pairs * hq * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _pages(case, slots, gen):
    """A cache whose physical pages are shuffled; the page table [B, max pages]."""
    size, hk, d = case["page"], case["kv_heads"], case["dim"]
    counts = [-(-s // size) for s in slots]
    total, most = max(1, sum(counts)), max(1, max(counts))
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    ends = torch.tensor(counts, device="cuda").cumsum(0)
    at = torch.arange(most, device="cuda")[None, :]
    begin = (ends - torch.tensor(counts, device="cuda"))[:, None]
    table = torch.where(at < (ends[:, None] - begin), order[(begin + at).clamp(max=total - 1)], 0)
    shape = (total, hk, size, d) if case["heads_first"] else (total, size, hk, d)
    both = []
    for _ in range(2):
        x = torch.empty(shape, dtype=TYPES[case["type"]], device="cuda").normal_(generator=gen)
        both.append(x if case["heads_first"] else x.transpose(1, 2))
    return both[0], both[1], table.to(torch.int32).contiguous()


def _inv_freq(rot, stretch):
    """Radians per position of each pair, in FP64; `stretch` slows the pairs
    that turn less than once in 4096 positions, for longer contexts."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    turns = 4096 * f / (2 * math.pi)
    return torch.where(turns < 1, f / stretch, f).cuda()


def prepare(case, seed):
    def tree_words(new, gen, width):
        """Ancestor bits of random draft trees, 63 or fewer bits used of each int64 word: [T, words] int64.
        The last of several drafts is padding that sees no draft at all."""
        rows = []
        for n in new:
            parent = [int(v * i) - 1 if i else -1 for i, v in enumerate(torch.rand(n, generator=gen).tolist())]
            seen = []
            for i in range(n):
                seen.append((seen[parent[i]] if parent[i] >= 0 else 0) | (1 << i))
            if n > 2:
                seen[n - 1] = 0
            rows += seen
        words = [[(m >> (64 * w)) & ((1 << 64) - 1) for w in range(width)] for m in rows]
        signed = [[v - (1 << 64) if v >> 63 else v for v in row] for row in words]
        return torch.tensor(signed, dtype=torch.int64).reshape(len(rows), width)

    lens, new = _sizes(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    dt = TYPES[case["type"]]
    B, hk, d = case["batch"], case["kv_heads"], case["dim"]
    t = sum(new)
    s = {"case": case, "keep": {}}
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor([0] + torch.tensor(new).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    s["k_cache"], s["v_cache"], s["table"] = _pages(case, [n + m for n, m in zip(lens, new)], gen)
    cap = max(8, -(-max(n + m for n, m in zip(lens, new)) // 8) * 8)
    if case["op"] == "evict":
        # positions in the order that earlier evictions left, weights with a
        # long tail, and slots that never received any (ties)
        acc = torch.empty(B, hk, cap, device="cuda").normal_(generator=gen).mul_(2).exp_()
        s["acc"] = torch.where(acc < 0.2, torch.zeros_like(acc), acc)
        s["pos"] = torch.rand(B, hk, cap, generator=gen, device="cuda").masked_fill_(
            torch.arange(cap, device="cuda") >= s["lens"][:, None, None], 2.0).argsort(dim=-1).argsort(dim=-1).to(torch.int32)
        s["next_pos"] = s["lens"].clone()
        s["sinks"], s["recent"] = 4, max(1, case["budget"] // 8)
        s["acc_out"], s["pos_out"] = torch.zeros_like(s["acc"]), torch.zeros_like(s["pos"])
        return s
    hq = case["q_heads"]
    qkv = torch.empty(t, (hq + 2 * hk) * d, dtype=dt, device="cuda").normal_(generator=gen)
    if case["op"] == "rope":
        qkv = qkv.mul_(3)
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hk) * d].view(t, hk, d)
        s["v"] = qkv[:, (hq + hk) * d:].view(t, hk, d)
        s["q_weight"] = torch.empty(d, dtype=dt, device="cuda").normal_(1.0, 0.1, generator=gen)
        s["k_weight"] = torch.empty(d, dtype=dt, device="cuda").normal_(1.0, 0.1, generator=gen)
        s["inv_freq"] = _inv_freq(case["rot"], case["stretch"])
        s["magnitude"] = 1.0 + 0.1 * math.log(case["stretch"])
        begin = torch.randint(0, int(200000 * case["stretch"]), (B,), generator=cpu)
        s["pos"] = torch.cat([torch.arange(m) // 2 + b for m, b in zip(new, begin.tolist())]).to(torch.int32).cuda()
        s["slot_pos"] = torch.zeros(B, hk, cap, dtype=torch.int32, device="cuda")
        return s
    s["q"] = qkv[:, :hq * d].reshape(t, hq, d).mul_(2)
    s["scale"] = d ** -0.5
    s["tree"] = None
    if case["tree"]:
        s["tree"] = tree_words(new, cpu, max(1, -(-max(new) // 64))).cuda()
    if case["op"] == "weights":
        # what the attention step left: the log of each row's sum (its mean
        # for normal keys), and the weights accumulated before
        total = torch.cat([torch.full((m,), math.log(max(1, n + m))) for n, m in zip(lens, new)]).cuda()
        s["lse"] = (total[:, None] + s["q"].float().square().sum(-1) * (0.5 * s["scale"] ** 2)).contiguous()
        s["acc"] = torch.empty(B, hk, cap, device="cuda").exponential_(generator=gen)
        s["acc_out"] = torch.zeros_like(s["acc"])
        s["decay"] = 0.9375
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from block_scaled_fp4_softmax_gb300 import attn

    keep, op = s["keep"], s["case"]["op"]
    if not keep:  # what a serving loop makes once: the cache's handle and the workspaces
        keep["cache"] = attn.attn_cache(s["k_cache"], s["v_cache"], s["table"])
        if op == "tree":
            keep["ws"] = attn.attn_tree_decode_workspace(keep["cache"])
        if op == "evict":
            keep["ws"] = attn.attn_cache_evict_workspace(keep["cache"], s["case"]["budget"])
    cache = keep["cache"]
    if op == "rope":
        q = attn.attn_qk_norm_rope(s["q"], s["k"], s["v"], s["pos"], s["cu"], s["lens"], cache, s["inv_freq"],
                                   q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                                   interleaved=s["case"]["interleaved"], magnitude=s["magnitude"],
                                   slot_pos=s["slot_pos"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], "slot_pos": s["slot_pos"]}
    if op == "tree":
        out, lse = attn.attn_tree_decode(s["q"], s["cu"], s["lens"], cache, tree=s["tree"], scale=s["scale"],
                                         workspace=keep["ws"])
        return {"out": out, "lse": lse}
    if op == "weights":
        return attn.attn_cache_weights(s["q"], s["lse"], s["cu"], s["lens"], cache, s["acc"], tree=s["tree"],
                                       scale=s["scale"], decay=s["decay"], acc_out=s["acc_out"])
    lens, acc, pos = attn.attn_cache_evict(cache, s["acc"], s["pos"], s["lens"], s["next_pos"], s["case"]["budget"],
                                           sinks=s["sinks"], recent=s["recent"], acc_out=s["acc_out"],
                                           pos_out=s["pos_out"], workspace=keep["ws"])
    return {"lens": lens, "acc": acc, "pos": pos, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain(s):
    return {"rope": _plain_rope, "tree": _plain_tree, "weights": _plain_weights, "evict": _plain_evict}[
        s["case"]["op"]](s)


def _owners(s):
    """Sequence and index in it of every token in flight."""
    t = torch.arange(s["q"].shape[0], dtype=torch.int32, device="cuda")
    b = torch.searchsorted(s["cu"], t, right=True) - 1
    return b, (t - s["cu"][b]).long()


def _rotated(x, w, s, angle):
    """Head norm, weight and rotation of x [T, heads, D] in FP32."""
    c = s["case"]
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    cos, sin = (f(angle).mul(s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        p = head.unflatten(-1, (-1, 2))
        a, b = p[..., 0], p[..., 1]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = head.chunk(2, -1)
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((head, rest), -1)


def _plain_rope(s):
    size, dt = s["case"]["page"], s["q"].dtype
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    b, i = _owners(s)
    slot = s["lens"].long()[b] + i
    page, row = s["table"].long()[b, slot // size], slot % size
    s["k_cache"][page, :, row] = _rotated(s["k"], s["k_weight"], s, angle).to(dt)
    s["v_cache"][page, :, row] = s["v"]
    s["slot_pos"][b, :, slot] = s["pos"][:, None]
    return {"q": _rotated(s["q"], s["q_weight"], s, angle).to(dt), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"], "slot_pos": s["slot_pos"]}


def _dense(x, table):
    """Every sequence's slots in order, FP32: [B, Hkv, S, D]."""
    return x[table.long()].float().transpose(1, 2).flatten(2, 3)


def _scores(s, slots):
    """Scores [B, Hkv, G, N, S] of the padded tokens, and which keys they see."""
    c = s["case"]
    b, i = _owners(s)
    n = c["drafts"]
    q = torch.zeros(c["batch"], n, c["q_heads"], c["dim"], device="cuda")
    q[b, i] = s["q"].float()
    q = q.unflatten(2, (c["kv_heads"], -1)).permute(0, 2, 3, 1, 4)
    k = _dense(s["k_cache"], s["table"])
    scores = (q.flatten(2, 3) @ k.transpose(-1, -2)).unflatten(2, (-1, n)) * s["scale"]
    at = torch.arange(slots, device="cuda")
    draft = at - s["lens"].long()[:, None]  # [B, S]: index among the sequence's drafts
    new = (s["cu"][1:] - s["cu"][:-1]).long()[:, None]
    row = torch.arange(n, device="cuda")[:, None]
    if s["tree"] is None:
        sees = draft[:, None] <= row
    else:
        words = torch.zeros(c["batch"], n, s["tree"].shape[1], dtype=torch.int64, device="cuda")
        words[b, i] = s["tree"]
        d = draft.clamp(0, 64 * s["tree"].shape[1] - 1)
        picked = words.gather(2, (d // 64)[:, None].expand(-1, n, -1))
        sees = ((picked >> (d % 64)[:, None]) & 1).bool() | (draft < 0)[:, None]
    return scores, (sees & (draft < new)[:, None])[:, None, None], b, i


def _plain_tree(s):
    c = s["case"]
    slots = s["table"].shape[1] * c["page"]
    scores, sees, b, i = _scores(s, slots)
    scores = scores.masked_fill_(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(top.masked_fill(top == -math.inf, 0.0)))
    total = p.sum(-1, keepdim=True)
    v = _dense(s["v_cache"], s["table"])
    out = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / total.masked_fill(total == 0, 1.0)
    lse = (top + total.log()).squeeze(-1)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i]
    return {"out": out.to(s["q"].dtype), "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[b, i]}


def _plain_weights(s):
    c = s["case"]
    slots = s["table"].shape[1] * c["page"]
    scores, sees, b, i = _scores(s, slots)
    lse = torch.full((c["batch"], c["drafts"], c["q_heads"]), math.inf, device="cuda")
    lse[b, i] = s["lse"]
    lse = lse.unflatten(2, (c["kv_heads"], -1)).permute(0, 2, 3, 1)
    w = torch.exp(scores.sub_(lse[..., None])).masked_fill_(~sees, 0.0).sum((2, 3))
    cap = s["acc"].shape[2]
    w = torch.nn.functional.pad(w, (0, max(0, cap - slots)))[..., :cap]
    at = torch.arange(cap, device="cuda")
    lens, new = s["lens"][:, None, None], (s["cu"][1:] - s["cu"][:-1])[:, None, None]
    total = s["acc"].masked_fill(at >= lens, 0.0) * s["decay"] + w
    s["acc_out"].copy_(torch.where(at < lens + new, total, s["acc_out"]))
    return s["acc_out"]


def _plain_evict(s):
    c = s["case"]
    k, size = c["budget"], c["page"]
    cap = s["acc"].shape[2]
    at = torch.arange(cap, device="cuda")
    lens = s["lens"].long()[:, None, None]
    held = (s["pos"] < s["sinks"]) | (s["pos"] >= s["next_pos"][:, None, None] - s["recent"])
    key = s["acc"].masked_fill(held, math.inf).masked_fill(at >= lens, -math.inf)
    order = key.argsort(dim=-1, descending=True, stable=True)
    kept = torch.zeros_like(held).scatter_(2, order[..., :k], True) & (at < lens)
    over = (lens > k).expand_as(kept)
    mover, hole = kept & (at >= k) & over, ~kept & (at < k) & over
    b, h, src = mover.nonzero(as_tuple=True)
    _, _, dst = hole.nonzero(as_tuple=True)
    table = s["table"].long()
    source, target = (table[b, src // size], h, src % size), (table[b, dst // size], h, dst % size)
    s["k_cache"][target] = s["k_cache"][source]
    s["v_cache"][target] = s["v_cache"][source]
    lens_out = s["lens"].clamp(max=k)
    stays = at < lens_out[:, None, None]
    s["acc_out"].copy_(torch.where(stays, s["acc"], s["acc_out"]))
    s["pos_out"].copy_(torch.where(stays, s["pos"], s["pos_out"]))
    s["acc_out"][b, h, dst] = s["acc"][b, h, src]
    s["pos_out"][b, h, dst] = s["pos"][b, h, src]
    return {"lens": lens_out, "acc": s["acc_out"], "pos": s["pos_out"], "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


# ---------------------------------------------------------------------------
# The definitions in FP64, sequence by sequence
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    g = case.get("q_heads", 0) // case["kv_heads"]

    def sequences():
        """Of each sequence: its index, committed length, token range and the cache rows of its slots."""
        lens, cu, size = s["lens"].tolist(), s["cu"].tolist(), case["page"]
        for b in range(len(lens)):
            at = torch.arange(lens[b] + cu[b + 1] - cu[b], device="cuda")
            yield b, lens[b], cu[b], cu[b + 1], (s["table"][b].long()[at // size], at % size)

    def rope():
        rot = case["rot"]
        first = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
        second = first + (1 if case["interleaved"] else rot // 2)
        turn = torch.polar(torch.tensor(s["magnitude"], dtype=torch.float64, device="cuda"),
                           torch.outer(s["pos"].double(), s["inv_freq"]))[:, None]

        def head(x, w):
            x = x.double()
            x = x / (x.square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt() * w.double()
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q, k = head(s["q"], s["q_weight"]), head(s["k"], s["k_weight"])
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        for _, n, lo, hi, (page, row) in sequences():
            for h in range(case["kv_heads"]):
                k_cache[page[n:], h, row[n:]] = k[lo:hi, h]
                v_cache[page[n:], h, row[n:]] = s["v"][lo:hi, h].double()
        return {"q": q, "k_cache": k_cache, "v_cache": v_cache, "slot_pos": None}

    def visible(n, lo, hi):
        """[tokens, slots] truth values of one sequence, bit by bit."""
        m = hi - lo
        sees = torch.ones(m, n + m, dtype=torch.bool)
        if s["tree"] is None:
            sees[:, n:] = torch.ones(m, m).tril().bool()
        else:
            words = s["tree"][lo:hi].tolist()
            sees[:, n:] = torch.tensor([[bool(w[j // 64] >> (j % 64) & 1) for j in range(m)] for w in words]).reshape(m, m)
        return sees.cuda()

    def scores(h, lo, hi, rows):
        """Scores [G, tokens, slots] of one sequence and KV head in FP64."""
        k = s["k_cache"][rows[0], h, rows[1]].double()
        return torch.einsum("tgd,sd->gts", s["q"][lo:hi, h * g:(h + 1) * g].double(), k) * s["scale"]

    def tree():
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for _, n, lo, hi, rows in sequences():
            if lo == hi:
                continue
            sees = visible(n, lo, hi)
            for h in range(case["kv_heads"]):
                x = scores(h, lo, hi, rows).masked_fill(~sees, -math.inf)
                total = torch.logsumexp(x, -1)
                p = torch.exp(x - total.masked_fill(total == -math.inf, 0.0)[..., None])
                out[lo:hi, h * g:(h + 1) * g] = torch.einsum("gts,sd->tgd", p, s["v_cache"][rows[0], h, rows[1]].double())
                lse[lo:hi, h * g:(h + 1) * g] = total.T
        return {"out": out, "lse": lse}

    def weights():
        acc = s["acc_out"].double()
        for b, n, lo, hi, rows in sequences():
            sees = visible(n, lo, hi)
            acc[b, :, :n] = s["acc"][b, :, :n].double() * s["decay"]
            acc[b, :, n:n + hi - lo] = 0
            for h in range(case["kv_heads"] if hi > lo else 0):
                x = scores(h, lo, hi, rows) - s["lse"][lo:hi, h * g:(h + 1) * g].double().T[..., None]
                acc[b, h, :n + hi - lo] += torch.exp(x).masked_fill(~sees, 0.0).sum((0, 1))
        return acc

    def evict():
        acc, pos = s["acc_out"].clone(), s["pos_out"].clone()
        k_cache, v_cache, table = s["k_cache"].double(), s["v_cache"].double(), s["table"].cpu().numpy()
        lens = s["lens"].tolist()
        for b in range(len(lens)):
            n, most = lens[b], min(lens[b], case["budget"])
            for h in range(case["kv_heads"]):
                w, at = s["acc"][b, h, :n].cpu().numpy(), s["pos"][b, h, :n].cpu().numpy()
                held = (at < s["sinks"]) | (at >= int(s["next_pos"][b]) - s["recent"])
                order = np.lexsort((np.arange(n), -w, ~held))
                stays = np.zeros(n, dtype=bool)
                stays[order[:most]] = True
                take = np.arange(most)
                take[~stays[:most]] = most + np.flatnonzero(stays[most:])
                take_on = torch.from_numpy(take).cuda()
                acc[b, h, :most], pos[b, h, :most] = s["acc"][b, h, take_on], s["pos"][b, h, take_on]
                to = np.flatnonzero(~stays[:most])
                spot = [torch.from_numpy(x).long().cuda() for x in (
                    table[b, take[to] // case["page"]], take[to] % case["page"], table[b, to // case["page"]],
                    to % case["page"])]
                k_cache[spot[2], h, spot[3]] = k_cache[spot[0], h, spot[1]]
                v_cache[spot[2], h, spot[3]] = v_cache[spot[0], h, spot[1]]
        return {"lens": s["lens"].clamp(max=case["budget"]), "acc": acc.double(), "pos": pos, "k_cache": k_cache,
                "v_cache": v_cache}

    return {"rope": rope, "tree": tree, "weights": weights, "evict": evict}[case["op"]]()
