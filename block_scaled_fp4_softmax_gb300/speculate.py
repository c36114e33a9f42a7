"""Example: greedy speculative decoding with trees of drafts over bounded caches.

A small decoder with random weights whose layers are the attention step of
:mod:`.attn` followed by the routed experts of :mod:`.moe`.  Each step puts the
last token and a tree of drafts of every sequence in flight:

  * ``attn_qk_norm_rope`` appends their keys and values behind the cache,
  * ``attn_tree_decode`` lets each see the cache and its own ancestors,
  * the drafts that the logits confirm are appended again, as a chain over the
    tree's slots, and ``attn_cache_weights`` adds up what they looked at,
  * ``attn_cache_evict`` shrinks caches that have outgrown their budget.

Run it with ``python -m block_scaled_fp4_softmax_gb300.speculate``.
"""

from __future__ import annotations

import argparse
import dataclasses

import torch

from . import attn, moe, synth


@dataclasses.dataclass
class Config:
    layers: int = 2
    vocab: int = 512
    hidden: int = 256
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    inter: int = 128
    experts: int = 16
    top_k: int = 4
    page: int = 16
    budget: int = 96     # slots a sequence is shrunk to ...
    slack: int = 32      # ... once it has so many more
    sinks: int = 4
    recent: int = 16
    most: int = 64       # tokens in flight of a sequence; a tree's ancestors are one 64-bit word
    decay: float = 0.95
    eps: float = 1e-6
    base: float = 10000.0


# ---------------------------------------------------------------------------
# Host side: drafts and their verification
# ---------------------------------------------------------------------------

def lookup(history, depth=4, width=3):
    """Drafts that followed earlier occurrences of the last token, the latest
    occurrences first, as a tree (tokens, parents); node 0 is the last token
    itself, and a parent comes before its children."""
    tokens, parents, children = [history[-1]], [-1], {}
    found = 0
    for i in range(len(history) - 2, -1, -1):
        if history[i] != history[-1]:
            continue
        at = 0
        for t in history[i + 1:i + 1 + depth]:
            if (at, t) not in children:
                children[at, t] = len(tokens)
                tokens.append(t)
                parents.append(at)
            at = children[at, t]
        found += 1
        if found == width:
            break
    return tokens, parents


def ancestors(parents):
    """Ancestor bits and depth of each node, the node itself included."""
    bits, depth = [], []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        depth.append(depth[p] + 1 if p >= 0 else 0)
    return bits, depth


def accept(tokens, parents, follow):
    """The path from the root that the model would have taken (follow[i]: the
    token it puts after node i), and the token behind its end."""
    path = [0]
    while True:
        want = follow[path[-1]]
        step = [i for i, p in enumerate(parents) if p == path[-1] and tokens[i] == want]
        if not step:
            return path, want
        path.append(step[0])


# ---------------------------------------------------------------------------
# Device side
# ---------------------------------------------------------------------------

class Layer:
    def __init__(self, cfg: Config, batch: int, seed: int, device):
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).to(torch.bfloat16)

        heads = cfg.q_heads + 2 * cfg.kv_heads
        self.qkv = weights(heads * cfg.head_dim, cfg.hidden, std=cfg.hidden ** -0.5)
        self.out = weights(cfg.hidden, cfg.q_heads * cfg.head_dim, std=(cfg.q_heads * cfg.head_dim) ** -0.5)
        self.q_norm, self.k_norm = (1 + weights(cfg.head_dim, std=0.1) for _ in range(2))
        self.router = synth.router_weights(cfg.experts, cfg.hidden, seed + 1, device=device)
        self.shape = moe.shape(cfg.hidden, cfg.inter, moe.FMT_NVFP4)
        self.records = [moe.fp4_pack_expert(*synth.expert_weights(cfg.hidden, cfg.inter, seed + 2 + e, device=device, std=0.05),
                                            self.shape) for e in range(cfg.experts)]
        self.experts = moe.pointer_table(self.records)
        # pages for a full cache and the tokens in flight, in no particular order
        per = -(-(cfg.budget + cfg.slack + cfg.most) // cfg.page)
        pages = batch * per
        shape = (pages, cfg.kv_heads, cfg.page, cfg.head_dim)
        self.cache = attn.attn_cache(torch.empty(shape, dtype=torch.bfloat16, device=device),
                                     torch.empty(shape, dtype=torch.bfloat16, device=device),
                                     torch.randperm(pages, generator=g, device=device).to(torch.int32).view(batch, per))
        state = (batch, cfg.kv_heads, per * cfg.page)
        self.weight, self.spare_weight = (torch.zeros(state, device=device) for _ in range(2))
        self.slot_pos, self.spare_pos = (torch.zeros(state, dtype=torch.int32, device=device) for _ in range(2))


class Decoder:
    """A batch of sequences; `lens` committed slots and `next_pos` positions each."""

    def __init__(self, cfg: Config, batch: int, seed: int = 0, device="cuda"):
        self.cfg, self.batch, self.device = cfg, batch, torch.device(device)
        g = torch.Generator(device=device).manual_seed(seed)
        self.embed = torch.randn(cfg.vocab, cfg.hidden, generator=g, device=device).to(torch.bfloat16)
        self.layers = [Layer(cfg, batch, seed + 1000 * (i + 1), self.device) for i in range(cfg.layers)]
        half = torch.arange(0, cfg.head_dim, 2, dtype=torch.float64, device=device)
        self.inv_freq = cfg.base ** (-half / cfg.head_dim)
        self.lens, self.next_pos = [0] * batch, [0] * batch
        cache = self.layers[0].cache
        self.tree_ws = attn.attn_tree_decode_workspace(cache)
        self.evict_ws = attn.attn_cache_evict_workspace(cache, cfg.budget)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def _ints(self, x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=self.device)

    def _append(self, layer, qkv, pos, cu, lens):
        cfg = self.cfg
        q, k, v = qkv.view(len(qkv), -1, cfg.head_dim).split([cfg.q_heads, cfg.kv_heads, cfg.kv_heads], dim=1)
        return attn.attn_qk_norm_rope(q, k, v, pos, cu, lens, layer.cache, self.inv_freq, layer.q_norm, layer.k_norm,
                                      cfg.eps, slot_pos=layer.slot_pos, dev_status=self.status)

    def _forward(self, tokens, pos, cu, tree):
        """The tokens in flight through all layers: the last hidden states, and of
        each layer what `_commit` needs of them."""
        cfg, lens = self.cfg, self._ints(self.lens)
        cu, pos = self._ints(cu), self._ints(pos)
        h = self.embed[self._ints(tokens, torch.int64)].float()
        kept = []
        for layer in self.layers:
            qkv = moe.moe_rmsnorm_bf16(h, cfg.eps) @ layer.qkv.T
            q = self._append(layer, qkv, pos, cu, lens)
            out, lse = attn.attn_tree_decode(q, cu, lens, layer.cache, tree, workspace=self.tree_ws,
                                             dev_status=self.status)
            h = h + (out.view(len(tokens), -1) @ layer.out.T).float()
            x, idx, w, _ = moe.moe_rmsnorm_router_topk(h, layer.router, None, cfg.top_k, cfg.eps)
            h = h + moe.moe_experts_decode(x, idx, w, layer.experts, layer.shape, dev_status=self.status)
            kept.append((qkv, lse))
        return h, kept, pos, lens

    def prefill(self, parts):
        """Tokens that are given: parts[b], maybe none, go behind sequence b as a chain."""
        tokens, pos, cu = [], [], [0]
        for b, t in enumerate(parts):
            if len(t) > self.cfg.most:
                raise ValueError(f"sequence {b}: {len(t)} tokens; {self.cfg.most} fit")
            tokens += t
            pos += range(self.next_pos[b], self.next_pos[b] + len(t))
            cu.append(len(tokens))
        _, kept, pos, lens = self._forward(tokens, pos, cu, None)
        self._commit(kept, pos, self._ints(range(len(tokens)), torch.int64), cu, lens)

    def step(self, drafts):
        """One step of every sequence: drafts[b] = (tokens, parents).  Returns the
        accepted tokens behind the root and the next one, and for each of them
        the logits that chose it."""
        cu, tokens, pos, rows = [0], [], [], []
        for b, (t, parents) in enumerate(drafts):
            if not 1 <= len(t) <= min(self.cfg.most, 64) or len(t) != len(parents):
                raise ValueError(f"sequence {b}: {len(t)} tokens and {len(parents)} parents; 1 to {min(self.cfg.most, 64)} fit")
            bits, depth = ancestors(parents)
            tokens += t
            pos += [self.next_pos[b] + d for d in depth]
            rows += [x - (1 << 64) if x >> 63 else x for x in bits]
            cu.append(len(tokens))
        h, kept, pos, lens = self._forward(tokens, pos, cu, self._ints(rows, torch.int64).view(-1, 1))
        logits = (moe.moe_rmsnorm_bf16(h, self.cfg.eps) @ self.embed.T).float()
        follow = logits.argmax(-1).tolist()  # the step's only wait for the device
        took, chosen, cu_new = [], [], [0]
        for b, (t, parents) in enumerate(drafts):
            path, after = accept(t, parents, follow[cu[b]:cu[b + 1]])
            took.append([t[i] for i in path[1:]] + [after])
            chosen += [cu[b] + i for i in path]
            cu_new.append(len(chosen))
        chosen = self._ints(chosen, torch.int64)
        self._commit(kept, pos, chosen, cu_new, lens)
        return took, logits[chosen].split([len(t) for t in took])

    def _commit(self, kept, pos, chosen, cu, lens_dev):
        """The chosen tokens become a chain behind the committed slots."""
        cfg = self.cfg
        cu_dev = self._ints(cu)
        for b in range(self.batch):
            self.lens[b] += cu[b + 1] - cu[b]
            self.next_pos[b] += cu[b + 1] - cu[b]
        full = max(self.lens) >= cfg.budget + cfg.slack
        if full:
            after_dev, next_dev = self._ints(self.lens), self._ints(self.next_pos)
        for layer, (qkv, lse) in zip(self.layers, kept):
            q = self._append(layer, qkv[chosen], pos[chosen], cu_dev, lens_dev)
            attn.attn_cache_weights(q, lse[chosen], cu_dev, lens_dev, layer.cache, layer.weight, decay=cfg.decay,
                                    acc_out=layer.weight, dev_status=self.status)
            if full:
                attn.attn_cache_evict(layer.cache, layer.weight, layer.slot_pos, after_dev, next_dev, cfg.budget,
                                      cfg.sinks, cfg.recent, acc_out=layer.spare_weight, pos_out=layer.spare_pos,
                                      workspace=self.evict_ws, dev_status=self.status)
                layer.weight, layer.spare_weight = layer.spare_weight, layer.weight
                layer.slot_pos, layer.spare_pos = layer.spare_pos, layer.slot_pos
        if full:
            self.lens = [min(n, cfg.budget) for n in self.lens]

    def check(self):
        """Raises if a kernel has reported a bad page, length or an expired wait."""
        code = int(self.status.item())
        if code:
            raise moe.MoeError(f"device status {code}")


def generate(decoder: Decoder, prompts, count: int, draft=lookup):
    """Appends at least `count` tokens to every prompt; draft(history) -> (tokens,
    parents) of the next step, as `lookup` gives them.  Returns the sequences and
    the number of steps."""
    text = [list(p) for p in prompts]
    chunk = decoder.cfg.most
    for at in range(0, max(map(len, prompts)) - 1, chunk):
        decoder.prefill([p[:-1][at:at + chunk] for p in prompts])
    steps = 0
    while min(len(t) - len(p) for t, p in zip(text, prompts)) < count:
        took, _ = decoder.step([draft(t) for t in text])
        for t, new in zip(text, took):
            t += new
        steps += 1
    decoder.check()
    return text, steps


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=200)
    p.add_argument("--batch", type=int, default=4)
    p.add_argument("--seed", type=int, default=0)
    args = p.parse_args()
    cfg = Config()
    g = torch.Generator().manual_seed(args.seed)
    prompts = [torch.randint(cfg.vocab, (5 + 7 * b,), generator=g).tolist() for b in range(args.batch)]
    decoder = Decoder(cfg, args.batch, args.seed)
    text, steps = generate(decoder, prompts, args.tokens)
    for b, (t, prompt) in enumerate(zip(text, prompts)):
        n = len(t) - len(prompt)
        print(f"sequence {b}: {n} tokens in {steps} steps, {n / steps:.2f} a step, {decoder.lens[b]} slots of "
              f"{decoder.next_pos[b]} positions kept")


if __name__ == "__main__":
    main()
