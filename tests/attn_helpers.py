"""A small batch over a paged cache on the device, and what the oracle needs of it."""
import numpy as np
import torch

from block_scaled_fp4_softmax_gb300 import attn
from oracle import attn as A


def f64(t):
    return t.detach().double().cpu().numpy()


def trees(new, seed, words=None, blind=()):
    """Random ancestor rows [T, words] uint64; drafts listed in `blind` (by
    index in their sequence) see no draft, themselves included."""
    rng = np.random.default_rng(seed)
    words = words or max(1, -(-max(new) // 64))
    rows = []
    for n in new:
        seen = []
        for i in range(n):
            p = int(rng.integers(-1, i)) if i else -1
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        for i in blind:
            if i < n:
                seen[i] = 0
        rows += seen
    out = np.zeros((len(rows), words), dtype=np.uint64)
    for r, m in enumerate(rows):
        for w in range(words):
            out[r, w] = (m >> (64 * w)) & 0xFFFFFFFFFFFFFFFF
    return out


class Batch:
    def __init__(self, dtype, lens, new, kv_heads, group, dim, page=16, heads_first=True, tree=None, seed=0, pad=0,
                 spare=3, sharp=1.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.dtype, self.kv_heads, self.group, self.dim, self.page = dtype, kv_heads, group, dim, page
        self.len_list, self.new_list = list(lens), list(new)
        self.B, self.T, self.q_heads = len(lens), sum(new), kv_heads * group
        counts = [-(-(n + m) // page) for n, m in zip(lens, new)]
        pages = sum(counts) + spare
        order = rng.permutation(pages)
        most = max(1, max(counts))
        table = np.full((self.B, most), -7, dtype=np.int32)  # entries past the end are never looked at
        at = 0
        for b, c in enumerate(counts):
            table[b, :c] = order[at:at + c]
            at += c
        self.table_np = table
        self.table = torch.from_numpy(table).cuda()
        shape = (pages, kv_heads, page, dim + pad) if heads_first else (pages, page, kv_heads, dim + pad)

        def cache():
            x = torch.randn(shape, generator=g, device="cuda").to(dtype)[..., :dim]
            return x if heads_first else x.transpose(1, 2)

        self.k, self.v = cache(), cache()
        # slots past the end hold what earlier sequences or nobody left there
        for b in range(self.B):
            for s in range(lens[b] + new[b], counts[b] * page):
                p, r = table[b, s // page], s % page
                self.k[p, :, r], self.v[p, :, r] = float("nan"), float("inf") if s % 2 else float("nan")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.cu_list = [0] + np.cumsum(new).tolist()
        self.cu = torch.tensor(self.cu_list, dtype=torch.int32, device="cuda")
        self.qkv = torch.randn(self.T, (self.q_heads + 2 * kv_heads) * dim + 8, generator=g, device="cuda").mul_(sharp).to(dtype)
        hd = self.q_heads * dim
        self.q = self.qkv[:, :hd].view(self.T, self.q_heads, dim)
        self.k_new = self.qkv[:, hd:hd + kv_heads * dim].view(self.T, kv_heads, dim)
        self.v_new = self.qkv[:, hd + kv_heads * dim:hd + 2 * kv_heads * dim].view(self.T, kv_heads, dim)
        self.tree_np = tree
        self.tree = None if tree is None else torch.from_numpy(tree.view(np.int64)).cuda()
        self.cache = attn.attn_cache(self.k, self.v, self.table)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = dim ** -0.5
        self.cap = max(8, max(n + m for n, m in zip(lens, new)))

    def rows(self, b):
        return A.slot_rows(self.table_np[b], self.page, np.arange(self.len_list[b] + self.new_list[b]))

    def masks(self, b):
        lo, hi = self.cu_list[b], self.cu_list[b + 1]
        words = None if self.tree_np is None else self.tree_np[lo:hi]
        return [A.sees(words, self.len_list[b], i, hi - lo) for i in range(hi - lo)]

    def expected_attention(self):
        """out, lse, and per element the sum of p |v|."""
        out, mag = np.zeros((2, self.T, self.q_heads, self.dim))
        lse = np.zeros((self.T, self.q_heads))
        q, k, v = f64(self.q), f64(self.k), f64(self.v)
        for b in range(self.B):
            page, row = self.rows(b)
            masks = self.masks(b)
            for h in range(self.kv_heads):
                kk, vv = k[page, h, row], v[page, h, row]
                for i, m in enumerate(masks):
                    for g in range(self.group):
                        t, hq = self.cu_list[b] + i, h * self.group + g
                        out[t, hq], lse[t, hq], mag[t, hq] = A.attend(q[t, hq], kk, vv, m, self.scale)
        return out, lse, mag

    def dot_bound(self):
        """Largest sum |q_d k_d| * scale of any row: FP32 sums of D products are off by at most D 2^-23 of it
        (each of the D additions by half a unit, or a whole one where the hardware truncates)."""
        q, k = np.abs(f64(self.q)), np.abs(f64(self.k))
        k = np.where(np.isfinite(k), k, 0.0)
        return float(q.max(axis=(0, 1)) @ k.max(axis=(0, 1, 2))) * self.scale

    def expected_weights(self, lse, acc, decay):
        out = np.full((self.B, self.kv_heads, self.cap), np.nan)
        q, k = f64(self.q), f64(self.k)
        for b in range(self.B):
            n, m = self.len_list[b], self.new_list[b]
            page, row = self.rows(b)
            masks = self.masks(b)
            for h in range(self.kv_heads):
                out[b, h, :n] = acc[b, h, :n] * decay
                out[b, h, n:n + m] = 0
                lo = self.cu_list[b]
                hs = slice(h * self.group, (h + 1) * self.group)
                for i in range(m):
                    out[b, h, :n + m] += A.received(q[lo + i, hs], lse[lo + i, hs], k[page, h, row],
                                                    [masks[i]] * self.group, self.scale)
        return out
