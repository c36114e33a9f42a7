"""Float64 numpy oracle of the attention operators over a paged cache.

Written from the definitions, sequence by sequence and head by head.  Test
infrastructure only: it shares no code with the GPU path."""
import numpy as np


def slot_rows(table_row, page_size, slots):
    """(page, row) of each slot of one sequence."""
    slots = np.asarray(slots)
    return np.asarray(table_row)[slots // page_size], slots % page_size


def head_rows(x, weight, eps, pos, inv_freq, interleaved, magnitude):
    """x [tokens, heads, D] -> head norm, weight and rotation, float64."""
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    rot = 2 * len(inv_freq)
    if rot == 0:
        return x
    j = np.arange(rot // 2)
    first, second = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
    theta = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)
    cos, sin = np.cos(theta)[:, None], np.sin(theta)[:, None]
    a, c = x[..., first], x[..., second]
    out = x.copy()
    out[..., first] = magnitude * (a * cos - c * sin)
    out[..., second] = magnitude * (a * sin + c * cos)
    return out


def sees(tree_rows, length, i, n):
    """Which of the length + n slots draft i sees.  tree_rows: the sequence's
    uint64 words [n, words], or None for a chain."""
    m = np.zeros(length + n, dtype=bool)
    m[:length] = True
    for j in range(n):
        if tree_rows is None:
            m[length + j] = j <= i
        else:
            w = j // 64
            m[length + j] = w < tree_rows.shape[1] and bool((int(tree_rows[i, w]) >> (j % 64)) & 1)
    return m


def attend(q, k, v, mask, scale):
    """One row: q [D], k, v [slots, D], mask [slots] -> (out, lse, sum p |v|)."""
    if not mask.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    s = (k[mask].astype(np.float64) @ q.astype(np.float64)) * scale
    top = s.max()
    p = np.exp(s - top)
    total = p.sum()
    vm = v[mask].astype(np.float64)
    return p @ vm / total, top + np.log(total), p @ np.abs(vm) / total


def received(q, lse, k, masks, scale):
    """Weight each slot receives: q [rows, D], lse [rows], masks [rows, slots]."""
    w = np.zeros(k.shape[0])
    for r in range(q.shape[0]):
        if np.isneginf(lse[r]):
            continue
        s = (k[masks[r]].astype(np.float64) @ q[r].astype(np.float64)) * scale
        w[masks[r]] += np.exp(s - float(lse[r]))
    return w


def evict(acc, pos, budget, sinks, recent, next_pos):
    """One sequence and head with len(acc) slots: (take, moves).  take[d] is
    the old slot whose row ends up in slot d; moves the (from, to) pairs."""
    n = len(acc)
    if n <= budget:
        return np.arange(n), []

    def key(j):  # protected, then larger weight, NaN below every number, then lower slot
        w = float(acc[j])
        free = not (pos[j] < sinks or pos[j] >= next_pos - recent)
        return (free, True, 0.0, j) if w != w else (free, False, -w, j)

    stays = set(sorted(range(n), key=key)[:budget])
    holes = [j for j in range(budget) if j not in stays]
    movers = [j for j in range(budget, n) if j in stays]
    take = np.arange(budget)
    take[holes] = movers
    return take, list(zip(movers, holes))
