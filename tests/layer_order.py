"""The declared orders of the head operators' sums, as numpy oracles beside layer_oracle's element-wise steps.

`head_sum` has a head's groups padded to at least four; `gain_grad` is the gains' gradient.
"""
import numpy as np

import layer_oracle as lo


def padded_groups(dim, rotary, interleaved, kind):
    """A head's groups of pairs, padded to a power of two of at least four."""
    n = len(lo.lanes(dim, rotary, interleaved, lo.vector_of(dim, kind)))
    p = 4
    while p < n:
        p *= 2
    return p


def head_sum(t, rotary, interleaved, kind):
    """The sum over a head of terms (last axis)."""
    dim = t.shape[-1]
    V = lo.vector_of(dim, kind)
    sums = np.zeros(t.shape[:-1] + (padded_groups(dim, rotary, interleaved, kind),), np.float32)
    for j, (index, counted) in enumerate(lo.lanes(dim, rotary, interleaved, V)):
        v = np.where(counted, t[..., index], np.float32(0))
        pairs = lo.add(v[..., 0::2], v[..., 1::2]) if interleaved else lo.add(v[..., :V], v[..., V:])
        sums[..., j] = lo.tree(pairs)
    return lo.tree(sums)


def rows_of(tokens, heads, dim, rotary, interleaved, kind):
    """(lists of a row, rows of each side)."""
    lists = 256 // padded_groups(dim, rotary, interleaved, kind)
    rows = [-(-tokens * h // lists) for h in heads]
    most = 768 if lo.vector_of(dim, kind) == 8 else 1280
    turns = max(1, -(-sum(rows) // most))
    return lists, [-(-r // turns) for r in rows]


def gain_grad(terms, side, heads, rotary, interleaved, kind):
    """The gradient of one side's gain from its terms dz * n, (batch, seq, heads[side], dim)."""
    b, s, h, dim = terms.shape
    assert h == heads[side]
    lists, rows = rows_of(b * s, heads, dim, rotary, interleaved, kind)
    rows = rows[side]
    terms = terms.reshape(-1, dim)
    sums = np.zeros((rows * lists, dim), np.float32)
    for at in range(0, len(terms), max(len(sums), 1)):
        part = terms[at:at + len(sums)]
        sums[:len(part)] = lo.add(sums[:len(part)], part)
    row = lo.tree(np.moveaxis(sums.reshape(rows, lists, dim), 1, 2))
    parts = np.zeros((128, dim), np.float32)
    for at in range(0, rows, 128):
        some = row[at:at + 128]
        parts[:len(some)] = lo.add(parts[:len(some)], some)
    n = 64
    while n:
        parts[:n] = lo.add(parts[:n], parts[n:2 * n])
        n //= 2
    return parts[0]
