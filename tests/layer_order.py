"""The declared orders of the head operators' sums, as numpy oracles beside layer_oracle's element-wise steps.

`head_sum` has a head's groups padded to at least four.
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
