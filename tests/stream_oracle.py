"""Plain implementations of the residual stream's operators for the tests.

`norm` and `norm_grad` repeat the library's binary32 operations in their
declared order (numpy float32, every input and result flushed); `norm64` and
`norm_grad64` are the definitions in 64 bits.  Rows are (rows, dim) arrays.
"""
import numpy as np
import torch

from layer_oracle import add, fl, mul, sub, tree

ONE = np.float32(1)


def rounded(x, kind):
    """x as a tensor of `kind` would hold it, in float32."""
    if kind == "f32":
        return np.asarray(x, np.float32)
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def lanes_of(dim):
    """(lanes of a row, sums that a lane holds)."""
    for lanes, most in ((64, 1024), (256, 4096), (512, 8192), (1024, 16384)):
        if dim <= most:
            return lanes, 2 if dim > most // 2 else 1
    raise ValueError(dim)


def row_sum(t):
    """The declared sum over the last axis of terms (rows, dim)."""
    rows, dim = t.shape
    lanes, each = lanes_of(dim)
    padded = np.zeros((rows, lanes * each * 8), np.float32)
    padded[:, :dim] = t
    groups = tree(padded.reshape(rows, each, lanes, 8))
    lane = groups[:, 0] if each == 1 else add(groups[:, 0], groups[:, 1])
    return tree(lane)[:, None]


def over_rows(t):
    """The declared sum over the rows of terms (rows, dim)."""
    rows, dim = t.shape
    G = 4 if dim <= 1024 else 1
    B = min(512, -(-rows // G))
    lists = np.zeros((B * G, dim), np.float32)
    for first in range(0, rows, B * G):
        part = t[first:first + B * G]
        lists[:len(part)] = add(lists[:len(part)], part)
    parts = lists.reshape(B, G, dim)
    while parts.shape[1] > 1:
        parts = add(parts[:, 0::2], parts[:, 1::2])
    parts = parts[:, 0]
    sums = np.zeros((128, dim), np.float32)
    for first in range(0, B, 128):
        part = parts[first:first + 128]
        sums[:len(part)] = add(sums[:len(part)], part)
    n = 64
    while n >= 1:
        sums = add(sums[:n], sums[n:2 * n])
        n //= 2
    return sums[0]


def _root(x, eps):
    inv = ONE / np.float32(x.shape[-1])
    d = add(mul(row_sum(mul(x, x)), inv), np.float32(eps))
    return fl(ONE / fl(np.sqrt(d, dtype=np.float32)))


def _after(u, block_gain, block_norm, eps):
    """(p, u * q, q)."""
    if not block_norm:
        return u, None, None
    q = _root(u, eps)
    n = mul(u, q)
    return (n if block_gain is None else mul(n, block_gain)), n, q


def norm(x, u, kind, gain=None, block_gain=None, gate=None, block_norm=False, x_scale=1.0, block_scale=1.0, eps=1e-6):
    """(y, z), before z is rounded to its type."""
    x, u, gain, block_gain, gate = (None if t is None else fl(t) for t in (x, u, gain, block_gain, gate))
    y = x
    if u is not None:
        t, _, _ = _after(u, block_gain, block_norm, eps)
        if gate is not None:
            t = mul(t, gate)
        y = fl(rounded(add(mul(x, np.float32(x_scale)), mul(t, np.float32(block_scale))), kind))
    z = mul(y, _root(y, eps))
    return y, (z if gain is None else mul(z, gain))


def norm_grad(y, u, dy, dz, gain=None, block_gain=None, gate=None, block_norm=False, x_scale=1.0, block_scale=1.0,
              eps=1e-6):
    """A dict of dx, dblock, dgain, dblock_gain and dgate (of every element; over the rows for a (dim) gate) before any
    is rounded to its type."""
    y, u, dy, dz, gain, block_gain, gate = (None if t is None else fl(t)
                                            for t in (y, u, dy, dz, gain, block_gain, gate))
    inv = ONE / np.float32(y.shape[-1])
    r = _root(y, eps)
    dn = dz if gain is None else mul(dz, gain)
    T = row_sum(mul(dn, y))
    w = mul(mul(mul(T, r), inv), r)
    Y = mul(sub(dn, mul(y, w)), r)
    if dy is not None:
        Y = add(dy, Y)
    out = {"dx": mul(Y, np.float32(x_scale)), "dgain": None if gain is None else over_rows(mul(dz, mul(y, r))),
           "dblock_gain": None, "dgate": None, "dblock": None}
    if u is None:
        return out
    P = mul(Y, np.float32(block_scale))
    p, n, q = _after(u, block_gain, block_norm, eps)
    if gate is not None:
        terms = mul(P, p)
        out["dgate"] = over_rows(terms) if gate.ndim == 1 else terms
        P = mul(P, gate)
    if block_norm:
        if block_gain is not None:
            out["dblock_gain"] = over_rows(mul(P, n))
            P = mul(P, block_gain)
        B = row_sum(mul(P, u))
        P = mul(sub(P, mul(u, mul(mul(mul(B, q), inv), q))), q)
    out["dblock"] = P
    return out


def norm64(x, u, kind, gain=None, block_gain=None, gate=None, block_norm=False, x_scale=1.0, block_scale=1.0,
           eps=1e-6, y=None):
    """(y, z, the magnitudes that bound y's rounding errors) in 64 bits; z is the norm of `y` where that is given."""
    x = np.asarray(x, np.float64)
    wide, size = x, np.abs(x)
    if u is not None:
        p = np.asarray(u, np.float64)
        if block_norm:
            p = p / np.sqrt(np.mean(p * p, -1, keepdims=True) + eps)
            p = p if block_gain is None else p * np.asarray(block_gain, np.float64)
        p = p if gate is None else p * np.asarray(gate, np.float64)
        wide = x * x_scale + p * block_scale
        size = np.abs(x * x_scale) + np.abs(p * block_scale)
    of = wide if y is None else np.asarray(y, np.float64)
    z = of / np.sqrt(np.mean(of * of, -1, keepdims=True) + eps)
    return wide, (z if gain is None else z * np.asarray(gain, np.float64)), size


def norm_grad64(y, u, dy, dz, gain=None, block_gain=None, gate=None, block_norm=False, x_scale=1.0, block_scale=1.0,
                eps=1e-6):
    """As norm_grad, in 64 bits: name -> (value, the magnitudes that bound its rounding errors)."""
    def wide(t):
        return None if t is None else np.asarray(t, np.float64)

    y, u, dy, dz, gain, block_gain, gate = (wide(t) for t in (y, u, dy, dz, gain, block_gain, gate))

    def through(x, d, size):
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
        n = x * r
        value = (d - n * (d * n).mean(-1, keepdims=True)) * r
        return value, (size + np.abs(n) * (size * np.abs(n)).mean(-1, keepdims=True)) * r, n

    g = 1.0 if gain is None else gain
    Y, size, n = through(y, dz * g, np.abs(dz * g))
    if dy is not None:
        Y, size = Y + dy, size + np.abs(dy)
    out = {"dx": (Y * x_scale, size * abs(x_scale))}
    if gain is not None:
        out["dgain"] = ((dz * n).sum(0), np.abs(dz * n).sum(0))
    if u is None:
        return out
    P, size = Y * block_scale, size * abs(block_scale)
    p = u
    if block_norm:
        nu = u / np.sqrt(np.mean(u * u, -1, keepdims=True) + eps)
        p = nu if block_gain is None else nu * block_gain
    if gate is not None:
        terms, of = P * p, size * np.abs(p)
        out["dgate"] = (terms, of) if gate.ndim == 2 else (terms.sum(0), of.sum(0))
        P, size = P * gate, size * np.abs(gate)
    if block_norm:
        if block_gain is not None:
            out["dblock_gain"] = ((P * nu).sum(0), (size * np.abs(nu)).sum(0))
            P, size = P * block_gain, size * np.abs(block_gain)
        P, size, _ = through(u, P, size)
    out["dblock"] = (P, size)
    return out
