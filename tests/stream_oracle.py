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


def over_rows(t, branch=True):
    """The declared sum over the rows of terms (rows, dim)."""
    rows, dim = t.shape
    G = 4 if dim <= 1024 else 1
    B = min(512 if branch else 1024, -(-rows // G))
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
    out = {"dx": mul(Y, np.float32(x_scale)), "dgain": None if gain is None else over_rows(mul(dz, mul(y, r)), block_norm or gate is not None),
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


# ------------------------------------------------------------ the vocabulary loss

L2E = np.float32(1.4426950408889634)
LN2 = 0.6931471805599453
POLY = [np.float32(float.fromhex(c)) for c in ("0x1.41d334p-13", "0x1.5f456ap-10", "0x1.3b2dbcp-7", "0x1.c6aed4p-5",
                                               "0x1.ebfbdap-3", "0x1.62e430p-1", "0x1p0")]


def bits16(x):
    """The bf16 bits of float32 values, rounded to nearest even."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(
        np.uint16)


def wide16(u):
    return (np.asarray(u, np.uint32) << 16).view(np.float32)


def parts(x):
    """(high, middle, low) as bf16 bits."""
    high = bits16(fl(x))
    fine = (high & 0x7f80) != 0x7f80
    with np.errstate(invalid="ignore"):
        rest = np.where(fine, sub(fl(x), wide16(high)), np.float32(0))
    middle = bits16(rest)
    return high, middle, bits16(sub(rest, wide16(middle)))


def product(a, b, kind):
    """The declared product of the rows of a and b (float32; of bf16 values for "bf16")."""
    import oracle
    if kind == "bf16":
        return oracle.block_product(bits16(a), bits16(b))
    a, b = parts(a), parts(b)
    acc = None
    for k in range(0, a[0].shape[1], 32):
        for i, j in ((2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)):
            acc = oracle.block_product(a[i][:, k:k + 32], b[j][:, k:k + 32], acc)
    return acc


def p2(t):
    import oracle
    t = np.fmin(np.fmax(t, np.float32(-200)), np.float32(1))
    u = np.rint(t)
    f = sub(t, u)
    p = np.full_like(f, POLY[0])
    for c in POLY[1:]:
        p = oracle.fma(p, f, np.full_like(f, c))
    return fl(np.ldexp(p, u.astype(np.int32)))


def scaled(l, shift):
    """fma(l, L2E, -shift)."""
    import oracle
    return oracle.fma(l, np.full_like(l, L2E), np.ascontiguousarray(np.broadcast_to(-shift, l.shape), np.float32))


def natural_log(v):
    f, e = np.frexp(v)
    low = f < float.fromhex("0x1.6a09e667f3bcdp-1")
    f, e = np.where(low, f * 2.0, f), np.where(low, e - 1, e)
    s = (f - 1.0) / (f + 1.0)
    q = s * s
    p = np.full_like(s, 1.0 / 23.0)
    for k in range(21, 0, -2):
        p = p * q + 1.0 / k
    return e * LN2 + 2.0 * s * p


def vocab_loss(x, w, labels, kind, z_weight=0.0, ignored=-100):
    """(loss, lse) of finite inputs in the declared order."""
    V = w.shape[0]
    l = product(w, x, kind).T
    blocks = -(-V // 128)
    padded = np.full((len(x), blocks * 128), -np.inf, np.float32)
    padded[:, :V] = l
    padded = padded.reshape(len(x), blocks, 128)
    n = np.rint(mul(padded.max(-1), L2E))
    terms = np.zeros_like(padded)
    real = np.isfinite(padded)
    terms[real] = p2(scaled(np.where(real, padded, np.float32(0)), n[..., None]))[real]
    terms = terms.reshape(len(x), blocks, 16, 8)
    chain = terms[:, :, 0]
    for i in range(1, 16):
        chain = add(chain, terms[:, :, i])
    s = tree(chain)
    top = n.max(-1)
    sums = np.zeros((len(x), 64))
    for b in range(blocks):
        sums[:, b % 64] += np.ldexp(s[:, b].astype(np.float64), (n[:, b] - top).astype(np.int32))
    while sums.shape[1] > 1:
        sums = sums[:, 0::2] + sums[:, 1::2]
    lse = top.astype(np.float64) * LN2 + natural_log(sums[:, 0])
    counted = labels != ignored
    picked = l[np.arange(len(x)), np.where(counted, labels, 0)].astype(np.float64)
    loss = (lse - picked) + float(np.float32(z_weight)) * (lse * lse)
    return np.where(counted, loss, 0.0).astype(np.float32), lse.astype(np.float32)


def spans_of(N, D, V):
    """(tokens of a tile, entries of a span) of the backward pass."""
    T = 64 if N <= 64 else 128 if N <= 128 else 256
    tiles = -(-N // T) * -(-D // 256)
    beside = max(1, 256 // tiles)
    padded = -(-N // T) * T
    wanted, shortest = (-(-512 // tiles), 512) if N <= 64 else (beside, 1024)
    spans = max(min(wanted, -(-V // shortest)), -(-padded * V * beside // 2 ** 27))
    return T, -(-(-(-V // spans)) // 256) * 256


def vocab_loss_grad(x, w, labels, lse, dloss, kind, z_weight=0.0, ignored=-100):
    """(dx, dw) of finite inputs in the declared order, before they are rounded to their type."""
    N, V = len(x), w.shape[0]
    l = product(w, x, kind).T
    c = (lse.astype(np.float64) * float.fromhex("0x1.71547652b82fep+0")).astype(np.float32)
    g = np.broadcast_to(np.asarray(dloss, np.float32), (N,))
    a = (g.astype(np.float64) * (1.0 + 2.0 * float(np.float32(z_weight)) * lse.astype(np.float64))).astype(np.float32)
    d = mul(p2(scaled(l, c[:, None])), a[:, None])
    counted = labels != ignored
    rows = np.flatnonzero(counted)
    d[rows, labels[rows]] = sub(d[rows, labels[rows]], g[rows])
    d[~counted] = 0
    T, span = spans_of(N, x.shape[1], V)
    dx = None
    for first in range(0, V, span):
        of, by = w[first:first + span].T, d[:, first:first + span]
        pad = -of.shape[1] % 256
        part = product(np.pad(of, ((0, 0), (0, pad))), np.pad(by, ((0, 0), (0, pad))), kind).T
        dx = part if dx is None else add(dx, part)
    pad = -N % T
    masked = np.where(counted[:, None], x, np.float32(0))
    dw = product(np.pad(masked.T, ((0, 0), (0, pad))), np.pad(d.T, ((0, 0), (0, pad))), kind).T
    dx[~counted] = 0
    return (fl(dx), fl(dw)) if kind == "bf16" else (dx, dw)  # the rounding to bf16 flushes


def vocab_loss64(x, w, labels, z_weight=0.0, ignored=-100):
    """(loss, lse, logits) in 64 bits."""
    l = np.asarray(x, np.float64) @ np.asarray(w, np.float64).T
    top = l.max(-1, keepdims=True)
    lse = (top + np.log(np.exp(l - top).sum(-1, keepdims=True)))[:, 0]
    counted = labels != ignored
    picked = l[np.arange(len(l)), np.where(counted, labels, 0)]
    return np.where(counted, lse - picked + z_weight * lse * lse, 0.0), lse, l


def vocab_loss_grad64(x, w, labels, lse, dloss, z_weight=0.0, ignored=-100):
    """(dx, dw, dl) in 64 bits."""
    x, w, lse = (np.asarray(t, np.float64) for t in (x, w, lse))
    g = np.broadcast_to(np.asarray(dloss, np.float64), (len(x),)) * (labels != ignored)
    dl = np.exp(x @ w.T - lse[:, None]) * (g * (1 + 2 * z_weight * lse))[:, None]
    dl[np.arange(len(x)), np.where(labels != ignored, labels, 0)] -= g
    return dl @ w, dl.T @ x, dl
