"""Plain implementations of the layer operators for the tests.

`heads` and `heads_grad` repeat the library's binary32 operations in their
declared order (numpy float32, every input and result flushed); `heads64` and
`heads_grad64` are the definitions in 64 bits.
"""
import numpy as np

TINY = np.float32(2.0 ** -126)


def fl(x):
    """A float32 result under the contract: subnormals become zeros of their sign."""
    x = np.asarray(x, np.float32)
    return np.where(np.abs(x) < TINY, np.copysign(np.float32(0), x), x)


def add(a, b):
    return fl(np.add(a, b, dtype=np.float32))


def sub(a, b):
    return fl(np.subtract(a, b, dtype=np.float32))


def mul(a, b):
    return fl(np.multiply(a, b, dtype=np.float32))


def tree(t):
    """Perfect pairwise tree over the last axis, padded with +0 to a power of two."""
    n = 1
    while n < t.shape[-1]:
        n *= 2
    t = np.concatenate([t, np.zeros(t.shape[:-1] + (n - t.shape[-1],), np.float32)], -1)
    while t.shape[-1] > 1:
        t = add(t[..., 0::2], t[..., 1::2])
    return t[..., 0]


def lanes(dim, rotary, interleaved, V):
    """[(elements of the lane's 2V places, counted places)] of one head, in lane order."""
    half = rotary // 2
    out = []
    for begin, count in ((0, half), (rotary, dim // 2 - half)):
        for want in range(0, count, V):
            first = min(want, count - V)
            if begin == 0:
                first = max(first, 0)
            pairs = range(first, first + V)
            ok = [want <= p < count for p in pairs]
            if interleaved:
                out.append(([begin + 2 * first + k for k in range(2 * V)], [ok[k // 2] for k in range(2 * V)]))
            else:
                out.append(([begin + p for p in pairs] + [begin + count + p for p in pairs], ok + ok))
    return out


def vector_of(dim, kind):
    """Pairs of a lane, for elements of kind "f32" or "bf16"."""
    if dim < 16:
        return 1
    return (4 if dim <= 32 else 8) if kind == "bf16" else (4 if dim <= 256 else 8)


def head_sum(t, rotary, interleaved, kind):
    """The declared tree over a head of terms (last axis)."""
    V = vector_of(t.shape[-1], kind)
    per_lane = []
    for index, counted in lanes(t.shape[-1], rotary, interleaved, V):
        v = np.where(counted, t[..., index], np.float32(0))
        p = add(v[..., 0::2], v[..., 1::2]) if interleaved else add(v[..., :V], v[..., V:])
        per_lane.append(tree(p))
    return tree(np.stack(per_lane, -1))


def _pairs(dim, rotary, interleaved):
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def _r(x, rotary, eps, interleaved, kind):
    S = head_sum(mul(x, x), rotary, interleaved, kind)
    inv = np.float32(1) / np.float32(x.shape[-1])
    d = add(mul(S, inv), np.float32(eps))
    return fl(np.float32(1) / fl(np.sqrt(d, dtype=np.float32)))[..., None]


def heads(x, gain, cos, sin, eps, interleaved, kind):
    """x (..., D) float32, cos and sin broadcastable to (..., h): the result before rounding to its type."""
    x, cos, sin = fl(x), fl(cos), fl(sin)
    gain = None if gain is None else fl(gain)
    rotary = 2 * cos.shape[-1]
    z = mul(x, _r(x, rotary, eps, interleaved, kind))
    if gain is not None:
        z = mul(z, gain)
    ia, ib = _pairs(x.shape[-1], rotary, interleaved)
    a, b = z[..., ia], z[..., ib]
    y = z.copy()
    y[..., ia] = sub(mul(a, cos), mul(b, sin))
    y[..., ib] = add(mul(b, cos), mul(a, sin))
    return y


def heads_grad(x, dy, gain, cos, sin, eps, interleaved, kind):
    """(dx before rounding to its type, the gain's terms dz * n)."""
    x, cos, sin = fl(x), fl(cos), fl(sin)
    gain = None if gain is None else fl(gain)
    rotary = 2 * cos.shape[-1]
    r = _r(x, rotary, eps, interleaved, kind)
    ia, ib = _pairs(x.shape[-1], rotary, interleaved)
    dy = fl(dy)
    dz = dy.copy()
    a, b = dy[..., ia], dy[..., ib]
    dz[..., ia] = add(mul(a, cos), mul(b, sin))
    dz[..., ib] = sub(mul(b, cos), mul(a, sin))
    n = mul(x, r)
    terms = mul(dz, n)
    dn = dz if gain is None else mul(dz, gain)
    T = head_sum(mul(dn, x), rotary, interleaved, kind)[..., None]
    w = mul(mul(mul(T, r), np.float32(1) / np.float32(x.shape[-1])), r)
    return mul(sub(dn, mul(x, w)), r), terms


def heads64(x, gain, cos, sin, eps, interleaved):
    """(y, the magnitudes that bound its rounding errors) in 64 bits."""
    x = np.asarray(x, np.float64)
    z = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if gain is not None:
        z = z * np.asarray(gain, np.float64)
    ia, ib = _pairs(x.shape[-1], 2 * cos.shape[-1], interleaved)
    a, b = z[..., ia], z[..., ib]
    y, size = z.copy(), np.abs(z)
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    size[..., ia] = np.abs(a * cos) + np.abs(b * sin)
    size[..., ib] = np.abs(b * cos) + np.abs(a * sin)
    return y, size


def heads_grad64(x, dy, gain, cos, sin, eps, interleaved):
    """(dx, its magnitudes, the gain's gradient, its magnitudes) in 64 bits."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    D = x.shape[-1]
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    ia, ib = _pairs(D, 2 * cos.shape[-1], interleaved)
    a, b = dy[..., ia], dy[..., ib]
    dz, size = dy.copy(), np.abs(dy)
    dz[..., ia], dz[..., ib] = a * cos + b * sin, b * cos - a * sin
    size[..., ia] = np.abs(a * cos) + np.abs(b * sin)
    size[..., ib] = np.abs(b * cos) + np.abs(a * sin)
    n = x * r
    axes = tuple(range(x.ndim - 1))
    dgain, dgain_size = (dz * n).sum(axes), (size * np.abs(n)).sum(axes)
    g = 1.0 if gain is None else np.asarray(gain, np.float64)
    dn, size = dz * g, size * np.abs(g)
    along = (dn * n).mean(-1, keepdims=True)
    dx = (dn - n * along) * r
    size = (size + np.abs(n) * (size * np.abs(n)).mean(-1, keepdims=True)) * r
    return dx, size, dgain, dgain_size
