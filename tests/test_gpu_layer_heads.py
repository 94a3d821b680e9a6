"""Norm and rotation of query and key heads on the GPU, and the backward pass.

Forward results and the input gradients equal the declared binary32 order
word for word (layer_oracle, numpy); both and the gains' gradients lie within
bounds derived below of the 64-bit definition.
"""
import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import layer_oracle as lo

pytestmark = pytest.mark.gpu

EPS = 1e-6
U = 2.0 ** -24  # a binary32 rounding
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _empty(b, s, hq, hk, d, dtype, layout):
    if layout == "packed":
        both = torch.empty(b, s, hq + hk, d, dtype=dtype, device="cuda")
        return both[:, :, :hq], both[:, :, hq:]
    if layout == "heads_first":
        return tuple(torch.empty(b, h, s, d, dtype=dtype, device="cuda").transpose(1, 2) for h in (hq, hk))
    if layout == "offset":  # one element off any vector's border, with gaps between heads
        return tuple(torch.empty(b * s * h * (d + 3) + 1, dtype=dtype, device="cuda")[1:].view(b, s, h, d + 3)[..., :d]
                     for h in (hq, hk))
    return tuple(torch.empty(b, s, h, d, dtype=dtype, device="cuda") for h in (hq, hk))


def _fill(t, gen, std):
    return t.copy_(torch.randn(t.shape, generator=gen).mul_(std))


def _table(rows, rotary):
    f = 5e5 ** (-np.arange(0, rotary, 2) / rotary)
    angle = np.arange(rows)[:, None] * f
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def _np(t):
    return t.detach().float().cpu().numpy()


def _make(b, s, hq, hk, d, rotary, kind, layout, gain, given, seed):
    gen = torch.Generator().manual_seed(seed)
    dtype = TYPES[kind]
    q, k = _empty(b, s, hq, hk, d, dtype, layout)
    _fill(q, gen, 1.5), _fill(k, gen, 0.7)
    dq, dk = _empty(b, s, hq, hk, d, dtype, "heads_first" if layout == "packed" else layout)
    _fill(dq, gen, 0.01), _fill(dk, gen, 1.0)
    rows = s + 40
    cos, sin = _table(rows, rotary)
    pos, where = None, np.broadcast_to(np.arange(s), (b, s))
    if given:
        where = torch.randint(0, rows, (b, s), generator=gen).numpy()
        pos = torch.from_numpy(where).to("cuda", torch.int32 if given == 32 else torch.int64)
    gains = [None, None]
    if gain:
        gains = [(1 + 0.2 * torch.randn(d, generator=gen)).to("cuda", TYPES[gain]) for _ in range(2)]
    return dict(q=q, k=k, dq=dq, dk=dk, cos=cos, sin=sin, pos=pos, where=where, gains=gains, dtype=dtype, kind=kind,
                layout=layout, shape=(b, s, hq, hk, d))


def _dev(x):
    return torch.from_numpy(x).cuda()


def _forward(m, interleaved):
    q_out, k_out = _empty(*m["shape"], m["dtype"], m["layout"])
    got = br.repro_qk_norm_rope(m["q"], m["k"], _dev(m["cos"]), _dev(m["sin"]), positions=m["pos"],
                                q_gain=m["gains"][0], k_gain=m["gains"][1], eps=EPS, interleaved=interleaved,
                                q_out=q_out, k_out=k_out)
    assert got[0] is q_out and got[1] is k_out
    return got


def _backward(m, interleaved):
    dq, dk = _empty(*m["shape"], m["dtype"], m["layout"])
    return br.repro_qk_norm_rope_backward(m["q"], m["k"], m["dq"], m["dk"], _dev(m["cos"]), _dev(m["sin"]),
                                          positions=m["pos"], q_gain=m["gains"][0], k_gain=m["gains"][1], eps=EPS,
                                          interleaved=interleaved, dq=dq, dk=dk)


def _rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)


def _same_words(got, want, what):
    g, w = got.cpu().contiguous(), want.contiguous()
    view = torch.int16 if g.dtype == torch.bfloat16 else torch.int32
    bad = (g.view(view) != w.view(view)).nonzero()
    assert not len(bad), f"{what}: {len(bad)} of {g.numel()} words differ, first at {bad[0].tolist()}"


def _check(m, interleaved):
    half_step = torch.finfo(m["dtype"]).eps / 2
    cos, sin = m["cos"][m["where"]][:, :, None], m["sin"][m["where"]][:, :, None]
    ys = _forward(m, interleaved)
    grads = _backward(m, interleaved)
    torch.cuda.synchronize()
    d = m["shape"][-1]
    for i, name in enumerate(("q", "k")):
        x, dy = _np(m[name]), _np(m["d" + name])
        gain = None if m["gains"][i] is None else _np(m["gains"][i])
        # The declared order, word for word.
        y = lo.heads(x, gain, cos, sin, EPS, interleaved, m["kind"])
        _same_words(ys[i], _rounded(y, m["dtype"]), name + " forward")
        dx, terms = lo.heads_grad(x, dy, gain, cos, sin, EPS, interleaved, m["kind"])
        _same_words(grads[i], _rounded(dx, m["dtype"]), name + " backward")
        # 64 bits.  S: log2(D) + 2 roundings; mean, eps, root, quotient: r is
        # off by at most (log2(D) + 5) / 2 + 2; n, z, product, sum: 4 more.
        depth = np.log2(d) + 2
        y64, size = lo.heads64(x, gain, cos.astype(np.float64), sin.astype(np.float64), EPS, interleaved)
        tol = (depth / 2 + 8) * U * size
        tol += half_step * (np.abs(y64) + tol)
        assert (np.abs(_np(ys[i]) - y64) <= tol + 1e-37).all(), name
        # Backward: dn 4 roundings of size; T as S over |dn x|, times r twice
        # off; the difference, the last product: 2 more.
        dx64, size, dgain64, dgain_size = lo.heads_grad64(x, dy, gain, cos.astype(np.float64), sin.astype(np.float64),
                                                          EPS, interleaved)
        tol = (3 * depth + 16) * U * size
        tol += half_step * (np.abs(dx64) + tol)
        assert (np.abs(_np(grads[i]) - dx64) <= tol + 1e-37).all(), "d" + name
        if gain is None:
            assert grads[2 + i] is None
        elif x.size:
            # Terms: dz 3 roundings, n depth / 2 + 4, product 1; sums: at most
            # 2 heads x 64 items in a lane here, then trees of at most 2^13.
            assert grads[2 + i].dtype == torch.float32
            tol = (depth / 2 + 8 + 128 + 16 + 13) * U * dgain_size
            assert (np.abs(_np(grads[2 + i]) - dgain64) <= tol).all(), name + " gain"


SHAPES = [  # batch, seq, q heads, k heads, dim, rotary
    (1, 1, 16, 4, 128, 128), (2, 67, 16, 4, 128, 128), (1, 1, 1, 1, 2, 2), (3, 5, 3, 1, 6, 4), (2, 9, 5, 2, 14, 14),
    (1, 33, 4, 2, 16, 6), (2, 31, 4, 4, 16, 16), (1, 17, 6, 2, 64, 64), (2, 19, 12, 4, 80, 64), (5, 33, 7, 1, 96, 48),
    (1, 13, 3, 3, 94, 36), (1, 13, 3, 3, 90, 86), (2, 7, 2, 2, 256, 256), (1, 6, 2, 1, 512, 130), (1, 3, 9, 5, 510, 508),
    (1, 300, 8, 8, 128, 2), (7, 1, 8, 1, 128, 64), (1, 130, 1, 1, 22, 16), (1, 700, 2, 1, 64, 32), (3, 5, 6, 2, 32, 32), (1, 9, 5, 3, 40, 10), (2, 3, 4, 4, 62, 58),
    (1, 4, 3, 2, 258, 258), (1, 5, 2, 2, 192, 192), (2, 6, 3, 1, 30, 8), (1, 4, 2, 1, 250, 6),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, kind, interleaved):
    print("heads", shape, kind, interleaved, flush=True)
    m = _make(*shape, kind, "packed", kind if shape[0] % 2 else None, 32 if shape[1] % 2 else 0, seed=sum(shape))
    _check(m, interleaved)


@pytest.mark.parametrize("layout", ["plain", "packed", "heads_first", "offset"])
@pytest.mark.parametrize("kind, gain", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", None)])
def test_layouts_and_gain_types(layout, kind, gain):
    print("heads", layout, kind, gain, flush=True)
    for dim, rotary in ((128, 128), (72, 26)):
        _check(_make(2, 21, 8, 2, dim, rotary, kind, layout, gain, 64, seed=dim), False)


@pytest.mark.parametrize("seed", range(24))
def test_random_sweep(seed):
    rng = np.random.default_rng(1000 + seed)
    dim = 2 * int(rng.integers(1, 257) if seed % 4 == 0 else rng.integers(1, 80))
    rotary = dim if rng.random() < 0.4 else 2 * int(rng.integers(1, dim // 2 + 1))
    b, s, hq, hk = (int(rng.integers(1, n)) for n in (5, 40, 14, 6))
    kind, layout = rng.choice(["bf16", "f32"]), rng.choice(["plain", "packed", "heads_first", "offset"])
    gain, given = rng.choice([None, "f32", "bf16"]), int(rng.choice([0, 32, 64]))
    interleaved = bool(rng.random() < 0.5)
    print("sweep", seed, b, s, hq, hk, dim, rotary, kind, layout, gain, given, interleaved, flush=True)
    _check(_make(b, s, hq, hk, dim, rotary, str(kind), str(layout), gain, given, seed=seed), interleaved)


def test_many_tokens():
    # Several passes of every workgroup of the gains' gradient, whose number
    # is bounded: 768 workgroups of 64 groups, and 420000 heads.
    m = _make(1, 140000, 2, 1, 64, 64, "bf16", "plain", "f32", 0, seed=5)
    _check(m, False)


def test_past_the_caches():
    # Enough data for the nontemporal accesses.
    for kind in ("bf16", "f32"):
        print("past the caches", kind, flush=True)
        _check(_make(1, 9000, 12, 4, 128, 128, kind, "packed", "f32", 32, seed=6), False)
    print("past the caches, ragged", flush=True)
    _check(_make(2, 15000, 6, 2, 72, 26, "bf16", "plain", None, 0, seed=7), True)
    _check(_make(1, 27000, 11, 5, 40, 40, "bf16", "packed", None, 0, seed=8), False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_subnormal_values(kind):
    # Elements, gradients and gains around 2^-126: operands and results flush
    # as the contract says, word for word.
    m = _make(1, 40, 4, 2, 64, 48, kind, "plain", "f32", 0, seed=11)
    gen = torch.Generator().manual_seed(1)
    for name in ("q", "k", "dq", "dk"):
        power = torch.randint(-149, -100, m[name].shape, generator=gen).float()
        m[name].copy_(torch.randn(m[name].shape, generator=gen) * torch.exp2(power))
    m["q"][0, 5:].copy_(torch.randn(35, 4, 64, generator=gen))
    m["gains"][0][::3] *= 1e-38
    for i, name in enumerate(("q", "k")):
        cos, sin = m["cos"][m["where"]][:, :, None], m["sin"][m["where"]][:, :, None]
        args = (_np(m["gains"][i]), cos, sin, EPS, False, kind)
        y = lo.heads(_np(m[name]), *args)
        _same_words(_forward(m, False)[i], _rounded(y, m["dtype"]), name)
        dx, _ = lo.heads_grad(_np(m[name]), _np(m["d" + name]), *args)
        _same_words(_backward(m, False)[i], _rounded(dx, m["dtype"]), "d" + name)


def test_one_gain_only_and_empty():
    m = _make(2, 5, 4, 2, 32, 32, "f32", "plain", "f32", 0, seed=1)
    m["gains"][1] = None
    _check(m, False)
    for b, s, hq, hk in ((0, 5, 4, 2), (2, 0, 4, 2), (2, 5, 0, 2), (2, 5, 4, 0)):
        m = _make(b, s, hq, hk, 32, 32, "bf16", "plain", "f32", 0, seed=1)
        _check(m, False)
        grads = _backward(m, False)
        for h, g in ((hq, grads[2]), (hk, grads[3])):
            if b * s * h == 0:
                assert (g == 0).all()  # the sum of no terms


def test_in_place_and_broadcast_inputs():
    m = _make(2, 11, 6, 3, 72, 26, "bf16", "packed", "bf16", 32, seed=3)
    args = (_dev(m["cos"]), _dev(m["sin"]))
    kw = dict(positions=m["pos"], q_gain=m["gains"][0], k_gain=m["gains"][1])
    want = br.repro_qk_norm_rope(m["q"], m["k"], *args, **kw)
    grads = br.repro_qk_norm_rope_backward(m["q"], m["k"], m["dq"], m["dk"], *args, **kw)
    # The gradients over their own upstream gradients.
    dq, dk = m["dq"].clone(), m["dk"].clone()
    br.repro_qk_norm_rope_backward(m["q"], m["k"], dq, dk, *args, dq=dq, dk=dk, **kw)
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])
    br.repro_qk_norm_rope(m["q"], m["k"], *args, q_out=m["q"], k_out=m["k"], **kw)
    assert torch.equal(m["q"], want[0]) and torch.equal(m["k"], want[1])
    # One key head of memory read as many, one row of positions for the batch.
    one = torch.randn(2, 11, 1, 72, device="cuda").bfloat16()
    pos = torch.arange(7, 18, device="cuda")
    wide, full = one.expand(2, 11, 4, 72), one.expand(2, 11, 4, 72).contiguous()
    a = br.repro_qk_norm_rope(wide, full, *args, positions=pos)
    assert torch.equal(a[0], a[1])
    b = br.repro_qk_norm_rope(wide, full, *args, positions=pos.expand(2, 11).int())
    assert torch.equal(a[0], b[0])


def test_bits_depend_on_the_head_alone():
    # A head's result is the same wherever it lies: layout, batch, neighbours.
    m = _make(3, 50, 5, 2, 128, 128, "bf16", "packed", None, 0, seed=9)
    cos, sin = _dev(m["cos"]), _dev(m["sin"])
    whole = br.repro_qk_norm_rope(m["q"], m["k"], cos, sin)
    pos = torch.tensor([[37]], device="cuda")
    for b, h in ((0, 0), (2, 4), (1, 3)):
        q = m["q"][b:b + 1, 37:38, h:h + 1].clone()
        one = br.repro_qk_norm_rope(q, q, cos, sin, positions=pos)
        assert torch.equal(one[0][0, 0, 0], whole[0][b, 37, h]) and torch.equal(one[0], one[1])


def test_bad_positions_and_values_stay_in_their_rows():
    m = _make(1, 6, 3, 2, 32, 16, "f32", "plain", None, 0, seed=2)
    cos, sin = _dev(m["cos"]), _dev(m["sin"])
    rows = cos.shape[0]
    pos = torch.tensor([0, -1, 5, rows, 2 ** 31 - 1, 3], dtype=torch.int32, device="cuda")
    clean = br.repro_qk_norm_rope(m["q"], m["k"], cos, sin, positions=pos.clamp(0, rows - 1))
    y = br.repro_qk_norm_rope(m["q"], m["k"], cos, sin, positions=pos)
    dx = br.repro_qk_norm_rope_backward(m["q"], m["k"], m["dq"], m["dk"], cos, sin, positions=pos)
    far = br.repro_qk_norm_rope(m["q"], m["k"], cos, sin, positions=pos.long() * (1 << 32))
    for i in range(2):
        for s in (1, 3, 4):
            assert y[i][0, s, :, :16].isnan().all() and dx[i][0, s].isnan().all()
            assert torch.equal(y[i][0, s, :, 16:], clean[i][0, s, :, 16:])
            assert far[i][0, s, :, :16].isnan().all()
        for s in (0, 2, 5):
            assert torch.equal(y[i][0, s], clean[i][0, s]) and dx[i][0, s].isfinite().all()
    # Infinities, NaN, zeros and the type's lowest value in some heads.
    low = torch.finfo(torch.float32).min
    for value in (float("inf"), float("nan"), 0.0, low):
        x = m["q"].clone()
        x[0, 2, 1] = value
        y = br.repro_qk_norm_rope(x, m["k"], cos, sin)
        ref = br.repro_qk_norm_rope(m["q"], m["k"], cos, sin)
        keep = torch.ones_like(x, dtype=torch.bool)
        keep[0, 2, 1] = False
        assert torch.equal(y[0][keep], ref[0][keep])
        head = y[0][0, 2, 1]
        if value == 0.0:
            assert (head == 0).all()  # eps alone: 0 * 1000
        elif value == low:
            assert (head.abs() == 0).all()  # the square sum is infinite, its reciprocal root 0
        else:
            assert head.isnan().all()


def test_refusals():
    m = _make(1, 4, 4, 2, 32, 32, "f32", "plain", None, 0, seed=2)
    q, k, cos, sin = m["q"], m["k"], _dev(m["cos"]), _dev(m["sin"])
    call = br.repro_qk_norm_rope
    bad = [
        (ValueError, lambda: call(q[0], k, cos, sin)), (ValueError, lambda: call(q, k[:, :3], cos, sin)),
        (ValueError, lambda: call(q, k[..., :16], cos, sin)), (TypeError, lambda: call(q, k.bfloat16(), cos, sin)),
        (TypeError, lambda: call(q.half(), k.half(), cos, sin)), (TypeError, lambda: call(q, k, cos.double(), sin)),
        (ValueError, lambda: call(q, k, cos, sin[:3])), (ValueError, lambda: call(q, k, cos[:, ::2], sin[:, ::2])),
        (br.ReproError, lambda: call(q, k, cos[:3], sin[:3])), (br.ReproError, lambda: call(q, k, cos, sin, eps=-1.0)),
        (TypeError, lambda: call(q, k, cos, sin, positions=torch.zeros(4, device="cuda"))),
        (ValueError, lambda: call(q, k, cos, sin, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))),
        (ValueError, lambda: call(q, k, cos, sin, q_gain=torch.zeros(16, device="cuda"))),
        (TypeError, lambda: call(q, k, cos, sin, q_gain=torch.zeros(32, device="cuda"),
                                 k_gain=torch.zeros(32, device="cuda").bfloat16())),
        (ValueError, lambda: call(q, k, cos, sin, q_out=k)),
        (br.ReproError, lambda: call(q, k, cos, sin, q_out=torch.zeros(1, 4, 1, 32, device="cuda").expand(1, 4, 4, 32))),
        (ValueError, lambda: call(q.transpose(2, 3).contiguous().transpose(2, 3), k, cos, sin)),
        (TypeError, lambda: call(q.cpu(), k, cos, sin)), (TypeError, lambda: call(q, k, cos, sin, q_out=q.cpu())),
    ]
    for kind, f in bad:
        with pytest.raises(kind):
            f()
    g = torch.ones(32, device="cuda")
    back = br.repro_qk_norm_rope_backward
    with pytest.raises(br.ReproError, match="workspace"):
        back(q, k, q, k, cos, sin, q_gain=g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        back(q, k, q, k, cos, sin, dq_gain=g)
    with pytest.raises(ValueError):
        back(q, k, q[:, :3], k, cos, sin)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradients_against_differences(interleaved):
    # Central differences of the 64-bit definition at steps of 1e-5: their own
    # error is about step^2 (third derivatives of order one), 1e-9 here.
    m = _make(1, 3, 2, 1, 20, 12, "f32", "plain", "f32", 0, seed=8)
    grads = [None if g is None else _np(g).astype(np.float64) for g in _backward(m, interleaved)]
    cos, sin = m["cos"][m["where"]][:, :, None].astype(np.float64), m["sin"][m["where"]][:, :, None].astype(np.float64)
    rng = np.random.default_rng(0)
    for i, name in enumerate(("q", "k")):
        x, dy, gain = (_np(t).astype(np.float64) for t in (m[name], m["d" + name], m["gains"][i]))

        def loss(x, gain):
            return float((lo.heads64(x, gain, cos, sin, EPS, interleaved)[0] * dy).sum())

        scale = np.abs(dy).max()
        for _ in range(12):
            at = tuple(rng.integers(n) for n in x.shape)
            step = np.zeros_like(x)
            step[at] = 1e-5
            diff = (loss(x + step, gain) - loss(x - step, gain)) / 2e-5
            assert abs(diff - grads[i][at]) <= 1e-5 * scale
            step = np.zeros_like(gain)
            step[at[-1]] = 1e-5
            diff = (loss(x, gain + step) - loss(x, gain - step)) / 2e-5
            assert abs(diff - grads[2 + i][at[-1]]) <= 1e-5 * scale * 6


def test_other_stream_and_graph():
    m = _make(2, 40, 6, 2, 80, 48, "bf16", "packed", "bf16", 32, seed=4)
    cos, sin = _dev(m["cos"]), _dev(m["sin"])
    kw = dict(positions=m["pos"], q_gain=m["gains"][0], k_gain=m["gains"][1])

    def both(**more):
        y = br.repro_qk_norm_rope(m["q"], m["k"], cos, sin, **kw, **more)
        return [*y, *br.repro_qk_norm_rope_backward(m["q"], m["k"], m["dq"], m["dk"], cos, sin, **kw, **more)]

    want = both()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = both(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(3):
        m["q"].mul_(-1.25)
        m["dk"].mul_(0.5)
        want = both()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


def test_offsets_past_32_bits():
    # One head every 2^31 + 2^27 elements: byte offsets past 2^32.
    stride = (1 << 31) + (1 << 27)
    flat = torch.empty(2 * stride + 128, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((1, 3, 1, 128), (0, stride, 128, 1))
    data = torch.randn(1, 3, 1, 128, device="cuda").bfloat16()
    x.copy_(data)
    cos, sin = (_dev(t) for t in _table(3, 128))
    want = br.repro_qk_norm_rope(data, data, cos, sin)
    got = br.repro_qk_norm_rope(x, data, cos, sin, q_out=x)
    assert torch.equal(got[0], want[0])
    assert torch.equal(x, want[0])
