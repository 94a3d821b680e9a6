"""The residual stream's norm and its gradients on the GPU.

Every result equals the declared binary32 order word for word (stream_oracle,
numpy) and lies within bounds derived below of the 64-bit definition.
"""
import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import stream_oracle as so

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # a binary32 rounding
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def empty(b, s, d, kind, layout):
    t = TYPES[kind]
    if layout == "packed":  # a part of wider rows
        return torch.empty(b, s, 3 * d, dtype=t, device="cuda")[..., d:2 * d]
    if layout == "seq_first":
        return torch.empty(s, b, d, dtype=t, device="cuda").transpose(0, 1)
    if layout == "offset":  # one element off any vector's border, with gaps between rows
        return torch.empty(b * s * (d + 3) + 1, dtype=t, device="cuda")[1:].view(b, s, d + 3)[..., :d]
    return torch.empty(b, s, d, dtype=t, device="cuda")


def fill(t, gen, std, mean=0.0):
    return t.copy_(torch.randn(t.shape, generator=gen).mul_(std).add_(mean))


def flat(t):
    return None if t is None else t.detach().float().cpu().numpy().reshape(-1, t.shape[-1])


def make(b, s, d, kind, layout, gain, block_norm, gate, x_scale, block_scale, seed):
    gen = torch.Generator().manual_seed(seed)
    of = {"f32": torch.float32, "bf16": torch.bfloat16}.get(gain, TYPES[kind])

    def channel(std, mean):
        return (torch.randn(d, generator=gen) * std + mean).to("cuda", of)

    m = dict(x=fill(empty(b, s, d, kind, layout), gen, 2.0), block=fill(empty(b, s, d, kind, layout), gen, 0.6),
             dy=fill(empty(b, s, d, kind, "plain"), gen, 0.01), dz=fill(empty(b, s, d, kind, layout), gen, 0.02))
    form = dict(gain=channel(0.2, 1.0) if gain else None, block_gain=channel(0.2, 1.0) if gain and block_norm else None,
                gate=None, block_norm=block_norm, x_scale=x_scale, block_scale=block_scale, eps=1e-6)
    if gate == "channel":
        form["gate"] = channel(0.3, 0.5)
    elif gate == "element":
        form["gate"] = fill(empty(b, s, d, kind, "plain"), gen, 0.3, 0.5)
    return m, form


def host(form):
    gate = form["gate"]
    gate = None if gate is None else gate.float().cpu().numpy() if gate.dim() == 1 else flat(gate)
    return dict(form, gate=gate, **{n: None if form[n] is None else form[n].float().cpu().numpy()
                                    for n in ("gain", "block_gain")})


def same_words(got, want, what):
    g = got.detach().cpu().contiguous()
    w = torch.from_numpy(np.ascontiguousarray(want)).to(g.dtype).reshape(g.shape)
    view = torch.int16 if g.dtype == torch.bfloat16 else torch.int32
    bad = (g.view(view) != w.view(view)).nonzero()
    assert not len(bad), f"{what}: {len(bad)} of {g.numel()} words differ, first at {bad[0].tolist()}"


def near(got, want, size, roundings, what, half_step=0.0):
    """|got - want| <= roundings * U * size, and half a step of the result's type."""
    got = got.detach().double().cpu().numpy().reshape(want.shape)
    tol = roundings * U * size
    tol += half_step * (np.abs(want) + tol)
    assert (np.abs(got - want) <= tol + 1e-37).all(), what


def check(m, form, kind, layout, dy=True):
    b, s, d = m["x"].shape
    half_step = torch.finfo(TYPES[kind]).eps / 2 if kind == "bf16" else 0.0
    y, z = br.repro_residual_norm(m["x"], m["block"], y=empty(b, s, d, kind, layout), out=empty(b, s, d, kind, layout),
                                  **form)
    h = host(form)
    want_y, want_z = so.norm(flat(m["x"]), flat(m["block"]), kind, **h)
    same_words(y, want_y, "y")
    same_words(z, want_z, "z")
    # A sum of D terms: log2(D) + 2 roundings at most, half of them in its
    # root, with four of their own; block: root, two products, gate, two
    # scales, the sum.
    root = (np.log2(d) + 2) / 2 + 4
    y64, z64, size = so.norm64(flat(m["x"]), flat(m["block"]), kind, y=flat(y), **h)
    near(y, y64, size, root + 6, "y", half_step)
    near(z, z64, np.abs(z64), root + 2, "z", half_step)

    got = br.repro_residual_norm_backward(y, m["block"], m["dy"] if dy else None, m["dz"],
                                          dx=empty(b, s, d, kind, layout), dblock=empty(b, s, d, kind, layout), **form)
    got = dict(zip(("dx", "dblock", "dgain", "dblock_gain", "dgate"), got))
    u = flat(m["block"])
    want = so.norm_grad(flat(y), u, flat(m["dy"]) if dy else None, flat(m["dz"]), **h)
    for name, t in got.items():
        if want[name] is None:
            assert t is None, name
        else:
            same_words(t, want[name], name)
    # Y: the sum over the row of |dn y| (log2 D + 4), two roots, six more;
    # behind it the block's own root twice, its sum, and eight more.  Over
    # the rows: 7 levels of the last tree, 2 of a part, at most rows / 512 + 5
    # in turn.
    rows = b * s
    steps = 2 * root + np.log2(d) + 12
    over = rows / 512 + 5 + 9
    for name, (value, size) in so.norm_grad64(flat(y), u, flat(m["dy"]) if dy else None, flat(m["dz"]), **h).items():
        of_rows = value.ndim == 2
        near(got[name], value, size, 2 * steps + root + 10 + (0 if of_rows else over), name,
             half_step if of_rows else 0.0)


CASES = [  # b, s, d, kind, layout, gain, block_norm, gate, x_scale, block_scale
    (1, 1, 1, "f32", "plain", "own", False, None, 1.0, 1.0),
    (1, 1, 1, "bf16", "plain", "own", True, "element", 1.0, 1.0),
    (1, 1, 2048, "bf16", "plain", "own", False, None, 1.0, 1.0),
    (2, 3, 7, "bf16", "offset", "f32", True, "channel", 0.9, 0.5),
    (2, 5, 8, "f32", "packed", None, True, "element", 1.0, 0.5),
    (3, 7, 9, "f32", "seq_first", "bf16", True, "channel", 0.9, 1.0),
    (2, 11, 511, "bf16", "packed", "own", False, "element", 1.0, 1.0),
    (2, 11, 512, "f32", "offset", "own", True, None, 1.0, 1.0),
    (1, 23, 513, "bf16", "plain", "own", True, "channel", 1.0, 1.0),
    (1, 13, 1023, "f32", "plain", None, False, None, 1.0, 0.5),
    (1, 13, 1024, "bf16", "seq_first", "own", True, "element", 1.0, 1.0),
    (3, 5, 1025, "bf16", "offset", "own", True, "channel", 0.5, 2.0),
    (5, 33, 1111, "bf16", "seq_first", "own", True, "element", 1.0, 1.0),
    (1, 700, 1056, "f32", "plain", "own", True, "channel", 1.0, 0.7),
    (1, 9, 2049, "f32", "packed", "own", True, "element", 1.0, 1.0),
    (1, 6, 4096, "bf16", "plain", "f32", True, "channel", 1.0, 1.0),
    (1, 5, 4097, "f32", "offset", "own", True, "channel", 1.0, 1.0),
    (1, 5, 8192, "bf16", "plain", "own", True, "element", 1.0, 1.0),
    (1, 4, 8193, "bf16", "offset", "own", True, "channel", 1.0, 0.5),
    (1, 3, 16384, "f32", "plain", "own", True, "element", 1.0, 1.0),
    (7, 301, 64, "bf16", "packed", "own", False, "channel", 1.0, 1.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_norm_and_gradients(case):
    b, s, d, kind, layout = case[:5]
    m, form = make(*case, seed=sum(case[:3]))
    check(m, form, kind, layout, dy=d != 1024)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(5,), (3, 65), (2, 4, 1030)])
def test_norm_alone(kind, shape):
    gen = torch.Generator().manual_seed(len(shape))
    x = torch.randn(shape, generator=gen).to("cuda", TYPES[kind])
    g = torch.randn(shape[-1], generator=gen).to("cuda")
    dz = torch.randn(shape, generator=gen).to("cuda", TYPES[kind])
    y, z = br.repro_residual_norm(x, gain=g)
    assert y is None
    same_words(z, so.norm(flat(x), None, kind, gain=g.cpu().numpy())[1], "z")
    dx, dblock, dgain, dblock_gain, dgate = br.repro_residual_norm_backward(x, None, None, dz, gain=g)
    assert dblock is None and dblock_gain is None and dgate is None
    want = so.norm_grad(flat(x), None, None, flat(dz), gain=g.cpu().numpy())
    same_words(dx, want["dx"], "dx")
    same_words(dgain, want["dgain"], "dgain")


def test_block_gradient_is_the_streams():
    m, form = make(2, 5, 96, "bf16", "plain", "own", False, None, 0.5, 0.5, seed=3)
    got = br.repro_residual_norm_backward(m["x"], m["block"], m["dy"], m["dz"], **form)
    assert got[1] is got[0]
    apart = br.repro_residual_norm_backward(m["x"], m["block"], m["dy"], m["dz"], dblock=torch.empty_like(m["x"]),
                                            **form)
    assert apart[1] is not apart[0] and torch.equal(apart[1], got[0]) and torch.equal(apart[0], got[0])


def test_in_place():
    for kind, d in (("bf16", 1000), ("f32", 3000), ("bf16", 16000)):
        m, form = make(2, 5, d, kind, "offset", "own", True, "element", 1.0, 0.5, seed=d)
        y, z = br.repro_residual_norm(m["x"], m["block"], **form)
        first = br.repro_residual_norm_backward(y, m["block"], m["dy"], m["dz"], **form)
        x, u, dy, dz, gate = (t.clone() for t in (m["x"], m["block"], m["dy"], m["dz"], form["gate"]))
        now = dict(form, gate=gate)
        again = br.repro_residual_norm(x, u, y=x, out=gate, **now)
        assert again[0] is x and torch.equal(x, y) and torch.equal(gate, z)
        now["gate"] = form["gate"].clone()
        got = br.repro_residual_norm_backward(x, u, dy, dz, dx=dy, dblock=u, dgate=now["gate"], **now)
        assert got[0] is dy and got[1] is u and got[4] is now["gate"]
        for a, b in zip(got, first):
            assert torch.equal(a, b)


def test_no_rows():
    x = torch.empty(0, 4, 24, device="cuda")
    g = torch.ones(24, device="cuda")
    y, z = br.repro_residual_norm(x, x.clone(), gain=g, gate=g, block_norm=True, block_gain=g)
    assert y.shape == z.shape == x.shape
    dx, dblock, dgain, dblock_gain, dgate = br.repro_residual_norm_backward(
        x, x.clone(), x.clone(), x.clone(), gain=g, gate=g, block_norm=True, block_gain=g)
    assert dx.shape == dblock.shape == x.shape
    for t in (dgain, dblock_gain, dgate):
        assert t.shape == (24,) and not t.any()


def test_values_that_are_not_finite_stay_in_their_rows():
    m, form = make(1, 9, 700, "bf16", "plain", "own", True, "channel", 1.0, 1.0, seed=1)
    clean = br.repro_residual_norm(m["x"], m["block"], **form)
    m["x"][0, 2, 5] = float("nan")
    m["block"][0, 4, 699] = float("inf")
    m["x"][0, 6] = 0
    m["block"][0, 6] = 0
    y, z = br.repro_residual_norm(m["x"], m["block"], **form)
    assert z[0, 2].isnan().all() and y[0, 2].isnan().sum() == 1
    assert z[0, 4].isnan().all()
    assert not z[0, 6].any() and not y[0, 6].any()  # eps keeps an empty row's root finite
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(z[0, keep], clean[1][0, keep]) and torch.equal(y[0, keep], clean[0][0, keep])
    dx = br.repro_residual_norm_backward(y, m["block"], m["dy"], m["dz"], **form)[0]
    assert dx[0, keep + [6]].isfinite().all()
