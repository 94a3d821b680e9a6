"""Norm and clipping of gradient lists, and rotation tables, on the GPU."""
import math

import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import layer_oracle as lo

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _grads(sizes, kinds, seed, std=1e-2, tight=False):
    gen = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dtype = TYPES[kinds[i % len(kinds)]]
        t = torch.empty(n + 1, dtype=dtype, device="cuda")[1:] if tight else torch.empty(n, dtype=dtype, device="cuda")
        out.append(t.copy_(torch.randn(n, generator=gen).mul_(std)))
    return out


def _norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def _tree(values):
    return np.float32(lo.tree(np.asarray(values, np.float32)))


def _check(grads, max_norm, outs="new"):
    before = [g.clone() for g in grads]
    dst = None if outs is None else [torch.full_like(g, 7) for g in grads]
    glist = br.GradList(grads, outs=dst)
    only = br.repro_grad_list_norm(glist)
    got = br.repro_clip_grad_list(glist, max_norm)
    torch.cuda.synchronize()
    norm, S, coef = got.cpu().numpy()
    # S is the fold of every tensor's own fold, as repro_grad_norm forms it.
    S_t = [float(br.repro_grad_norm(g.clone())[1]) if g.numel() else 0.0 for g in before]
    want = _tree(S_t) if S_t else np.float32(0)
    assert np.float32(S) == want and norm == np.sqrt(want, dtype=np.float32)
    assert only[0].item() == norm and only[1].item() == S and only[2].item() == 1.0
    # 64 bits: a tree of depth log2(n) and one of log2(tensors), then the
    # root halves the error and rounds once.
    n = max([g.numel() for g in grads] + [1])
    roundings = math.log2(n) + math.log2(max(len(grads), 1)) + 3
    exact = _norm64(before)
    assert abs(float(norm) - exact) <= (roundings / 2 + 1) * 2.0 ** -24 * exact
    # The coefficient and every element: one rounding each.
    c = np.float32(max_norm) / np.float32(norm + np.float32(1e-6))
    assert coef == (min(c, np.float32(1)) if max_norm > 0 else 1)
    for g, b, o in zip(grads, before, glist.outs):
        if coef == 1:
            ref = b
        else:
            ref = torch.from_numpy(lo.mul(b.float().cpu().numpy(), coef)).to(b.dtype).cuda()
        assert torch.equal(o, ref)
        if outs is not None:
            assert torch.equal(g, b)
    return got


LISTS = [
    [1], [0], [0, 0, 3], [5, 1, 0, 7], [2047, 2048, 2049, 8191, 8192, 8193], [4095, 4096, 4097], [100003],
    [2048] * 49, [1 + (i * 7919) % 2500 for i in range(300)], [3] * 1025, [(i * 31) % 40 for i in range(5000)],
    [4096 * 1000 + 1, 5, 0, 4096 * 20], [4096 * 1023, 7], [4096 * 1024, 7], [4096 * (1 + i % 5) + i for i in range(330)],
    [8192 * 3, 4097, 12289, 1] * 60, [16384 * 4096 // 16 + 5, 9, 20000], [16384 * 4097 + 3], [17, 33000000, 16384, 8],
]


@pytest.mark.parametrize("kinds", [("f32",), ("bf16",), ("bf16", "f32")], ids=str)
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{max(s)}")
def test_lists(sizes, kinds):
    print("list", len(sizes), max(sizes), kinds, flush=True)
    grads = _grads(sizes, kinds, seed=len(sizes))
    _check(grads, 0.5)
    _check(grads, 1e6)


@pytest.mark.parametrize("seed", range(12))
def test_random_sweep(seed):
    rng = np.random.default_rng(seed)
    sizes = [int(2 ** rng.uniform(0, rng.choice([6, 12, 19]))) - 1 for _ in range(int(rng.integers(1, 120)))]
    kinds = [str(k) for k in rng.choice(["f32", "bf16"], size=5)]
    print("list sweep", seed, len(sizes), max(sizes), kinds, flush=True)
    _check(_grads(sizes, kinds, seed=seed, tight=bool(seed % 2)), float(rng.choice([0.01, 0.5, 1e5])),
           outs=None if seed % 3 == 0 else "new")


@pytest.mark.parametrize("kinds", [("f32",), ("bf16", "f32")], ids=str)
def test_off_alignment(kinds):
    print("list off alignment", kinds, flush=True)
    _check(_grads([1, 2, 3, 15, 16, 4097, 20011, 70001], kinds, seed=3, tight=True), 0.25)


def test_in_place():
    for max_norm in (0.5, 1e6, 0.0):
        print("in place", max_norm, flush=True)
        _check(_grads([30011, 5, 0, 8192], ("bf16", "f32"), seed=1, tight=True), max_norm, outs=None)


def test_no_tensors():
    glist = br.GradList([])
    assert br.repro_clip_grad_list(glist, 1.0).tolist() == [0.0, 0.0, 1.0]
    assert br.repro_grad_list_norm(glist).tolist() == [0.0, 0.0, 1.0]


def test_values_that_are_not_finite():
    for value, norm, coef in ((float("inf"), float("inf"), 0.0), (float("nan"), float("nan"), float("nan"))):
        grads = _grads([1000, 40], ("f32",), seed=2)
        grads[1][3] = value
        outs = [torch.empty_like(g) for g in grads]
        got = br.repro_clip_grad_list(br.GradList(grads, outs), 1.0)
        want = torch.tensor([norm, norm, coef], device="cuda")
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(5.0), want.nan_to_num(5.0))
        ref = [g * coef for g in grads]
        for o, r in zip(outs, ref):
            assert torch.equal(o.isnan(), r.isnan()) and torch.equal(o.nan_to_num(5.0), r.nan_to_num(5.0))
    # All zero: nothing to clip.
    z = [torch.zeros(77, device="cuda")]
    assert br.repro_clip_grad_list(br.GradList(z), 1.0).tolist() == [0.0, 0.0, 1.0]


def test_one_gradient_twice():
    # Reading a gradient twice is fine where the outs are apart.
    t = torch.ones(16, device="cuda")
    outs = [torch.empty(16, device="cuda"), torch.empty(8, device="cuda")]
    got = br.repro_clip_grad_list(br.GradList([t, t[8:]], outs), 1e6)
    assert got[1].item() == 24.0 and (outs[0] == 1).all() and (outs[1] == 1).all()


def test_moved_tensors_are_refused():
    for move in (lambda t: t.resize_(1 << 16), lambda t: t.set_(torch.zeros(64, device="cuda")), lambda t: t.resize_(8)):
        for side in (0, 1):
            tensors = [torch.ones(64, device="cuda"), torch.ones(64, device="cuda")]
            glist = br.GradList([torch.ones(5, device="cuda"), tensors[0]], [torch.ones(5, device="cuda"), tensors[1]])
            br.repro_clip_grad_list(glist, 1.0)
            move(tensors[side])
            for call in (br.repro_grad_list_norm, lambda g: br.repro_clip_grad_list(g, 1.0)):
                with pytest.raises(ValueError, match="has moved"):
                    call(glist)


def test_bf16_nan_and_largest_survive():
    g = torch.tensor([float("nan"), 3.3895e38, -3.3895e38, 1.0, -0.0], device="cuda").bfloat16()
    out = torch.empty_like(g)
    br.repro_clip_grad_list(br.GradList([g], [out]), 0.0)  # no clip: the bits
    assert torch.equal(out.view(torch.int16), g.view(torch.int16))


def test_refusals():
    t = torch.zeros(16, device="cuda")
    for kind, f in [
        (TypeError, lambda: br.GradList([t.half()])), (TypeError, lambda: br.GradList([t], [t.bfloat16()])),
        (ValueError, lambda: br.GradList([t], [])), (ValueError, lambda: br.GradList([t], [t[:8]])),
        (ValueError, lambda: br.GradList([t[::2]])), (TypeError, lambda: br.GradList([t.cpu()])),
        (TypeError, lambda: br.GradList([t], [t.cpu()])),
        (ValueError, lambda: br.GradList([t, t])), (ValueError, lambda: br.GradList([t[:8], t[4:12]])),
        (ValueError, lambda: br.GradList([t[:8]], [t[4:12]])),
        (ValueError, lambda: br.GradList([t[:4], t[8:12]], [t[8:12], t[12:]])),
        (TypeError, lambda: br.repro_clip_grad_list([t], 1.0)),
        (br.ReproError, lambda: br.repro_clip_grad_list(br.GradList([t]), float("nan"))),
        (ValueError, lambda: br.repro_clip_grad_list(br.GradList([t]), 1.0, out=t[:2])),
        (TypeError, lambda: br.repro_clip_grad_list(br.GradList([t]), 1.0, out=t.double())),
    ]:
        with pytest.raises(kind):
            f()


def test_other_stream_and_graph():
    grads = _grads([40000, 3, 2048, 100], ("bf16", "f32"), seed=6)
    outs = [torch.empty_like(g) for g in grads]
    glist = br.GradList(grads, outs)
    want, want_outs = br.repro_clip_grad_list(glist, 0.5), None
    torch.cuda.synchronize()
    want_outs = [o.clone() for o in outs]
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = br.repro_clip_grad_list(glist, 0.5, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(outs, want_outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = br.repro_clip_grad_list(glist, 0.5)
    for i in range(3):
        for g in grads:
            g.mul_(1.5)
        other = [torch.empty_like(g) for g in grads]
        want = br.repro_clip_grad_list(br.GradList(grads, other), 0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, want) and all(torch.equal(a, b) for a, b in zip(outs, other)), i


# ------------------------------------------------------------------- tables


BITS = 200


def _two_pi():
    """2 pi * 2^BITS as a whole number (pi / 4 = 4 atan(1/5) - atan(1/239))."""
    def atan(x):
        total, term, k = 0, (1 << BITS + 20) // x, 0
        while term:
            total += (term if k % 2 == 0 else -term) // (2 * k + 1)
            term //= x * x
            k += 1
        return total
    return 8 * (4 * atan(5) - atan(239)) >> 20


def _exact_table(f, start, length):
    """80-bit functions of the angle, whose product and reduction are exact whole numbers: at far positions the
    product alone holds more than 80 bits."""
    turn = _two_pi()
    scaled = [n * (1 << BITS) // d for n, d in (float(x).as_integer_ratio() for x in f)]
    left = [[(p * x % turn) >> (BITS - 60) for x in scaled] for p in range(start, start + length)]
    angle = np.array(left, np.int64).reshape(length, len(f)).astype(np.longdouble) * np.longdouble(2.0) ** -60
    return np.cos(angle), np.sin(angle)


@pytest.mark.parametrize("rotary, start, length, theta", [
    (128, 0, 4096, 5e5), (128, 1 << 20, 300, 5e5), (2, 0, 1001, 1e4), (6, 5, 1, 1e4), (10, 0, 3, 1e4), (94, 77, 129, 1e4),
    (64, (1 << 31) - 50, 50, 1e4), (8192, 3, 5, 5e5),
])
def test_tables(rotary, start, length, theta):
    print("table", rotary, start, length, flush=True)
    f = theta ** (-np.arange(0, rotary, 2) / rotary) * 1.0037
    if start + length > 1 << 30:
        f = f / 2.1  # angles up to 2^30
    cos, sin = br.repro_rope_table(torch.from_numpy(f).cuda(), length, start=start)
    for got, want in zip((cos, sin), _exact_table(f, start, length)):
        got = got.cpu().numpy()
        # Half a step of binary32, 2^-24 of the value, and the 64-bit steps
        # before it: a remainder off by 2^-53 + 2^-53 and sums cut at 2.1e-14.
        tol = np.abs(want) * 2.0 ** -24 * (1 + 1e-6) + 3e-14
        assert (np.abs(got - want) <= tol).all()


def test_table_entries_depend_on_the_position_alone():
    f = torch.from_numpy(5e5 ** (-np.arange(0, 46, 2) / 46)).cuda()
    cos, sin = br.repro_rope_table(f, 500)
    for start, length in ((0, 1), (3, 100), (499, 1), (250, 250)):
        c, s = br.repro_rope_table(f, length, start=start)
        assert torch.equal(c, cos[start:start + length]) and torch.equal(s, sin[start:start + length])


def test_table_edges_and_refusals():
    f = torch.tensor([0.0, float("inf"), float("nan"), 1e300, 2.0 ** 31, -1.0], dtype=torch.float64, device="cuda")
    cos, sin = br.repro_rope_table(f, 2)
    assert cos[0, 0] == 1 and sin[0, 0] == 0 and cos[1, 0] == 1 and sin[1, 0] == 0
    assert cos[1, 1:5].isnan().all() and sin[1, 1:5].isnan().all()
    # An angle of zero is zero at position 0, of a frequency that is a number.
    assert cos[0, 3:].tolist() == [1.0, 1.0, 1.0] and cos[0, 1:3].isnan().all()
    assert abs(cos[1, 5].item() - math.cos(1)) < 1e-7 and abs(sin[1, 5].item() + math.sin(1)) < 1e-7
    empty = br.repro_rope_table(f, 0)
    assert empty[0].shape == (0, 6)
    out = torch.empty(2, 6, device="cuda"), torch.empty(2, 6, device="cuda")
    got = br.repro_rope_table(f, 2, cos=out[0], sin=out[1])
    assert got[0] is out[0] and got[1] is out[1]
    for kind, call in [
        (TypeError, lambda: br.repro_rope_table(f.float(), 2)), (TypeError, lambda: br.repro_rope_table(f[::2], 2)),
        (ValueError, lambda: br.repro_rope_table(f, -1)), (br.ReproError, lambda: br.repro_rope_table(f, 2, start=-1)),
        (br.ReproError, lambda: br.repro_rope_table(f, 2, start=1 << 31)),
        (ValueError, lambda: br.repro_rope_table(f, 2, cos=out[0][:1])),
        (TypeError, lambda: br.repro_rope_table(f, 2, cos=out[0].cpu())),
        (br.ReproError, lambda: br.repro_rope_table(f[:0], 2)),
    ]:
        with pytest.raises(kind):
            call()
