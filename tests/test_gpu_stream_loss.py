"""The loss over a vocabulary and its gradients on the GPU.

Every result equals the declared order word for word (stream_oracle, on the
CPU oracle's block products) and lies within bounds derived below of the
64-bit definition.
"""
import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import oracle
import stream_oracle as so

pytestmark = pytest.mark.gpu

U = 2.0 ** -24  # a binary32 rounding
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def make(N, D, V, kind, padded=0, ignored=0.2, seed=0, lean=8.0):
    gen = torch.Generator().manual_seed(seed)
    t = TYPES[kind]
    w = (torch.randn(V, D + padded, generator=gen) * D ** -0.5).to(t)
    labels = torch.randint(V, (N,), generator=gen)
    x = torch.randn(N, D + padded, generator=gen)
    x[:, :D] += lean * torch.rand(N, 1, generator=gen) * w[labels, :D].float()
    labels[torch.rand(N, generator=gen) < ignored] = -100
    dloss = torch.rand(N, generator=gen)
    return x.to(t).cuda()[:, :D], w.cuda()[:, :D], labels.cuda(), dloss.cuda()


def host(t):
    return t.detach().float().cpu().numpy()


def same_words(got, want, what):
    g = got.detach().cpu().contiguous()
    w = torch.from_numpy(np.ascontiguousarray(want)).to(g.dtype).reshape(g.shape)
    view = torch.int16 if g.dtype == torch.bfloat16 else torch.int32
    bad = (g.view(view) != w.view(view)).nonzero()
    assert not len(bad), f"{what}: {len(bad)} of {g.numel()} words differ, first at {bad[0].tolist()}"


def test_block_products_are_the_oracles():
    # A wide range of exponents, through the logits of one label each: V = 1
    # makes the loss 0 and lse the logit, to half a step; here the words of
    # the gradient are compared instead, whose product over the tokens starts
    # from dl = -g exactly.
    rng = np.random.default_rng(5)
    for N, D in ((40, 64), (200, 192), (4000, 1024)):
        x = rng.standard_normal((N, D)) * 2.0 ** rng.integers(-12, 13, (N, D))
        x = so.wide16(so.bits16(x.astype(np.float32)))
        w = np.zeros((256, D), np.float32)
        labels = np.zeros(N, np.int64)
        g = so.wide16(so.bits16((rng.standard_normal(N) * 2.0 ** rng.integers(-12, 13, N)).astype(np.float32)))
        lse = np.full(N, 1e4, np.float32)  # so that no other entry has a gradient
        dx, dw = br.repro_vocab_loss_backward(
            torch.from_numpy(x).cuda().bfloat16(), torch.from_numpy(w).cuda().bfloat16(),
            torch.from_numpy(labels).cuda(), torch.from_numpy(lse).cuda(), torch.from_numpy(g).cuda())
        pad = -N % 256
        want = oracle.block_product(so.bits16(np.pad(x.T, ((0, 0), (0, pad)))),
                                    so.bits16(np.pad(-g[None], ((0, 0), (0, pad)))))
        same_words(dw[0], want[:, 0], "dw")
        assert not dw[1:].any() and not dx.any()


CASES = [  # N, D, V, kind, padded, z_weight
    (1, 64, 128, "bf16", 0, 0.0),
    (1, 1, 1, "bf16", 0, 1e-2),
    (1, 200, 1, "f32", 0, 0.0),
    (2, 7, 3, "f32", 3, 1e-4),
    (3, 65, 129, "bf16", 1, 1e-4),
    (33, 128, 1000, "bf16", 0, 1e-3),
    (64, 64, 255, "f32", 0, 1e-4),
    (65, 100, 257, "bf16", 28, 0.0),
    (100, 320, 300, "f32", 0, 1e-4),
    (128, 128, 512, "bf16", 64, 1e-4),
    (129, 72, 513, "bf16", 0, 0.0),
    (257, 64, 700, "f32", 5, 1e-4),
    (300, 257, 640, "bf16", 0, 1e-4),
    (17, 64, 5000, "bf16", 0, 1e-4),  # ten spans
    (5, 33, 4500, "f32", 0, 1e-4),
    (40, 61, 1500, "bf16", 0, 1e-4),  # rows of no vector's alignment, few tokens
    (20, 99, 2100, "f32", 2, 1e-3),
    (130, 64, 3000, "bf16", 0, 0.0),  # three spans
    (270, 40, 1300, "f32", 0, 1e-4),
    (700, 33, 400, "f32", 0, 0.0),
    (520, 64, 300, "bf16", 0, 0.0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_loss_and_gradients(case):
    N, D, V, kind, padded, z = case
    x, w, labels, dloss = make(N, D, V, kind, padded, seed=N + D + V)
    if N % 2:
        labels = labels.int()
    loss, lse = br.repro_vocab_loss(x, w, labels, z_weight=z)
    hx, hw, hl, hg = host(x), host(w), labels.cpu().numpy().astype(np.int64), host(dloss)
    want_loss, want_lse = so.vocab_loss(hx, hw, hl, kind, z)
    same_words(lse, want_lse, "lse")
    same_words(loss, want_loss, "loss")
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, z_weight=z)
    want_dx, want_dw = so.vocab_loss_grad(hx, hw, hl, want_lse, hg, kind, z)
    same_words(dx, want_dx, "dx")
    same_words(dw, want_dw, "dw")

    # 64 bits.  A logit: one rounding of the chain for every eight products
    # (six times as many for binary32), a truncation below a quarter of it, and
    # for binary32 the three smallest products, 3 * 2^-24 together; each
    # relative to the sum of the products' sizes.  lse moves by at most the
    # largest error of a logit, and by p2 (12 roundings, 2 |t| for its argument)
    # and the sums (16 + 3 levels).
    parts = 1 if kind == "bf16" else 6
    ax, aw = np.abs(hx.astype(np.float64)), np.abs(hw.astype(np.float64))
    loss64, lse64, l64 = so.vocab_loss64(hx, hw, hl, z)

    def off(k, sizes):
        return (1.25 * (k / 8 + 8) * parts + 4) * U * sizes

    dl_err = off(D, ax @ aw.T)
    lse_err = dl_err.max(-1) + (40 + 2 * np.abs(l64).max(-1)) * U + U * np.abs(lse64)
    assert (np.abs(host(lse) - lse64) <= lse_err).all()
    assert (np.abs(host(loss) - loss64) <= lse_err + dl_err.max(-1) + 2 * z * np.abs(lse64) * lse_err
            + U * np.abs(loss64)).all()
    dx64, dw64, dl64 = so.vocab_loss_grad64(hx, hw, hl, want_lse, hg, z)
    # dl: relative errors of the exponential (its argument's, c's and 14
    # roundings), the label's subtraction, and half a step of bf16 in dl.
    size = np.abs(dl64) + 2 * np.abs(hg)[:, None] * (np.arange(V)[None] == hl[:, None])
    t = np.abs(l64) + np.abs(want_lse.astype(np.float64))[:, None]
    rel = dl_err + (16 + 3 * t) * U
    step = torch.finfo(torch.bfloat16).eps / 2 if kind == "bf16" else 2 * U
    err = size * (rel + step)
    half = torch.finfo(TYPES[kind]).eps / 2
    T, span = so.spans_of(N, D, V)
    for got, exact, other, e, k in ((dx, dx64, aw, err, min(span, V)), (dw, dw64, ax, err.T, N)):
        sizes = (np.abs(dl64) if k != N or got is dx else np.abs(dl64).T) @ other
        tol = e @ other + off(k, sizes + e @ other) + (V / span + 1) * U * sizes
        tol += half * (np.abs(exact) + tol)
        assert (np.abs(host(got) - exact) <= tol + 1e-30).all()


def test_gradient_against_differences():
    # Central differences of the loss in the direction of the gradient.  The
    # losses are off by some 1e-6 each, 1e-4 of the difference; the third
    # derivative's part is below 1e-3 of it.
    x, w, labels, dloss = make(50, 96, 400, "f32", seed=3)
    loss, lse = br.repro_vocab_loss(x, w, labels, z_weight=1e-3)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, z_weight=1e-3)
    for at, d in ((x, dx), (w, dw)):
        step = 1e-2 / d.norm().item()
        value = []
        for sign in (1, -1):
            moved = [at + sign * step * d if t is at else t for t in (x, w)]
            value.append((br.repro_vocab_loss(*moved, labels, z_weight=1e-3)[0].double() * dloss).sum().item())
        want = d.double().square().sum().item()
        assert abs((value[0] - value[1]) / (2 * step) - want) < 5e-3 * want


def test_one_gradient_for_all_and_strided_ones():
    x, w, labels, dloss = make(70, 64, 300, "bf16", seed=4)
    _, lse = br.repro_vocab_loss(x, w, labels)
    one = torch.tensor(0.125, device="cuda")
    a = br.repro_vocab_loss_backward(x, w, labels, lse, one)
    for many in (torch.full((70,), 0.125, device="cuda"), one.expand(70), torch.full((140,), 0.125, device="cuda")[::2]):
        b = br.repro_vocab_loss_backward(x, w, labels, lse, many)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    spread = torch.full((140,), 7, device="cuda")
    spread[::2] = labels
    b = br.repro_vocab_loss_backward(x, w, spread[::2], lse, one)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_ignored_tokens_and_labels_outside(kind):
    x, w, labels, dloss = make(90, 64, 333, kind, ignored=0.0, seed=6)
    labels[5] = labels[40] = -100
    clean = br.repro_vocab_loss(x, w, labels)
    clean_grads = br.repro_vocab_loss_backward(x, w, labels, clean[1], dloss)
    assert clean[0][5] == 0 and not clean_grads[0][5].any()
    # Whatever an ignored token holds reaches nothing else.
    x[5] = float("nan")
    x[40] = float("inf")
    dloss[5] = float("nan")
    loss, lse = br.repro_vocab_loss(x, w, labels)
    assert torch.equal(loss, clean[0])
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    assert torch.equal(dx, clean_grads[0]) and torch.equal(dw, clean_grads[1])
    # A label outside the vocabulary, either way, is its token's alone.
    for bad in (333, -1, -2 ** 40, 2 ** 40):
        labels[7] = bad
        loss, lse = br.repro_vocab_loss(x, w, labels)
        assert loss[7].isnan() and loss.isnan().sum() == 1
        dx, _ = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
        assert dx[7].isnan().all() and dx.isnan().any(-1).sum() == 1
    # Another index to ignore, one of the vocabulary's own.
    labels[7] = 12
    loss, _ = br.repro_vocab_loss(x, w, labels, ignore_index=12)
    assert loss[7] == 0 and loss[5].isnan()


def test_all_ignored_and_no_tokens():
    x, w, labels, dloss = make(40, 64, 200, "bf16", seed=7)
    labels.fill_(-100)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    assert not loss.any() and not dx.any() and not dw.any()
    for kind in ("bf16", "f32"):
        none = torch.empty(0, 64, device="cuda", dtype=TYPES[kind])
        weight = w.to(TYPES[kind])
        loss, lse = br.repro_vocab_loss(none, weight, labels[:0])
        assert loss.shape == lse.shape == (0,)
        dw = torch.full_like(weight, 3)
        dx, dw = br.repro_vocab_loss_backward(none, weight, labels[:0], lse, dloss[:0], dweight=dw)
        assert dx.shape == (0, 64) and not dw.any()


def test_values_that_are_not_finite():
    x, w, labels, _ = make(20, 64, 300, "bf16", ignored=0.0, seed=8)
    clean = br.repro_vocab_loss(x, w, labels)
    x[3, 10] = float("nan")
    x[4, 20] = float("inf")
    loss, lse = br.repro_vocab_loss(x, w, labels)
    keep = [i for i in range(20) if i not in (3, 4)]
    assert not lse[3].isfinite() and not lse[4].isfinite()
    assert torch.equal(loss[keep], clean[0][keep])
    # Entries that cannot occur (a logit of -inf for every token): as if they
    # were not there.
    x, w, labels, dloss = make(20, 64, 300, "bf16", ignored=0.0, seed=9)
    x[:, 0] = 1.0
    w[:, 0] = 0.0
    labels %= 100
    without = br.repro_vocab_loss(x, w[:128], labels)
    w[128:] = 0.0
    w[128:, 0] = -float("inf")
    loss, lse = br.repro_vocab_loss(x, w, labels)
    assert torch.equal(loss, without[0]) and torch.equal(lse, without[1])


def test_large_logits_keep_their_losses():
    # Logits of some thousands: no term of a block leaves the range.
    x, w, labels, _ = make(30, 64, 500, "f32", ignored=0.0, seed=10)
    loss, lse = br.repro_vocab_loss(x * 300, w * 10, labels)
    loss64, lse64, l64 = so.vocab_loss64(host(x * 300), host(w * 10), labels.cpu().numpy())
    sizes = (np.abs(host(x * 300)).astype(np.float64) @ np.abs(host(w * 10)).astype(np.float64).T).max(-1)
    assert (np.abs(host(lse) - lse64) <= (1.25 * 16 * 6 + 50) * U * sizes).all()
    assert (np.abs(host(loss) - loss64) <= 2 * (1.25 * 16 * 6 + 50) * U * sizes).all()


def test_nothing_is_written_beside_the_outputs():
    for kind, D in (("bf16", 64), ("bf16", 61), ("f32", 67)):
        x, w, labels, dloss = make(37, D, 301, kind, seed=11)
        _, lse = br.repro_vocab_loss(x, w, labels)
        wide_x = torch.full((38, D + 9), 5.0, device="cuda", dtype=TYPES[kind])
        wide_w = torch.full((302, D + 9), 5.0, device="cuda", dtype=TYPES[kind])
        dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, dx=wide_x[:37, 3:3 + D],
                                              dweight=wide_w[:301, 3:3 + D])
        ref = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
        assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
        for wide, rows in ((wide_x, 37), (wide_w, 301)):
            assert (wide[:, :3] == 5).all() and (wide[:, 3 + D:] == 5).all() and (wide[rows:] == 5).all()
