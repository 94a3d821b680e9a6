"""The residual stream's norm and the loss together, as a model's last block uses them, and the ways of calling them:
other streams, threads, captured graphs, rows far apart, memory beside the outputs, refusals."""
import threading

import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import stream_oracle as so
import test_gpu_stream_loss as tl
import test_gpu_stream_norm as tn

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6


class Last:
    """A model's last block: y = x + gate * norm(u) * block_gain, z = norm(y) * gain, the mean loss of z against an
    embedding, and every gradient."""

    def __init__(self, b, s, d, vocab, kind, seed):
        gen = torch.Generator().manual_seed(seed)
        t = tn.TYPES[kind]
        self.kind = kind
        self.x, self.u = (torch.randn(b, s, d, generator=gen).to("cuda", t) for _ in range(2))
        self.gains = [(1 + 0.2 * torch.randn(d, generator=gen)).to("cuda", t) for _ in range(3)]
        self.w = (torch.randn(vocab, d, generator=gen) * d ** -0.5).to("cuda", t)
        self.labels = torch.randint(vocab, (b * s,), generator=gen)
        self.labels[torch.rand(b * s, generator=gen) < 0.2] = -100
        self.labels = self.labels.cuda()
        self.form = dict(gain=self.gains[0], block_gain=self.gains[1], gate=self.gains[2], block_norm=True,
                         block_scale=0.5, eps=EPS)
        self.each = torch.full((), 1.0 / (b * s), device="cuda")

    def run(self, **more):
        y, z = br.repro_residual_norm(self.x, self.u, **self.form, **more)
        rows = z.view(-1, z.shape[-1])
        loss, lse = br.repro_vocab_loss(rows, self.w, self.labels, z_weight=1e-3, **more)
        dz, dw = br.repro_vocab_loss_backward(rows, self.w, self.labels, lse, self.each, z_weight=1e-3, **more)
        grads = br.repro_residual_norm_backward(y, self.u, None, dz.view_as(z), **self.form, **more)
        return [y, z, loss, lse, dw, *grads]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_last_block(kind):
    m = Last(2, 23, 96, 400, kind, seed=1)
    y, z, loss, lse, dw, dx, du, dgain, dblock_gain, dgate = m.run()
    h = dict(m.form, **{n: tn.flat(m.form[n])[0] if m.form[n].dim() > 1 else m.form[n].float().cpu().numpy()
                        for n in ("gain", "block_gain", "gate")})
    want_y, want_z = so.norm(tn.flat(m.x), tn.flat(m.u), kind, **h)
    tn.same_words(y, want_y, "y")
    tn.same_words(z, want_z, "z")
    zw = tl.host(z).reshape(-1, 96)
    labels, w = m.labels.cpu().numpy(), tl.host(m.w)
    want_loss, want_lse = so.vocab_loss(zw, w, labels, kind, 1e-3)
    tl.same_words(loss, want_loss, "loss")
    want_dz, want_dw = so.vocab_loss_grad(zw, w, labels, want_lse, np.full(46, np.float32(1 / 46)), kind, 1e-3)
    tl.same_words(dw, want_dw, "dw")
    want = so.norm_grad(tn.flat(y), tn.flat(m.u), None, so.rounded(want_dz, kind), **h)
    for name, got in (("dx", dx), ("dblock", du), ("dgain", dgain), ("dblock_gain", dblock_gain), ("dgate", dgate)):
        tn.same_words(got, want[name], name)
    if kind == "bf16":
        return

    # The whole, as 64-bit autograd differentiates the formulas.  Relative to a
    # gradient's length: a logit is off by (1.25 (96 / 8 + 8) 6 + 4) U = 154 U
    # of its products' sizes, at most |z| |w| < 20, so dl by 3100 U; dz and the
    # norm's gradient add no more than 500 U; sqrt(96) for products whose
    # lengths cancel: (3100 + 500) * 10 U = 2.2e-3.
    x, u, gain, bgain, gate, wt = (t.double().cpu().requires_grad_()
                                   for t in (m.x, m.u, m.gains[0], m.gains[1], m.gains[2], m.w))

    def norm(t):
        return t * (t.pow(2).mean(-1, keepdim=True) + EPS).rsqrt()

    y64 = x + 0.5 * gate * norm(u) * bgain
    logits = (norm(y64) * gain).view(-1, 96) @ wt.T
    lse64 = logits.logsumexp(-1)
    at = m.labels.cpu()
    each = lse64 - logits.gather(1, at.clamp(min=0)[:, None])[:, 0] + 1e-3 * lse64 ** 2
    each.masked_fill(at < 0, 0).sum().div(46).backward()
    assert (loss.cpu().double() - each.masked_fill(at < 0, 0).detach()).abs().max() <= 2.2e-3
    for got, leaf in ((dx, x), (du, u), (dgain, gain), (dblock_gain, bgain), (dgate, gate), (dw, wt)):
        assert (got.cpu().double() - leaf.grad).norm() <= 2.2e-3 * leaf.grad.norm()


def test_norm_gradients_against_differences():
    # Central differences of the 64-bit definition at steps of 1e-5, whose own
    # error is about 1e-9; the gradients' roundings, about 60 U = 4e-6 of the
    # magnitudes, are far below the 2e-5 that is asked.
    m, form = tn.make(1, 4, 20, "f32", "plain", "own", True, "channel", 0.9, 0.5, seed=6)
    h = tn.host(form)
    args = {"x": tn.flat(m["x"]), "block": tn.flat(m["block"]), "gain": h["gain"], "block_gain": h["block_gain"],
            "gate": h["gate"]}
    args = {k: v.astype(np.float64) for k, v in args.items()}
    dy, dz = (tn.flat(m[n]).astype(np.float64) for n in ("dy", "dz"))

    def value(a):
        y, z, _ = so.norm64(a["x"], a["block"], "f32", **dict(h, gain=a["gain"], block_gain=a["block_gain"],
                                                             gate=a["gate"]))
        return float((y * dy).sum() + (z * dz).sum())

    y, _ = br.repro_residual_norm(m["x"], m["block"], **form)
    got = br.repro_residual_norm_backward(y, m["block"], m["dy"], m["dz"], **form)
    rng = np.random.default_rng(0)
    for name, g in zip(("x", "block", "gain", "block_gain", "gate"), got):
        g = g.double().cpu().numpy().reshape(args[name].shape)
        for _ in range(12):
            at = tuple(rng.integers(n) for n in g.shape)
            step = np.zeros_like(g)
            step[at] = 1e-5
            diff = (value(dict(args, **{name: args[name] + step})) - value(dict(args, **{name: args[name] - step}))) / 2e-5
            assert abs(diff - g[at]) <= 2e-5 * max(np.abs(g).max(), np.abs(dz).max()), (name, at)


def words(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def equal(a, b):
    """The same words, NaN among them (labels outside the vocabulary)."""
    return all((p is None and q is None) or torch.equal(words(p), words(q)) for p, q in zip(a, b))


def test_other_stream_threads_and_one_workspace():
    models = [Last(2, 40, 128, 700, "bf16", 2), Last(3, 77, 99, 1500, "f32", 3), Last(1, 1, 64, 3000, "bf16", 4)]
    want = [m.run() for m in models]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [m.run(stream=side) for m in models]
    side.synchronize()
    assert all(equal(a, b) for a, b in zip(got, want))

    results, errors = [None] * 3, []

    def worker(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(4):
                    results[i] = models[i].run()
            s.synchronize()
        except Exception as e:  # reported in the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors and not any(t.is_alive() for t in threads)
    assert all(equal(a, b) for a, b in zip(results, want))

    # A caller's workspace, with what the last call left in it.
    m = models[1]
    space = torch.full((64 << 20,), 0xff, dtype=torch.uint8, device="cuda")
    z = want[1][1].view(-1, 99)
    for _ in range(2):
        loss, lse = br.repro_vocab_loss(z, m.w, m.labels, z_weight=1e-3, workspace=space)
        dz, dw = br.repro_vocab_loss_backward(z, m.w, m.labels, lse, m.each, z_weight=1e-3, workspace=space)
        grads = br.repro_residual_norm_backward(want[1][0], m.u, None, dz.view_as(m.x), workspace=space, **m.form)
        assert equal([loss, lse, dw, *grads], [want[1][2], want[1][3], *want[1][4:]])


@pytest.mark.parametrize("form", [(2, 40, 128, 700, "bf16"), (3, 77, 99, 1500, "f32"), (1, 1, 64, 3000, "bf16"),
                                  (1, 1100, 64, 300, "bf16")], ids=str)
def test_captured_step_replays_bit_for_bit(form):
    m = Last(*form, seed=5)
    m.run()
    torch.cuda.synchronize()
    graphs, held = [], []
    space = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    rows = m.x.view(-1, m.x.shape[-1])
    for shared in (False, True):  # two graphs, the second with a workspace of the caller's
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            if not shared:
                held.append(m.run())
            else:
                loss, lse = br.repro_vocab_loss(rows, m.w, m.labels, workspace=space)
                held.append([loss, lse, *br.repro_vocab_loss_backward(rows, m.w, m.labels, lse, m.each,
                                                                      workspace=space)])
    for i in range(3):
        m.x.mul_(-1.25)
        m.w.mul_(0.875)
        m.labels.add_(1).clamp_(max=form[3] - 1)
        want = m.run()
        loss, lse = br.repro_vocab_loss(rows, m.w, m.labels, workspace=space)
        alone = [loss, lse, *br.repro_vocab_loss_backward(rows, m.w, m.labels, lse, m.each, workspace=space)]
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert equal(held[0], want) and equal(held[1], alone), i


@pytest.mark.parametrize("case", [
    (1, 2600, 1032, "bf16", "plain", "own", False, None, 1.0, 1.0),  # more rows than workgroups
    (3, 1400, 40, "f32", "plain", "own", False, None, 1.0, 0.5),
    (1, 5003, 200, "bf16", "plain", "own", True, "element", 1.0, 1.0),
    (1, 1500, 1112, "f32", "plain", "own", True, "channel", 1.0, 1.0),
], ids=lambda c: "-".join(map(str, c)))
def test_norm_of_many_rows(case):
    m, form = tn.make(*case, seed=sum(case[:3]))
    tn.check(m, form, case[3], case[4])


def test_norm_writes_nothing_beside_its_outputs():
    for d, kind in ((61, "bf16"), (64, "f32"), (1030, "bf16"), (5, "f32"), (9001, "bf16")):
        t = tn.TYPES[kind]
        m, form = tn.make(2, 3, d, kind, "plain", "own", True, "element", 1.0, 0.5, seed=d)
        wide = [torch.full((2, 4, d + 6), 5.0, dtype=t, device="cuda") for _ in range(5)]
        out = [w[:, :3, 3:3 + d] for w in wide]
        y, z = br.repro_residual_norm(m["x"], m["block"], y=out[0], out=out[1], **form)
        br.repro_residual_norm_backward(y, m["block"], m["dy"], m["dz"], dx=out[2], dblock=out[3], dgate=out[4], **form)
        for w in wide:
            assert (w[..., :3] == 5).all() and (w[..., 3 + d:] == 5).all() and (w[:, 3:] == 5).all()


def test_row_views_with_strides_that_are_zero_or_past_32_bits():
    m, form = tn.make(1, 1, 64, "bf16", "plain", "own", True, "channel", 1.0, 1.0, seed=3)
    x, u = (m[n].expand(3, 5, 64) for n in ("x", "block"))  # one row for all
    want = br.repro_residual_norm(m["x"], m["block"], **form)
    got = br.repro_residual_norm(x, u, **form)
    assert all(torch.equal(g, w.expand(3, 5, 64)) for g, w in zip(got, want))
    stride = (1 << 31) + (1 << 27)  # byte offsets past 2^32
    far = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device="cuda").as_strided((1, 3, 64), (0, stride, 1))
    near = torch.randn(1, 3, 64, device="cuda").bfloat16()
    far.copy_(near)
    want = br.repro_residual_norm(near, near.clone(), **form)
    y, z = br.repro_residual_norm(far, near.clone(), y=far, **form)
    assert y is far and torch.equal(y, want[0]) and torch.equal(z, want[1])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [3, 30, 60, 300])
def test_rows_far_apart(kind, tokens):
    # 2^22 elements between rows, past a tile's reach in 32 bits.
    x, w, labels, dloss = tl.make(tokens, 64, 70, kind, seed=tokens)
    t = tl.TYPES[kind]
    loss, lse = br.repro_vocab_loss(x, w, labels)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    flat = torch.empty((1 << 22) * 70, dtype=t, device="cuda")
    far_w = flat.as_strided((70, 64), (1 << 22, 1))
    far_w.copy_(w)
    far_dw = flat[64:].as_strided((70, 64), (1 << 22, 1))
    got = br.repro_vocab_loss(x, far_w, labels)
    assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
    grads = br.repro_vocab_loss_backward(x, far_w, labels, lse, dloss, dweight=far_dw)
    assert torch.equal(grads[0], dx) and torch.equal(grads[1], dw)
    if tokens <= 60:
        far_x = flat[128:].as_strided((tokens, 64), (1 << 22, 1))
        far_x.copy_(x)
        got = br.repro_vocab_loss(far_x, w, labels)
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse)
        grads = br.repro_vocab_loss_backward(far_x, w, labels, lse, dloss)
        assert torch.equal(grads[0], dx) and torch.equal(grads[1], dw)


def test_refusals():
    x = torch.zeros(2, 3, 16, device="cuda")
    g = torch.ones(16, device="cuda")
    norm, back = br.repro_residual_norm, br.repro_residual_norm_backward
    rows, w = torch.zeros(4, 16, device="cuda"), torch.zeros(9, 16, device="cuda")
    labels, lse = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    loss, grad = br.repro_vocab_loss, br.repro_vocab_loss_backward
    for kind, call in [
        (TypeError, lambda: norm(x.half())), (TypeError, lambda: norm(x.cpu())), (TypeError, lambda: norm(x, x.bfloat16())),
        (ValueError, lambda: norm(x, x[:, :2])), (ValueError, lambda: norm(x.transpose(1, 2))),
        (TypeError, lambda: norm(x, gain=g.double())), (ValueError, lambda: norm(x, gain=g[:8])),
        (TypeError, lambda: norm(x, x, gain=g, gate=g.bfloat16())), (ValueError, lambda: norm(x, x, block_gain=g)),
        (br.ReproError, lambda: norm(x, x, eps=-1.0)), (br.ReproError, lambda: norm(x, x, x_scale=float("inf"))),
        (br.ReproError, lambda: norm(x, x, y=torch.zeros(1, 3, 16, device="cuda").expand(2, 3, 16))),
        (ValueError, lambda: back(x, x, x[:1], x, gain=g)),
        (br.ReproError, lambda: back(x, x, x, x, gain=g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
        (TypeError, lambda: loss(rows.half(), w.half(), labels)), (TypeError, lambda: loss(rows, w.bfloat16(), labels)),
        (ValueError, lambda: loss(rows, w[:, :8], labels)), (ValueError, lambda: loss(rows, w, labels[:3])),
        (TypeError, lambda: loss(rows, w, labels.float())), (TypeError, lambda: loss(rows, w.cpu(), labels)),
        (ValueError, lambda: loss(rows.t(), w, labels)), (br.ReproError, lambda: loss(rows, w, labels, z_weight=float("nan"))),
        (ValueError, lambda: grad(rows, w, labels, lse[:2], lse)), (TypeError, lambda: grad(rows, w, labels, lse, lse.double())),
        (br.ReproError, lambda: grad(rows, w, labels, lse, lse, dx=rows)),
        (br.ReproError, lambda: grad(rows, w, labels, lse, lse, dweight=w)),
        (br.ReproError, lambda: loss(rows, w, labels, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
    ]:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [(-132, 30), (-60, -70)])  # subnormal operands, subnormal products
def test_subnormal_operands_and_results(kind, scale):
    rng = np.random.default_rng(7)
    N, D, V = 48, 64, 256
    x = rng.standard_normal((N, D)) * 2.0 ** (scale[0] + rng.integers(-4, 5, (N, D)))
    g = rng.standard_normal(N) * 2.0 ** (scale[1] + rng.integers(-4, 5, N))
    x, g = so.rounded(x.astype(np.float32), kind), so.rounded(g.astype(np.float32), "bf16")
    t = tl.TYPES[kind]
    w = torch.zeros(V, D, dtype=t, device="cuda")
    labels = torch.zeros(N, dtype=torch.int64, device="cuda")
    lse = torch.full((N,), 1e4, device="cuda")  # so that no other entry has a gradient
    hx, hg = torch.from_numpy(x).to(t).cuda(), torch.from_numpy(g).cuda()
    dx, dw = br.repro_vocab_loss_backward(hx, w, labels, lse, hg)
    want_dx, want_dw = so.vocab_loss_grad(x, tl.host(w), np.zeros(N, np.int64), tl.host(lse), g, kind)
    tl.same_words(dw, want_dw, "dw")
    tl.same_words(dx, want_dx, "dx")
    # The logits themselves, from a vocabulary of one.
    one = torch.full((1, D), 2.0 ** 126, dtype=t, device="cuda")
    loss, got = br.repro_vocab_loss(hx, one, labels)
    want_loss, want = so.vocab_loss(x, tl.host(one), np.zeros(N, np.int64), kind)
    tl.same_words(got, want, "lse")
    tl.same_words(loss, want_loss, "loss")


def test_more_tiles_than_one_launch_holds():
    # 2^20 tokens and 2^19 entries: 2^23 tiles of 512 threads.
    x = torch.zeros(1 << 20, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1 << 19, 64, dtype=torch.bfloat16, device="cuda")
    labels = torch.arange(1 << 20, device="cuda") % (1 << 19)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    want = float(np.float32(19 * np.log(2.0)))
    assert (lse == want).all() and (loss == want).all()
    del loss, lse
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tokens", [16, 17, 64, 125, 256, 300])
def test_embedding_that_ends_in_a_tiles_first_half(tokens):
    # 7700 entries are 20 past a multiple of 256: the second block of the last
    # tile has none.  Rows of 15 KB, so that a read of that block would leave
    # the embedding by 2 MB.
    D, V = 3852, 7700
    x, w, labels, dloss = tl.make(tokens, D, V, "f32", ignored=0.0, seed=tokens)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    l = x.double() @ w.double().T
    lse64 = l.logsumexp(-1)
    # Relative to the sizes of what a product adds (|x| |w| for a logit): a
    # rounding for each eight of six parts' terms and three more.
    off = (1.25 * (D / 8 + 8) * 6 + 4) * U * (x.double().norm(dim=-1) * w.double().norm(dim=-1).max())
    assert ((lse - lse64).abs() <= off + 100 * U * lse64.abs()).all()
    dl = (l - lse64[:, None]).exp()
    dl[torch.arange(tokens), labels] -= 1
    dl *= dloss.double()[:, None]
    # An error of 2 off in each entry's exponent, and the products' own.
    more = 2 * off.max() + (1.25 * (V / 8 + 8) * 6 + 100) * U
    for got, want, sizes in ((dx, dl @ w.double(), dl.abs() @ w.double().abs()),
                             (dw, dl.T @ x.double(), dl.abs().T @ x.double().abs())):
        label = torch.zeros_like(l)
        label[torch.arange(tokens), labels] = dloss.double()
        sizes = sizes + (label @ w.double().abs() if got is dx else label.T @ x.double().abs())
        assert ((got - want).abs() <= more * sizes + 1e-30).all()


def test_norm_of_tensors_larger_than_the_caches():
    # From 128 MB on the stores bypass the caches: the same words as in parts.
    rows, d = 32768 + 8, 2056
    x, u, dy, dz = (torch.randn(rows, d, device="cuda").bfloat16() for _ in range(4))
    g = torch.rand(d, device="cuda").bfloat16()
    form = dict(gain=g, block_gain=g, gate=g, block_norm=True, block_scale=0.5)
    y, z = br.repro_residual_norm(x, u, **form)
    dx, du = br.repro_residual_norm_backward(y, u, dy, dz, **form)[:2]
    for part in (slice(0, 9000), slice(9000, 20000), slice(20000, rows)):
        want = br.repro_residual_norm(x[part], u[part], **form)
        assert torch.equal(y[part], want[0]) and torch.equal(z[part], want[1])
        want = br.repro_residual_norm_backward(y[part], u[part], dy[part], dz[part], **form)
        assert torch.equal(dx[part], want[0]) and torch.equal(du[part], want[1])


def smallest(call, most):
    """The least workspace that `call` takes, in bytes."""
    low, high = 0, most
    while low < high:
        at = (low + high) // 2
        try:
            call(torch.empty(at, dtype=torch.uint8, device="cuda"))
            high = at
        except br.ReproError:
            low = at + 1
    return low


@pytest.mark.parametrize("form", [(1, 64, 300, "bf16"), (40, 61, 1500, "bf16"), (333, 130, 900, "bf16"),
                                  (5, 33, 700, "f32"), (30, 70, 2100, "f32"), (300, 64, 520, "f32")], ids=str)
def test_nothing_is_written_beside_the_smallest_workspace(form):
    x, w, labels, dloss = tl.make(*form, seed=9)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    want = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    for call in (lambda s: br.repro_vocab_loss(x, w, labels, workspace=s),
                 lambda s: br.repro_vocab_loss_backward(x, w, labels, lse, dloss, workspace=s)):
        size = smallest(call, 64 << 20)
        space = torch.full((size + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
        got = call(space[4096:4096 + size])
        assert (space[:4096] == 0x5a).all() and (space[4096 + size:] == 0x5a).all()
    assert equal(got, want)
    m, norm = tn.make(3, 400, 65, form[3], "plain", "own", True, "channel", 1.0, 1.0, seed=4)
    y, _ = br.repro_residual_norm(m["x"], m["block"], **norm)

    def back(s):
        return br.repro_residual_norm_backward(y, m["block"], m["dy"], m["dz"], workspace=s, **norm)

    size = smallest(back, 8 << 20)
    space = torch.full((size + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
    got = back(space[4096:4096 + size])
    assert (space[:4096] == 0x5a).all() and (space[4096 + size:] == 0x5a).all()
    assert equal(got, back(None))


@pytest.mark.parametrize("seed", range(24))
def test_random_norms(seed):
    rng = np.random.default_rng(seed)
    kind = str(rng.choice(["f32", "bf16"]))
    b, s = int(rng.integers(1, 5)), int(rng.integers(1, 40))
    d = int(rng.choice([rng.integers(1, 40), rng.integers(40, 1100), rng.integers(1000, 4500)]))
    layout = str(rng.choice(["plain", "packed", "seq_first", "offset"]))
    norm = bool(rng.integers(2))
    gate = [None, "channel", "element"][rng.integers(3)]
    gain = [None, "own", "f32", "bf16"][rng.integers(4)]
    m, form = tn.make(b, s, d, kind, layout, gain, norm, gate, float(rng.choice([1.0, 0.9])),
                      float(rng.choice([1.0, 0.5])), seed=seed)
    tn.check(m, form, kind, layout, dy=bool(rng.integers(2)))


@pytest.mark.parametrize("seed", range(24))
def test_random_losses(seed):
    rng = np.random.default_rng(100 + seed)
    kind = str(rng.choice(["f32", "bf16"]))
    N = int(rng.choice([rng.integers(1, 20), rng.integers(17, 140), rng.integers(120, 600)]))
    D = int(rng.choice([rng.integers(1, 70), 64, 128, rng.integers(60, 300)]))
    V = int(rng.choice([rng.integers(1, 140), rng.integers(100, 1400), rng.integers(1000, 2600)]))
    z = float(rng.choice([0.0, 1e-4, 1e-2]))
    x, w, labels, dloss = tl.make(N, D, V, kind, int(rng.integers(0, 9)), seed=seed)
    loss, lse = br.repro_vocab_loss(x, w, labels, z_weight=z)
    hx, hw, hl, hg = tl.host(x), tl.host(w), labels.cpu().numpy(), tl.host(dloss)
    want_loss, want_lse = so.vocab_loss(hx, hw, hl, kind, z)
    tl.same_words(lse, want_lse, "lse")
    tl.same_words(loss, want_loss, "loss")
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, z_weight=z)
    want_dx, want_dw = so.vocab_loss_grad(hx, hw, hl, want_lse, hg, kind, z)
    tl.same_words(dx, want_dx, "dx")
    tl.same_words(dw, want_dw, "dw")
