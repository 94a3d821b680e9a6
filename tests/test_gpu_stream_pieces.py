"""The loss and its gradients at sizes that run in several pieces of the vocabulary, with large tiles and with chains of the
widths that models have.

Whole results lie within bounds derived below of 64-bit products on the GPU; samples of tokens (losses, dx) and of
entries (dw) equal the declared order word for word.
"""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import stream_oracle as so
import test_gpu_stream_loss as tl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture
def side_by_side(monkeypatch):
    """so.product in parts of the longer side's rows, which the oracle computes at once."""
    one = so.product

    def product(a, b, kind):
        longer = a if len(a) >= len(b) else b
        edges = np.linspace(0, len(longer), min(16, len(longer)) + 1).astype(int)

        def part(i):
            of = longer[edges[i]:edges[i + 1]]
            return one(of, b, kind) if longer is a else one(a, of, kind)

        with ThreadPoolExecutor(8) as pool:
            return np.concatenate(list(pool.map(part, range(len(edges) - 1))), 0 if longer is a else 1)

    monkeypatch.setattr(so, "product", product)


def pieces_of(N, D, V):
    """(pieces, spans, spans of a piece, large tiles of dw in a whole piece) of the backward pass."""
    T, span = so.spans_of(N, D, V)
    spans, padded = -(-V // span), -(-N // T) * T
    together = min(max(1, 2 ** 27 // (span * padded)), spans)
    tiles = -(-D // 256) * -(-min(together * span, V) // 256)
    return -(-spans // together), spans, together, tiles if padded > 512 else 0


def close_to_64_bits(x, w, labels, loss, lse, dloss, dx, dw, kind, z):
    """Each entry against 64 bits, in blocks of tokens."""
    N, D = x.shape
    V = len(w)
    half = torch.finfo(x.dtype).eps / 2
    parts = 1 if kind == "bf16" else 6

    # As test_gpu_stream_loss derives them, with |x| |w| for a logit's sum of
    # sizes: a rounding for each eight products of a chain, less than a quarter
    # of it for their cuts, four more.
    def off(k):
        return (1.25 * (k / 8 + 8) * parts + 4) * U

    w64 = w.double()
    aw, w_most = w64.abs(), w64.norm(dim=-1).max()
    # dl: half a step of bf16, or two of binary32's.
    step = 2.0 ** -8 if kind == "bf16" else 2 * U
    span = so.spans_of(N, D, V)[1]
    of_dx, of_dw = off(min(span, V)) + (V / span + 1) * U, off(N)
    dw64, dw_tol = torch.zeros_like(w64), torch.zeros_like(w64)
    for first in range(0, N, 2048):
        part = slice(first, first + 2048)
        x64, y, stat = x[part].double(), labels[part], lse[part].double()
        counted = y != -100
        l = x64 @ w64.T
        lse64 = l.logsumexp(-1)
        l_off = off(D) * x64.norm(dim=-1) * w_most
        tol = l_off + (40 + 2 * l.abs().amax(-1)) * U + U * lse64.abs()
        assert ((stat - lse64).abs() <= tol).all()
        picked = l.gather(1, y.clamp(min=0)[:, None])[:, 0]
        want = torch.where(counted, lse64 - picked + z * lse64.square(), 0.0)
        assert ((loss[part].double() - want).abs() <= tol + l_off + 2 * z * lse64.abs() * tol + U * want.abs()).all()
        # The gradients, from lse as it is stored.
        g = torch.where(counted, dloss[part].double(), 0.0)
        t = l.abs().amax(-1) + stat.abs()
        dl = (l - stat[:, None]).exp_() * (g * (1 + 2 * z * stat))[:, None]
        del l
        size = dl.abs()
        rows = torch.arange(len(y), device=y.device)
        dl[rows, y.clamp(min=0)] -= g
        size[rows, y.clamp(min=0)] += 2 * g.abs()
        err = size * (l_off + (16 + 3 * t) * U + step)[:, None]
        err += size * of_dx
        exact, more = dl @ w64, err @ aw
        assert ((dx[part].double() - exact).abs() <= more + half * (exact.abs() + more) + 1e-30).all()
        err += size * (of_dw - of_dx)
        dw64 += dl.T @ x64
        dw_tol += err.T @ x64.abs()
    assert ((dw.double() - dw64).abs() <= dw_tol + half * (dw64.abs() + dw_tol) + 1e-30).all()


def sampled_words(x, w, labels, loss, lse, dloss, dx, dw, kind, z, tokens, entries, columns):
    """The declared words of some tokens and entries."""
    hw, hl, hs, hg = tl.host(w), labels.cpu().numpy(), tl.host(lse), tl.host(dloss)
    N, D = x.shape
    T, span = so.spans_of(N, D, len(hw))
    hx = tl.host(x[tokens])
    want_loss, want_lse = so.vocab_loss(hx, hw, hl[tokens], kind, z)
    tl.same_words(lse[tokens], want_lse, "lse")
    tl.same_words(loss[tokens], want_loss, "loss")

    def dlogits(l, at, entry0):
        """dl of the tokens `at` from their logits l, whose first entry is entry0."""
        c = (hs[at].astype(np.float64) * float.fromhex("0x1.71547652b82fep+0")).astype(np.float32)
        a = (hg[at].astype(np.float64) * (1.0 + 2.0 * float(np.float32(z)) * hs[at].astype(np.float64)))
        d = so.mul(so.p2(so.scaled(l, c[:, None])), a.astype(np.float32)[:, None])
        label = np.arange(entry0, entry0 + l.shape[1])[None] == hl[at][:, None]
        d[label] = so.sub(d, hg[at][:, None])[label]
        d[hl[at] == -100] = 0
        return d

    out = so.fl if kind == "bf16" else lambda t: t
    d = dlogits(so.product(hw, hx, kind).T, tokens, 0)
    sums = None
    for first in range(0, len(hw), span):
        of, by = hw[first:first + span, columns].T, d[:, first:first + span]
        pad = -of.shape[1] % 256
        part = so.product(np.pad(of, ((0, 0), (0, pad))), np.pad(by, ((0, 0), (0, pad))), kind).T
        sums = part if sums is None else so.add(sums, part)
    sums[hl[tokens] == -100] = 0
    tl.same_words(dx[tokens][:, columns], out(sums), "dx")
    every = np.arange(N)
    hx = tl.host(x)
    hx[hl == -100] = 0
    pad = -N % T
    for entry in entries:
        d = dlogits(so.product(hw[entry:entry + 1], tl.host(x), kind).T, every, entry)
        want = so.product(np.pad(hx[:, columns].T, ((0, 0), (0, pad))), np.pad(d.T, ((0, 0), (0, pad))), kind)
        tl.same_words(dw[entry][columns], out(want)[:, 0], f"dw of entry {entry}")


PIECES = [  # N, D, V, kind, padded, z_weight; (pieces, spans, spans of a piece), whether dw's tiles are the large ones
    (16384, 64, 50000, "bf16", 0, 1e-3, (7, 25, 4), False),
    (16384, 2560, 50000, "bf16", 0, 1e-4, (7, 7, 1), True),   # each piece a span, four of whose sums wait
    (4096, 1001, 70000, "bf16", 3, 0.0, (3, 9, 4), True),     # the embedding is copied, in pieces
    (8192, 260, 50000, "f32", 0, 1e-4, (4, 13, 4), False),
    (2048, 600, 200000, "f32", 0, 0.0, (4, 31, 9), True),
    (520, 4096, 4096, "bf16", 0, 0.0, (1, 4, 4), True),       # one piece
    (520, 4096, 4096, "f32", 0, 1e-4, (1, 4, 4), True),
]


@pytest.mark.parametrize("case", PIECES, ids=lambda c: "-".join(map(str, c[:6])))
def test_pieces(case, side_by_side):
    N, D, V, kind, padded, z, shape, large = case
    *found, tiles = pieces_of(N, D, V)
    assert tuple(found) == shape and (tiles >= 256) == large
    x, w, labels, dloss = tl.make(N, D, V, kind, padded, seed=N + V)
    labels[-1] = V - 1  # the last piece's last entry, and the last token, count
    loss, lse = br.repro_vocab_loss(x, w, labels, z_weight=z)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, z_weight=z)
    again = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, z_weight=z)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    del again
    close_to_64_bits(x, w, labels, loss, lse, dloss, dx, dw, kind, z)
    ignored = int((labels == -100).nonzero()[0])
    tokens = np.array([N - 1, ignored] if V < 10000 else [N - 1])
    assert not dx[ignored].any() and loss[ignored] == 0
    columns = np.unique(np.r_[0, np.linspace(0, D - 1, 24).astype(int), D - 1])
    sampled_words(x, w, labels, loss, lse, dloss, dx, dw, kind, z, tokens, [0, V // 2, V - 1], columns)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 20, 100, 300])
@pytest.mark.parametrize("dim", [2048, 2050])
def test_words_of_wide_chains(tokens, dim, kind, side_by_side):
    # A logit's chain of 2048 k, on every kernel's way; some tokens' losses and
    # dx and some entries' dw.
    x, w, labels, dloss = tl.make(tokens, dim, 700, kind, seed=tokens)
    labels[0] = 699
    loss, lse = br.repro_vocab_loss(x, w, labels, z_weight=1e-4)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss, z_weight=1e-4)
    at = np.unique(np.linspace(0, tokens - 1, 6).astype(int))
    columns = np.unique(np.linspace(0, dim - 1, 40).astype(int))
    sampled_words(x, w, labels, loss, lse, dloss, dx, dw, kind, 1e-4, at, [0, 130, 699], columns)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_the_pages_width_and_vocabulary(kind, side_by_side):
    # 128256 entries of width 2048, one token alone and one of 40.
    for tokens in (1, 40):
        x, w, labels, dloss = tl.make(tokens, 2048, 128256, kind, ignored=0.0, seed=tokens)
        loss, lse = br.repro_vocab_loss(x, w, labels, z_weight=1e-4)
        at = [tokens // 2]
        want_loss, want_lse = so.vocab_loss(tl.host(x[at]), tl.host(w), labels[at].cpu().numpy(), kind, 1e-4)
        tl.same_words(lse[at], want_lse, "lse")
        tl.same_words(loss[at], want_loss, "loss")
