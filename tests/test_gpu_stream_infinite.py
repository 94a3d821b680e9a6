"""Weights that are infinite, or so large that bf16 rounds them to infinity: an entry that cannot occur in bf16, NaN in
binary32, whose product is one of three bf16 parts, and the words of the declared order just below."""
import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import stream_oracle as so
import test_gpu_stream_loss as tl

pytestmark = pytest.mark.gpu

BORDER = float.fromhex("0x1.ffp+127")


def scored(kind, tokens, value):
    """Tokens whose first element is 1, against 300 entries of which 200 has `value` there and the others 0."""
    x, w, labels, dloss = tl.make(tokens, 40, 300, kind, ignored=0.0, seed=tokens)
    labels %= 200
    x[:, 0], w[:, 0] = 1.0, 0.0
    w[200, 0] = value
    return x, w, labels, dloss


@pytest.mark.parametrize("tokens", [3, 20, 100, 300])
@pytest.mark.parametrize("value", [-float("inf"), -BORDER, float(np.finfo(np.float32).min)], ids=str)
def test_infinite_weights(tokens, value):
    x, w, labels, dloss = scored("f32", tokens, value)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    assert loss.isnan().all() and lse.isnan().all()
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    assert dx.isnan().all() and dw.isnan().all()
    # bf16: the entry is as if it were not there, with 1 for it to be multiplied with.
    x, w, labels, dloss = scored("bf16", tokens, value)
    _, lse = br.repro_vocab_loss(x, w, labels)
    keep = torch.arange(300, device="cuda") != 200
    l = x.double() @ w.double()[keep].T
    lse64 = l.logsumexp(-1)
    # As test_gpu_stream_loss has it, |x| |w| for the sizes of a logit's terms.
    off = (1.25 * (40 / 8 + 8) + 4) * x.double().norm(dim=-1) * w.double()[keep].norm(dim=-1).max()
    assert ((lse - lse64).abs() <= (off + 40 + 2 * l.abs().amax(-1) + lse64.abs()) * 2.0 ** -24).all()


@pytest.mark.parametrize("tokens", [3, 20, 100, 300])
def test_largest_weights_of_finite_parts(tokens):
    value = -float(np.nextafter(np.float32(BORDER), np.float32(0)))
    x, w, labels, dloss = scored("f32", tokens, value)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    want_loss, want_lse = so.vocab_loss(tl.host(x), tl.host(w), labels.cpu().numpy(), "f32")
    assert np.isfinite(want_lse).all()
    tl.same_words(lse, want_lse, "lse")
    tl.same_words(loss, want_loss, "loss")
