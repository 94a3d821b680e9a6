"""The loss's gradients where the vocabulary ends in the first half of a tile of 256, so that the second half's workgroup
has no entries: the declared words, and nothing of what lies around the operands in them."""
import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import stream_oracle as so
import test_gpu_stream_loss as tl

pytestmark = pytest.mark.gpu


def amid(t, beside):
    """t as a view of rows 3 elements longer, `beside` elements of NaN on either side of it."""
    rows, dim = t.shape
    wide = torch.full((rows * (dim + 3) + 2 * beside,), float("nan"), dtype=t.dtype, device=t.device)
    view = wide[beside:].as_strided((rows, dim), (dim + 3, 1), beside)
    return view.copy_(t)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 16, 17, 64, 65, 200, 256])
@pytest.mark.parametrize("dim", [31, 33, 64, 97])
def test_no_entries_in_a_tiles_second_half(kind, tokens, dim):
    vocab = 256 + 44 + dim % 3
    x, w, labels, dloss = tl.make(tokens, dim, vocab, kind, seed=tokens + dim)
    x, w = amid(x, 5000), amid(w, 300 * 100)
    loss, lse = br.repro_vocab_loss(x, w, labels)
    dx, dw = br.repro_vocab_loss_backward(x, w, labels, lse, dloss)
    hx, hw, hl = tl.host(x), tl.host(w), labels.cpu().numpy()
    want_loss, want_lse = so.vocab_loss(hx, hw, hl, kind)
    tl.same_words(loss, want_loss, "loss")
    tl.same_words(lse, want_lse, "lse")
    want_dx, want_dw = so.vocab_loss_grad(hx, hw, hl, want_lse, tl.host(dloss), kind)
    tl.same_words(dx, want_dx, "dx")
    tl.same_words(dw, want_dw, "dw")
    assert np.isfinite(want_dx).all() and np.isfinite(want_dw).all()
