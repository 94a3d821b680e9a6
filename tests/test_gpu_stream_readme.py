"""README's example between two blocks and at the end runs as it stands and gives the declared words."""
import pytest
import torch

import bitwise_reproducible_amd as br
import stream_oracle as so
import test_readme_blocks as readme
from test_gpu_stream_norm import flat, same_words

pytestmark = pytest.mark.gpu


def test_example_gives_the_declared_words():
    gen = torch.Generator().manual_seed(2)

    def normal(*shape, mean=0.0):
        return (torch.randn(*shape, generator=gen) + mean).bfloat16().cuda()

    dim, vocab = 72, 300
    space = dict(br=br, x=normal(2, 5, dim), block=normal(2, 5, dim), g=normal(dim, mean=1.0), dim=dim,
                 embedding=normal(vocab, dim), labels=torch.randint(vocab, (10,), generator=gen).cuda(),
                 dloss=torch.rand(10, generator=gen).cuda())
    exec(readme.block("py"), space)
    g, labels = space["g"].float().cpu().numpy(), space["labels"].cpu().numpy()
    y, z = so.norm(flat(space["x"]), flat(space["block"]), "bf16", gain=g)
    y, z = so.rounded(y, "bf16"), so.rounded(z, "bf16")
    same_words(space["y"], y, "y")
    same_words(space["z"], z, "z")
    w = flat(space["embedding"])
    loss, lse = so.vocab_loss(z, w, labels, "bf16", 1e-4)
    same_words(space["loss"], loss, "loss")
    same_words(space["lse"], lse, "lse")
    dz, dw = so.vocab_loss_grad(z, w, labels, lse, space["dloss"].cpu().numpy(), "bf16", 1e-4)
    dz = so.rounded(dz, "bf16")
    same_words(space["dz"], dz, "dz")
    same_words(space["dw"], dw, "dw")
    want = so.norm_grad(y, None, None, dz, gain=g)
    same_words(space["dx"], want["dx"], "dx")
    same_words(space["dg"], want["dgain"], "dg")
    assert space["dblock"] is space["dx"]
