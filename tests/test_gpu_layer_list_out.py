"""The statistics of a gradient list may not lie in its tensors' memory."""
import pytest
import torch

import bitwise_reproducible_amd as br

pytestmark = pytest.mark.gpu


def test_out_in_the_list_is_refused():
    flat = torch.ones(64, device="cuda")
    grads, outs = [flat[4:20], flat[:0], flat[32:40].bfloat16()], [flat[40:56], flat[:0], torch.empty(8).bfloat16().cuda()]
    glist = br.GradList(grads, outs)
    half = grads[2].view(torch.float32)
    for call in (br.repro_grad_list_norm, lambda g, out: br.repro_clip_grad_list(g, 0.5, out=out)):
        for bad in (flat[4:7], flat[17:20], flat[2:5], flat[19:22], flat[40:43], flat[53:56], flat[38:41], half[:3]):
            with pytest.raises(ValueError, match="out shares memory with"):
                call(glist, out=bad)
        # Beside the tensors, and larger than three elements, whose rest is not written.
        for good in (flat[:3], flat[1:4], flat[20:23], flat[37:40], flat[20:], flat[56:59]):
            assert call(glist, out=good) is good
            assert good[0].item() == pytest.approx(24 ** 0.5, rel=1e-6) and good[1].item() == 24.0


def test_tensors_laid_out_anew_are_refused():
    def spread(t):  # every other element of a larger buffer: as many, from the same address
        t.as_strided_((64,), (2,))

    def narrow(t):  # as many of another type, at the same address
        t.data = t.data.view(torch.bfloat16)[:64]

    for change in (spread, narrow):
        for side in (0, 1):
            tensors = [torch.ones(128, device="cuda")[:64] for _ in range(2)]
            glist = br.GradList([tensors[0]], [tensors[1]])
            br.repro_clip_grad_list(glist, 1.0)
            change(tensors[side])
            for call in (br.repro_grad_list_norm, lambda g: br.repro_clip_grad_list(g, 1.0)):
                with pytest.raises(ValueError, match="has moved"):
                    call(glist)
