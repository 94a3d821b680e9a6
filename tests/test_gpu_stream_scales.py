"""Scales without a block: both passes of the norm refuse them alike."""
import pytest
import torch

import bitwise_reproducible_amd as br

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scales", [dict(x_scale=0.5), dict(block_scale=0.5), dict(x_scale=2.0, block_scale=2.0)], ids=str)
@pytest.mark.parametrize("shape", [(16,), (4, 16), (2, 3, 16)])
def test_scales_need_a_block(shape, scales):
    x = torch.randn(shape, device="cuda")
    with pytest.raises(br.ReproError):
        br.repro_residual_norm(x, **scales)
    for dy in (None, x):
        with pytest.raises(br.ReproError):
            br.repro_residual_norm_backward(x, None, dy, x, **scales)
        # Of one, and with a block, they are taken.
        br.repro_residual_norm_backward(x, None, dy, x, x_scale=1.0, block_scale=1.0)
        assert br.repro_residual_norm_backward(x, x, dy, x, **scales)[1] is not None


def test_no_rows_have_any_scale():
    none = torch.empty(0, 16, device="cuda")
    assert br.repro_residual_norm(none, x_scale=0.5)[1].shape == (0, 16)
    assert br.repro_residual_norm_backward(none, None, None, none, x_scale=0.5)[0].shape == (0, 16)
