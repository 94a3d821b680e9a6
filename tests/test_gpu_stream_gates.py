"""A row of its own, (dim), has a gate of its own shape and type; rows of more dimensions tell a vector for the channels
from one for each element."""
import pytest
import torch

import bitwise_reproducible_amd as br

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16], ids=str)
def test_gates_of_one_row(kind):
    gen = torch.Generator().manual_seed(4)
    x, u, gate, dz = (torch.randn(70, generator=gen).to("cuda", kind) for _ in range(4))
    gain = torch.randn(70, generator=gen).cuda()
    y, z = br.repro_residual_norm(x, u, gain=gain, gate=gate)
    got = br.repro_residual_norm_backward(y, u, None, dz, gain=gain, gate=gate)
    assert [t.dtype for t in (y, z, got[0], got[1], got[2], got[4])] == [kind] * 4 + [torch.float32, kind]
    # As one row of two dimensions with a gate for each element.
    y2, z2 = br.repro_residual_norm(x[None], u[None], gain=gain, gate=gate[None])
    want = br.repro_residual_norm_backward(y2, u[None], None, dz[None], gain=gain, gate=gate[None])
    assert torch.equal(y, y2[0]) and torch.equal(z, z2[0])
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b.view(70))
    # A vector for the channels: of the gains' type, its gradient in binary32.
    y3, _ = br.repro_residual_norm(x[None], u[None], gain=gain, gate=gate.float())
    assert torch.equal(y3, y2)
    dgate = br.repro_residual_norm_backward(y3, u[None], None, dz[None], gain=gain, gate=gate.float())[4]
    assert dgate.dtype == torch.float32 and torch.equal(dgate.to(kind), got[4])
    if kind is torch.bfloat16:
        with pytest.raises(TypeError):
            br.repro_residual_norm(x, u, gain=gain, gate=gate.float())
