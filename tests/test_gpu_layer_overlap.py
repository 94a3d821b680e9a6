"""Outputs that share memory with a call's other tensors are refused through the Python entry points, and what may
be shared is not."""
import pytest
import torch

import bitwise_reproducible_amd as br

pytestmark = pytest.mark.gpu


@pytest.fixture
def m():
    gen = torch.Generator().manual_seed(3)
    q, k, dq, dk = (torch.randn(2, 5, 4, 32, generator=gen).cuda() for _ in range(4))
    f = 5e5 ** (-torch.arange(0, 32, 2, dtype=torch.float64) / 32)
    cos, sin = br.repro_rope_table(f.cuda(), 5)
    gains = [(1 + 0.1 * torch.randn(32, generator=gen)).cuda() for _ in range(2)]
    return dict(q=q, k=k, dq=dq, dk=dk, table=(cos, sin), gains=gains)


def test_shared_outputs_are_refused(m):
    q, k, dq, dk, table, (qg, kg) = (m[n] for n in ("q", "k", "dq", "dk", "table", "gains"))
    new = torch.empty_like(q)
    call, back = br.repro_qk_norm_rope, br.repro_qk_norm_rope_backward
    gains = dict(q_gain=qg, k_gain=kg)
    one = torch.empty(32, device="cuda")
    for f in (
        lambda: call(q, k, *table, q_out=k), lambda: call(q, k, *table, k_out=q),
        lambda: call(q, k, *table, q_out=new, k_out=new), lambda: call(q, q, *table, q_out=q),
        lambda: call(q[:, :4], k[:, :4], *table, q_out=q[:, 1:]),
        lambda: back(q, k, dq, dk, *table, dq=dk), lambda: back(q, k, dq, dk, *table, dq=new, dk=new),
        lambda: back(q, k, dq, dq, *table, dq=dq), lambda: back(q, k, dq, dk, *table, dk=q),
        lambda: back(q, k, dq, dk, *table, **gains, dq_gain=one, dk_gain=one),
        lambda: back(q, k, dq, dk, *table, **gains, dq_gain=new[0, 0, 0], dq=new),
    ):
        with pytest.raises(br.ReproError, match="invalid argument"):
            f()


def test_in_place_and_side_by_side_are_not_refused(m):
    q, k, dq, dk, table, (qg, kg) = (m[n] for n in ("q", "k", "dq", "dk", "table", "gains"))
    gains = dict(q_gain=qg, k_gain=kg)
    want = br.repro_qk_norm_rope_backward(q, k, dq, dk, *table, **gains)
    # Both sides in one buffer: beside each other in each token, and by turns.
    for split in (lambda t: (t[:, :, :4], t[:, :, 4:]), lambda t: (t[:, :, ::2], t[:, :, 1::2])):
        out = split(torch.empty(2, 5, 8, 32, device="cuda"))
        got = br.repro_qk_norm_rope_backward(q, k, dq, dk, *table, **gains, dq=out[0], dk=out[1])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # Over the upstream gradients, over the inputs, and the gains' over the gains.
    a, b, ga, gb = dq.clone(), dk.clone(), qg.clone(), kg.clone()
    got = br.repro_qk_norm_rope_backward(q, k, a, b, *table, q_gain=ga, k_gain=gb, dq=a, dk=b, dq_gain=ga, dk_gain=gb)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(a, want[0]) and torch.equal(ga, want[2])
    a, b = q.clone(), k.clone()
    got = br.repro_qk_norm_rope_backward(a, b, dq, dk, *table, **gains, dq=a, dk=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and torch.equal(a, want[0])
    # The same memory read by both sides, written elsewhere.
    got = br.repro_qk_norm_rope(q, q, *table)
    assert torch.equal(got[0], got[1])
