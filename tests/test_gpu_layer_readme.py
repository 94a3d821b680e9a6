"""README's Python example runs as it stands, and clips the gradients of every step."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_example_clips_every_step():
    with open(README) as fh:
        code, = re.findall(r"```python\n(.*?)```", fh.read(), re.S)
    gen = torch.Generator().manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=gen).cuda()

    params = [normal(40, 30).requires_grad_(), normal(30).requires_grad_()]
    optimizer = torch.optim.SGD(params, lr=1e-3)
    norms = []

    class Optimizer:
        def zero_grad(self, *args, **kw):
            optimizer.zero_grad(*args, **kw)

        def step(self):
            # What the optimizer is given has been clipped.
            total = torch.stack([p.grad.double().square().sum() for p in params]).sum().sqrt().item()
            norms.append(total)
            optimizer.step()

    def loss(x):
        return 7 * (x @ params[0] + params[1]).square().sum()

    space = dict(torch=torch, seq=6, inv_freq=5e5 ** (-torch.arange(0, 32, 2, dtype=torch.float64).cuda() / 32),
                 q=normal(2, 6, 4, 32), k=normal(2, 6, 2, 32), gq=normal(32), gk=normal(32), dq_out=normal(2, 6, 4, 32),
                 dk_out=normal(2, 6, 2, 32), params=params, optimizer=Optimizer(), loss=loss,
                 batches=[normal(5, 40) for _ in range(3)])
    exec(code, space)
    # A coefficient of 1 / (norm + 1e-6), products and norm: a few roundings of binary32.
    assert norms == pytest.approx([1.0] * 3, rel=1e-5)
