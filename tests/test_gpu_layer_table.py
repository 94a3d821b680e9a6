"""Rotation tables within the declared distance of the exact values, near their zeros too."""
import math

import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import test_gpu_layer_list as tl

pytestmark = pytest.mark.gpu

BOUND = 7e-15  # of repro.h: before the rounding to binary32


def _check(f, start, length, what):
    print("table", what, len(f), start, length, flush=True)
    cos, sin = br.repro_rope_table(torch.from_numpy(f).cuda(), length, start=start)
    for got, want in zip((cos, sin), tl._exact_table(f, start, length)):
        got = got.cpu().numpy().astype(np.longdouble)
        # The reference's own error: 2^-60 of the reduced angle, 2^-61 of its
        # 80-bit form and one step of the function, 2e-18 together.
        off = BOUND + 2e-18
        tol = off + (np.abs(want) + off) * np.longdouble(2.0) ** -24  # half a step of binary32
        bad = np.argwhere(np.abs(got - want) > tol)
        assert not len(bad), (what, bad[:3].tolist())


@pytest.mark.parametrize("position", [15, 31, 47, 1039, 4095, 65551, (1 << 20) - 1, (1 << 24) + 14, (1 << 31) - 1])
def test_near_the_zeros(position):
    # Frequencies that bring one position, the last of its sixteen rows or one
    # before it, to within its rounding of a multiple of pi / 2.
    m = np.concatenate([np.arange(1, 41), [97, 1001, 65537, 1 << 20, (1 << 28) + 1]]).astype(np.float64)
    f = m * (math.pi / 2) / position
    f = f[f * (position + 20) < 2.0 ** 30]
    start = max(0, position - 21)
    _check(f, start, min(40, (1 << 31) - start), "zeros")


@pytest.mark.parametrize("start, length", [(0, 3000), (1 << 16, 500), ((1 << 20) + 3, 500), ((1 << 31) - 64, 64)])
def test_all_rows(start, length):
    rng = np.random.default_rng(start % 97)
    top = (2.0 ** 30 - 1) / (start + length)
    f = np.minimum(np.concatenate([5e5 ** (-np.arange(0, 128, 2) / 128), rng.uniform(0, min(top, 8.0), 60),
                                   10.0 ** rng.uniform(-12, 0, 60)]), top)
    _check(f * rng.choice([-1.0, 1.0], len(f)), start, length, "rows")
