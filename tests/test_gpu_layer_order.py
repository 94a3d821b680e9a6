"""The orders of the head operators' sums, word for word as the header declares them."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import layer_order
import test_gpu_layer_heads as th

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim, rotary", [(2, 2), (4, 2), (4, 4), (6, 2), (16, 8), (32, 32)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_sums_of_few_groups_are_padded_to_four(dim, rotary, kind):
    # Upstream gradients of -0: the sum of a head's terms is +0 once +0 is
    # added to it, and -0 else, which the sign of dx shows.
    for interleaved in (False, True):
        print("negative zeros", dim, rotary, kind, interleaved, flush=True)
        m = th._make(1, 6, 3, 2, dim, rotary, kind, "plain", None, 0, seed=dim)
        m["dq"].fill_(-0.0)
        m["dk"].copy_(torch.copysign(torch.zeros_like(m["dk"]), m["dk"]))
        cos, sin = m["cos"][m["where"]][:, :, None], m["sin"][m["where"]][:, :, None]
        grads = th._backward(m, interleaved)
        for i, name in enumerate(("q", "k")):
            want = _grad(th._np(m[name]), th._np(m["d" + name]), cos, sin, interleaved, kind)
            th._same_words(grads[i], th._rounded(want, m["dtype"]), name)


def _grad(x, dy, cos, sin, interleaved, kind):
    """lo.heads_grad's dx without gains, with the padded sums."""
    rotary, inv = 2 * cos.shape[-1], np.float32(1) / np.float32(x.shape[-1])
    mean = lo.mul(layer_order.head_sum(lo.mul(x, x), rotary, interleaved, kind), inv)
    r = lo.fl(np.float32(1) / lo.fl(np.sqrt(lo.add(mean, np.float32(th.EPS)), dtype=np.float32)))[..., None]
    ia, ib = lo._pairs(x.shape[-1], rotary, interleaved)
    dz = dy.copy()
    a, b = dy[..., ia], dy[..., ib]
    dz[..., ia] = lo.add(lo.mul(a, cos), lo.mul(b, sin))
    dz[..., ib] = lo.sub(lo.mul(b, cos), lo.mul(a, sin))
    T = layer_order.head_sum(lo.mul(dz, x), rotary, interleaved, kind)[..., None]
    w = lo.mul(lo.mul(lo.mul(T, r), inv), r)
    return lo.mul(lo.sub(dz, lo.mul(x, w)), r)


def _check_gains(m, interleaved, what):
    """Both sides' gain gradients of a call, word for word."""
    print("gain gradients", what, m["shape"], flush=True)
    grads = th._backward(m, interleaved)
    torch.cuda.synchronize()
    cos, sin = m["cos"][m["where"]][:, :, None], m["sin"][m["where"]][:, :, None]
    for i, name in enumerate(("q", "k")):
        if m["gains"][i] is None:
            assert grads[2 + i] is None
            continue
        _, terms = lo.heads_grad(th._np(m[name]), th._np(m["d" + name]), th._np(m["gains"][i]), cos, sin, th.EPS,
                                 interleaved, m["kind"])
        want = layer_order.gain_grad(terms, i, m["shape"][2:4], 2 * cos.shape[-1], interleaved, m["kind"])
        th._same_words(grads[2 + i], torch.from_numpy(want), name + " gain")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", th.SHAPES, ids=str)
def test_gain_gradients(shape, kind, interleaved):
    m = th._make(*shape, kind, "packed", "f32" if shape[1] % 2 else "bf16", 32, seed=sum(shape))
    _check_gains(m, interleaved, kind)
    for i in range(2):  # one side without a gain: its heads count all the same
        one = dict(m, gains=[g if j == i else None for j, g in enumerate(m["gains"])])
        _check_gains(one, interleaved, f"{kind}, side {i} alone")


@pytest.mark.parametrize("shape, kind", [
    # Several turns of every list: 768 rows of 16, 32 and 64 lists, 1280 of 8, 32 and 64, and one row more than the
    # bound, as each side's are rounded up for itself.
    ((1, 9001, 12, 4, 128, 128), "bf16"), ((3, 15001, 5, 2, 64, 64), "bf16"), ((1, 140000, 2, 1, 34, 20), "bf16"),
    ((2, 3001, 7, 3, 128, 96), "f32"), ((1, 60001, 3, 1, 32, 32), "f32"), ((2, 70001, 1, 2, 14, 6), "f32"),
    ((1, 1024, 64, 8, 128, 128), "bf16"), ((1, 6000, 3, 2, 258, 258), "f32"),
], ids=str)
def test_gain_gradients_of_many_heads(shape, kind):
    for interleaved in (False, True):
        _check_gains(th._make(*shape, kind, "plain", "f32", 0, seed=shape[1]), interleaved, kind)


def test_gain_gradients_of_no_heads():
    for shape in ((0, 5, 4, 2, 32, 32), (2, 5, 0, 2, 32, 32), (2, 5, 4, 0, 32, 32)):
        _check_gains(th._make(*shape, "bf16", "plain", "f32", 0, seed=1), False, "empty")
