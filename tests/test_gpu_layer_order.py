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
