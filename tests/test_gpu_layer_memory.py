"""The layer operators write their outputs and nothing beside them, at odd offsets, in place and past the caches.

Outputs lie in buffers of a fixed pattern with gaps between them; after a call every gap has to hold it still.
"""
import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import layer_oracle as lo
import layer_order
import test_gpu_layer_heads as th

pytestmark = pytest.mark.gpu

PATTERN = 0x5A
TYPES = th.TYPES
SIZE = {"f32": 4, "bf16": 2}


class Buffer:
    """Tensors of odd offsets, with gaps between and around them, in one buffer of bytes."""

    def __init__(self, sizes, kinds, shift):
        starts, at = [], 64
        for i, n in enumerate(sizes):
            size = SIZE[kinds[i % len(kinds)]]
            at = (at + 31) // 16 * 16 + size * (1 + (shift + 2 * i) % (16 // size))  # 1 .. 16 / size elements past a vector
            starts.append((at, n * size, TYPES[kinds[i % len(kinds)]]))
            at += n * size
        self.bytes = torch.full((at + 4096,), PATTERN, dtype=torch.uint8, device="cuda")
        self.gap = torch.ones(at + 4096, dtype=torch.bool, device="cuda")
        self.tensors = []
        for first, count, dtype in starts:
            self.gap[first:first + count] = False
            self.tensors.append(self.bytes[first:first + count].view(dtype))

    def check(self):
        assert (self.bytes[self.gap] == PATTERN).all()


LARGE = [12000001, 4096003, 5, 0, 700001, 16384, 1]  # 67 MB in FP32
SMALL = [4096, 4097, 3, 0, 8193, 1, 20011, 15]
LISTS = [(SMALL, ("f32",)), (SMALL, ("bf16",)), (SMALL, ("bf16", "f32")), (LARGE, ("f32",)),
         (LARGE + [18000007], ("bf16", "f32")), (LARGE[:2] + [18000013, 3], ("bf16",)),
         ([7 + i % 900 for i in range(1300)], ("f32", "bf16"))]


@pytest.mark.parametrize("max_norm", [0.5, 1e9], ids=["clipped", "kept"])
@pytest.mark.parametrize("case", range(len(LISTS)))
def test_lists(case, max_norm):
    sizes, kinds = LISTS[case]
    total = sum(n * SIZE[kinds[i % len(kinds)]] for i, n in enumerate(sizes))
    assert (total >= 64 << 20) == (case in (3, 4, 5))  # the two forms of the kernels
    gen = torch.Generator().manual_seed(case)
    src = Buffer(sizes, kinds, 1)
    for t in src.tensors:
        t.copy_(torch.randn(t.shape, generator=gen).mul_(0.01))
    before = src.bytes.clone()
    want = None
    # To tensors at other offsets, and to such at the same ones.
    for shift in (4, 1):
        print("list", case, sizes[:3], kinds, max_norm, shift, flush=True)
        dst = Buffer(sizes, kinds, shift)
        got = br.repro_clip_grad_list(br.GradList(src.tensors, dst.tensors), max_norm)
        torch.cuda.synchronize()
        dst.check()
        assert torch.equal(src.bytes, before)
        coef = got[2].item()
        assert (coef < 1) == (max_norm == 0.5)
        if want is None:
            want = got
            for t, o in zip(src.tensors, dst.tensors):
                ref = t if coef == 1 else torch.from_numpy(lo.mul(t.float().cpu().numpy(), np.float32(coef))).to(t.dtype)
                assert torch.equal(o.cpu(), ref.cpu())
            outs = [t.clone() for t in dst.tensors]
        assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(dst.tensors, outs))
    print("list in place", case, flush=True)
    glist = br.GradList(src.tensors)
    assert torch.equal(br.repro_grad_list_norm(glist)[:2], want[:2])
    assert torch.equal(src.bytes, before)
    assert torch.equal(br.repro_clip_grad_list(glist, max_norm), want)
    src.check()
    assert all(torch.equal(a, b) for a, b in zip(src.tensors, outs))


class Heads:
    """A (batch, seq, heads, dim) output `further` elements past a vector's border, with gaps after each head, each
    token and each batch."""

    def __init__(self, b, s, h, d, kind, further):
        whole = torch.int16 if kind == "bf16" else torch.int32
        shape = (b, s, h, d)
        strides = (s * (h * (d + 3) + 1) + 5, h * (d + 3) + 1, d + 3, 1)
        self.words = torch.full((b * strides[0] + 2048,), PATTERN, dtype=whole, device="cuda")
        at = 1024 + further
        self.tensor = self.words.view(TYPES[kind]).as_strided(shape, strides, at)
        self.gap = torch.ones_like(self.words, dtype=torch.bool)
        self.gap.as_strided(shape, strides, at).fill_(False)

    def check(self):
        assert (self.words[self.gap] == PATTERN).all()


HEADS = [  # batch, seq, q heads, k heads, dim, rotary
    (2, 9, 5, 2, 128, 128), (1, 7, 3, 1, 128, 36), (2, 5, 3, 2, 40, 10), (1, 4, 2, 1, 2, 2), (1, 3, 2, 1, 14, 6),
    (2, 6, 3, 1, 30, 8), (1, 5, 4, 4, 80, 64), (1, 3, 2, 1, 512, 130), (1, 4, 3, 2, 258, 258), (1, 33, 1, 1, 22, 2),
    (2, 4200, 12, 4, 128, 128), (1, 8201, 12, 5, 122, 50),  # past the caches
]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", HEADS, ids=str)
def test_heads(shape, kind):
    b, s, hq, hk, d, rotary = shape
    assert (b * s * (hq + hk) * d * SIZE[kind] >= 32 << 20) == (s > 1000)
    m = th._make(*shape, kind, "plain", "f32", 0, seed=d)
    table = th._dev(m["cos"]), th._dev(m["sin"])
    gains = dict(q_gain=m["gains"][0], k_gain=m["gains"][1])
    for interleaved in (False, True):
        for further in (0, 1):
            print("heads", shape, kind, interleaved, further, flush=True)
            outs = [Heads(b, s, h, d, kind, further) for h in (hq, hk)]
            want = br.repro_qk_norm_rope(m["q"], m["k"], *table, **gains, interleaved=interleaved)
            br.repro_qk_norm_rope(m["q"], m["k"], *table, **gains, interleaved=interleaved, q_out=outs[0].tensor,
                                  k_out=outs[1].tensor)
            for o, w in zip(outs, want):
                o.check()
                assert torch.equal(o.tensor, w)
            for given in (gains, {}):
                outs = [Heads(b, s, h, d, kind, further) for h in (hq, hk)]
                want = br.repro_qk_norm_rope_backward(m["q"], m["k"], m["dq"], m["dk"], *table, **given,
                                                      interleaved=interleaved)
                room = torch.full((2, d + 64), float(PATTERN), device="cuda")
                more = dict(dq_gain=room[0, 31:31 + d], dk_gain=room[1, 31:31 + d]) if given else {}
                br.repro_qk_norm_rope_backward(m["q"], m["k"], m["dq"], m["dk"], *table, **given, **more,
                                               interleaved=interleaved, dq=outs[0].tensor, dk=outs[1].tensor)
                for o, w in zip(outs, want):
                    o.check()
                    assert torch.equal(o.tensor, w)
                if given:
                    assert torch.equal(room[:, 31:31 + d], torch.stack(want[2:]))
                    assert (room[:, :31] == PATTERN).all() and (room[:, 31 + d:] == PATTERN).all()


def test_workspace_and_table_ends():
    m = th._make(2, 700, 12, 4, 96, 48, "f32", "plain", "f32", 0, seed=1)
    table = th._dev(m["cos"]), th._dev(m["sin"])
    args = (m["q"], m["k"], m["dq"], m["dk"], *table)
    gains = dict(q_gain=m["gains"][0], k_gain=m["gains"][1])
    want = br.repro_qk_norm_rope_backward(*args, **gains)
    rows = sum(layer_order.rows_of(1400, [12, 4], 96, 48, False, "f32")[1])
    need = rows * 96 * 4
    space = torch.full((need + 8192,), PATTERN, dtype=torch.uint8, device="cuda")
    got = br.repro_qk_norm_rope_backward(*args, **gains, workspace=space[:need])
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and (space[need:] == PATTERN).all()
    with pytest.raises(br.ReproError, match="workspace"):
        br.repro_qk_norm_rope_backward(*args, **gains, workspace=space[:need - 16])
    for half, start, length in ((1, 3, 5), (5, 0, 33), (64, 15, 17), (47, 9, 100)):
        f = torch.linspace(0.1, 1.0, half, dtype=torch.float64, device="cuda")
        room = torch.full((2, 33 + half * length + 33), float(PATTERN), device="cuda")
        cos, sin = (r[33:33 + half * length].view(length, half) for r in room)
        br.repro_rope_table(f, length, start=start, cos=cos, sin=sin)
        want = br.repro_rope_table(f, length, start=start)
        assert torch.equal(cos, want[0]) and torch.equal(sin, want[1])
        assert (room[:, :33] == PATTERN).all() and (room[:, 33 + half * length:] == PATTERN).all()
