"""Host logic of the layer operators (CPU only: no call here reaches a kernel)."""
import ctypes
import os
import re
import sys

import numpy as np
import pytest
import torch

import bitwise_reproducible_amd as br
import layer_oracle as lo

sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "bitwise_reproducible_amd", "csrc"))
import build as lib_build  # noqa: E402

SOURCES = ["heads.hip", "heads_grad.hip", "grad_list.hip", "rope_table.hip"]


def test_lanes_partition_every_head():
    # Every place a lane reads lies inside the head, and each element is
    # counted by exactly one lane, for every even head size and rotary part.
    for dim in list(range(2, 300, 2)) + [384, 510, 512]:
        for rotary in range(2, dim + 1, 2):
            for interleaved, kind in ((False, "bf16"), (True, "bf16"), (False, "f32"), (True, "f32")):
                ls = lo.lanes(dim, rotary, interleaved, lo.vector_of(dim, kind))
                assert len(ls) <= 64
                index = np.array([i for i, _ in ls])
                counted = np.array([c for _, c in ls])
                assert index.min() >= 0 and index.max() < dim, (dim, rotary)
                assert sorted(index[counted]) == list(range(dim)), (dim, rotary, interleaved)


# ---------------------------------------------------------------- the binding

F32, BF16 = torch.float32, torch.bfloat16


def _z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


HOST_CASES = {
    "repro_rope_table": lambda: br.repro_rope_table(_z(4, dtype=torch.float64), 8),
    "repro_qk_norm_rope": lambda: br.repro_qk_norm_rope(_z(1, 2, 2, 8), _z(1, 2, 1, 8), _z(2, 4), _z(2, 4)),
    "repro_qk_norm_rope_backward": lambda: br.repro_qk_norm_rope_backward(
        _z(1, 2, 2, 8), _z(1, 2, 1, 8), _z(1, 2, 2, 8), _z(1, 2, 1, 8), _z(2, 4), _z(2, 4)),
    "GradList": lambda: br.GradList([_z(4)]),
    "repro_grad_list_norm": lambda: br.repro_grad_list_norm([_z(4)]),
    "repro_clip_grad_list": lambda: br.repro_clip_grad_list([_z(4)], 1.0),
}


@pytest.mark.parametrize("name", sorted(HOST_CASES))
def test_host_tensor_is_refused(name):
    with pytest.raises(TypeError, match="ROCm device"):
        HOST_CASES[name]()


def test_every_entry_point_is_covered():
    assert set(br.layer.__all__) == set(HOST_CASES)
    for name in br.layer.__all__:
        assert getattr(br, name) is getattr(br.layer, name)
    with pytest.raises(AttributeError):
        br.no_such_entry_point


# ------------------------------------------------------------------- the ABI

P = 4096  # an aligned address that no call below reads


class View(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("seq", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class Args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("seq", ctypes.c_int64), ("heads", ctypes.c_int32 * 2),
                ("dim", ctypes.c_int32), ("rotary", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("gain_dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("position_bytes", ctypes.c_int32),
                ("cos", ctypes.c_void_p), ("sin", ctypes.c_void_p), ("table_rows", ctypes.c_int64),
                ("table_stride", ctypes.c_int64), ("positions", ctypes.c_void_p), ("pos_batch", ctypes.c_int64),
                ("pos_seq", ctypes.c_int64), ("gain", ctypes.c_void_p * 2), ("x", View * 2), ("out", View * 2),
                ("dy", View * 2), ("dgain", ctypes.c_void_p * 2), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


def _args(**changes):
    a = Args(batch=2, seq=3, dim=16, rotary=8, cos=P, sin=P, table_rows=3, table_stride=4, position_bytes=4, eps=1e-6)
    a.heads[:] = [4, 2]
    for i, h in enumerate(a.heads):
        for views in (a.x, a.out, a.dy):
            views[i] = View(P, 3 * h * 16, h * 16, 16)
    for name, value in changes.items():
        if callable(value):
            value(a)
        else:
            setattr(a, name, value)
    return a


def _set(what, i, **fields):
    def change(a):
        for k, v in fields.items():
            setattr(getattr(a, what)[i], k, v)
    return change


def _item(what, i, value):
    def change(a):
        getattr(a, what)[i] = value
    return change


REFUSED = {  # name: (changes, status, also without the backward pass)
    "negative batch": (dict(batch=-1), -1, True),
    "too many tokens": (dict(batch=1 << 20, seq=1 << 20), -1, True),
    "token count wraps": (dict(batch=1 << 40, seq=1 << 40), -1, True),
    "too many heads": (dict(batch=1 << 12, seq=1 << 16, table_rows=1 << 20, c=_item("heads", 0, 1 << 20)), -1, True),
    "negative heads": (dict(c=_item("heads", 1, -1)), -1, True),
    "odd dim": (dict(dim=15), -1, True),
    "dim 0": (dict(dim=0), -1, True),
    "dim too large": (dict(dim=514), -1, True),
    "rotary 0": (dict(rotary=0), -1, True),
    "rotary odd": (dict(rotary=7), -1, True),
    "rotary above dim": (dict(rotary=18, table_stride=9), -1, True),
    "dtype": (dict(dtype=2), -1, True),
    "interleaved": (dict(interleaved=2), -1, True),
    "reserved": (dict(reserved=1), -1, True),
    "eps negative": (dict(eps=-1.0), -1, True),
    "eps nan": (dict(eps=float("nan")), -1, True),
    "eps inf": (dict(eps=float("inf")), -1, True),
    "no cos": (dict(cos=None), -1, True),
    "cos misaligned": (dict(cos=P + 2), -2, True),
    "table stride": (dict(table_stride=3), -1, True),
    "table short": (dict(table_rows=2), -1, True),
    "table wraps": (dict(table_rows=1 << 40, table_stride=1 << 40), -1, True),
    "position size": (dict(positions=P, position_bytes=2), -1, True),
    "position stride": (dict(positions=P, pos_seq=-1), -1, True),
    "position misaligned": (dict(positions=P + 4, position_bytes=8), -2, True),
    "gain dtype": (dict(gain_dtype=5, c=_item("gain", 0, P), d=_item("dgain", 0, P)), -1, True),
    "gain misaligned": (dict(gain_dtype=1, c=_item("gain", 0, P + 1), d=_item("dgain", 0, P)), -2, True),
    "no x": (dict(c=_set("x", 0, data=None)), -1, True),
    "x misaligned": (dict(c=_set("x", 1, data=P + 2)), -2, True),
    "x negative stride": (dict(c=_set("x", 0, seq=-64)), -1, True),
    "x wraps": (dict(c=_set("x", 0, batch=1 << 62)), -1, True),
    "out overlaps": (dict(c=_set("out", 0, head=8)), -1, True),
    "out broadcast": (dict(c=_set("out", 1, batch=0)), -1, True),
    "out tokens cross heads": (dict(c=_set("out", 0, seq=32)), -1, True),
    "no dy": (dict(c=_set("dy", 0, data=None)), -1, False),
    "no dgain": (dict(c=_item("gain", 0, P)), -1, False),
    "dgain misaligned": (dict(c=_item("gain", 0, P), d=_item("dgain", 0, P + 2)), -2, False),
}


@pytest.mark.parametrize("name", sorted(REFUSED))
def test_qk_arguments_are_refused(name):
    lib = br.layer._lib()
    changes, status, forward = REFUSED[name]
    buf = bytes(_args(**changes))
    if forward:
        assert lib.repro_qk_norm_rope(buf, None) == status
    assert lib.repro_qk_norm_rope_backward(buf, P, 1 << 40, None) == status


def test_qk_workspace():
    lib = br.layer._lib()
    assert ctypes.sizeof(Args) == br.layer._load().QK_ARGS_BYTES
    assert lib.repro_qk_norm_rope(None, None) == -1
    assert lib.repro_qk_workspace_bytes(None) == -1
    assert lib.repro_qk_workspace_bytes(bytes(_args(dim=15))) == -1
    assert lib.repro_qk_workspace_bytes(bytes(_args())) == 0
    gains = dict(c=_item("gain", 0, P), d=_item("gain", 1, P), e=_item("dgain", 0, P), f=_item("dgain", 1, P))
    buf = bytes(_args(**gains))
    need = lib.repro_qk_workspace_bytes(buf)
    assert need > 0
    assert lib.repro_qk_norm_rope_backward(buf, P, need - 1, None) == -4
    assert lib.repro_qk_norm_rope_backward(buf, P + 8, need, None) == -2
    assert lib.repro_qk_norm_rope_backward(buf, None, need, None) == -1
    # Nothing to do: no pointer is looked at.
    empty = _args(batch=0, cos=None, sin=None)
    for views in (empty.x, empty.out, empty.dy):
        for i in range(2):
            views[i] = View(None, 0, 0, 0)
    assert lib.repro_qk_norm_rope(bytes(empty), None) == 0
    assert lib.repro_qk_norm_rope_backward(bytes(empty), None, 0, None) == 0


def test_rope_table_arguments():
    f = br.layer._lib().repro_rope_table
    assert f(P, 0, 0, 4, P, P, None) == -1
    assert f(P, 4097, 0, 4, P, P, None) == -1
    assert f(P, 4, -1, 4, P, P, None) == -1
    assert f(P, 4, 0, -1, P, P, None) == -1
    assert f(P, 4, 1 << 31, 1, P, P, None) == -1
    assert f(P, 4, 1, 2**63 - 1, P, P, None) == -1
    assert f(P, 1024, 0, 1 << 31, P, P, None) == -1
    assert f(None, 4, 0, 4, P, P, None) == -1
    assert f(P + 4, 4, 0, 4, P, P, None) == -2
    assert f(P, 4, 0, 4, P + 2, P, None) == -2
    assert f(None, 4, 0, 0, None, None, None) == 0


# --------------------------------------------------------------- list's plan


def _plan(sizes, types, grads=None, outs=None, room=None):
    lib = br.layer._lib()
    n = len(sizes)
    s = (ctypes.c_int64 * n)(*sizes)
    t = (ctypes.c_int32 * n)(*types)
    nbytes = lib.repro_grad_list_bytes(s, t, n)
    if nbytes < 0:
        return int(nbytes), None
    grads = [P * (i + 1) for i in range(n)] if grads is None else grads
    g = (ctypes.c_void_p * n)(*grads)
    o = None if outs is None else (ctypes.c_void_p * n)(*outs)
    host = np.zeros(nbytes + 16, np.uint8)
    skip = -host.ctypes.data % 16
    host = host[skip:skip + nbytes]
    st = lib.repro_grad_list_plan(g, o, s, t, n, host.ctypes.data, nbytes if room is None else room)
    return st, host


TILE = np.dtype([("src", "<u8"), ("dst", "<u8"), ("n", "<i4"), ("bf16", "<i4"), ("index", "<i4"), ("count", "<i4")])


def _read(host):
    head = host[:64].view("<i8")
    tiles, tensors, first, sums = (int(x) for x in head[2:6])
    chunks, most = int(host[48:52].view("<i4")[0]), int(head[7])
    assert int(head[1]) == len(host)
    return dict(tiles=host[64:64 + 32 * tiles].view(TILE), first=host[first:first + 8 * (tensors + 1)].view("<i8"),
                chunks=chunks, most=most, sums=sums, tensors=tensors)


@pytest.mark.parametrize("sizes, types", [
    ([1], [0]), ([0], [1]), ([0, 0, 5], [0, 1, 0]), ([4096, 4097, 8191, 8192, 8193], [0, 0, 1, 1, 1]),
    ([1 << 24, 16384, 16385, 1], [0, 0, 0, 1]), ([1 << 25, 32768, 32769, 0], [1, 1, 1, 0]),
    ([7] * 2000, [i % 2 for i in range(2000)]),
])
def test_plan_covers_every_element_once(sizes, types):
    st, host = _plan(sizes, types, outs=[1 << 40 | P * (i + 1) for i in range(len(sizes))])
    assert st == 0
    plan = _read(host)
    total = sum(n * (2 if t else 4) for n, t in zip(sizes, types))
    assert plan["chunks"] == (16 if total >= 64 << 20 else 4)
    assert plan["first"][0] == 0 and plan["first"][-1] == len(plan["tiles"])
    most = 0
    for i, (n, t) in enumerate(zip(sizes, types)):
        size = 2 if t else 4
        per = 4096 * plan["chunks"] // size
        tiles = plan["tiles"][plan["first"][i]:plan["first"][i + 1]]
        assert len(tiles) == max(1, -(-n // per))
        most = max(most, len(tiles))
        at = np.arange(len(tiles)) * per
        assert (tiles["src"] == P * (i + 1) + at * size).all()
        assert (tiles["dst"] == (1 << 40 | P * (i + 1)) + at * size).all()
        assert (tiles["n"] == np.minimum(per, n - at)).all() and (tiles["bf16"] == t).all()
        assert (tiles["index"] == np.arange(len(tiles))).all() and (tiles["count"] == len(tiles)).all()
    assert plan["most"] == most
    # Room for the tiles' sums, the tensors' and the total.
    assert plan["sums"] + 4 * (len(plan["tiles"]) + len(sizes) + 1) <= len(host)


def test_list_arguments_are_refused():
    lib = br.layer._lib()
    assert _plan([-1], [0])[0] == -1
    assert _plan([1], [2])[0] == -1
    assert _plan([1 << 45], [0])[0] == -1
    assert _plan([1 << 43], [0])[0] == -1  # more tiles than a plan holds
    assert lib.repro_grad_list_bytes(None, None, 1) == -1
    assert lib.repro_grad_list_bytes(None, None, -1) == -1
    assert lib.repro_grad_list_bytes(None, None, (1 << 20) + 1) == -1
    assert _plan([4], [0], grads=[None])[0] == -1
    assert _plan([4], [0], grads=[P + 2])[0] == -2
    assert _plan([4], [1], grads=[P + 2])[0] == 0
    assert _plan([4], [1], grads=[P + 1])[0] == -2
    assert _plan([4], [0], outs=[P + 2])[0] == -2
    assert _plan([4], [0], room=64)[0] == -4
    assert _plan([0], [0], grads=[None])[0] == 0
    st, host = _plan([4], [0])
    head = bytes(host[:64])
    for f, extra in ((lib.repro_grad_list_norm, ()), (lib.repro_clip_grad_list, (1.0,))):
        assert f(None, P, *extra, P, None) == -1
        assert f(head, None, *extra, P, None) == -1
        assert f(head, P, *extra, None, None) == -1
        assert f(head, P + 16, *extra, P, None) == -2
        assert f(head, P, *extra, P + 2, None) == -2
        assert f(b"\0" * 64, P, *extra, P, None) == -1
    assert lib.repro_clip_grad_list(head, P, float("nan"), P, None) == -1


# ------------------------------------------------------------- instructions


@pytest.fixture(scope="module")
def kernels():
    from concurrent.futures import ThreadPoolExecutor
    out = {}
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        for asm in ex.map(lib_build.disassemble, SOURCES):
            scratch = dict(re.findall(r"\.name:\s+(_Z\S+)\n(?:\s+\.[^\n]*\n)*?\s+\.private_segment_fixed_size:\s+(\d+)",
                                      asm))
            for part in re.split(r"\n(?=_Z[^\s:]+:)", asm):
                m = re.match(r"(_Z[^\s:]+):", part)
                if m:
                    body = part.split(".Lfunc_end")[0]
                    out[m.group(1)] = (re.findall(r"^\s+([a-z][a-z0-9_]+)", body, re.M), int(scratch[m.group(1)]))
    assert len(out) >= 20, sorted(out)
    return out


def test_kernels_are_unfused_and_need_no_scratch(kernels):
    # As the other kernels' audit: fused binary32 steps only inside the
    # compiler's correctly rounded division and square root (at most 5 each).
    # k_rope_table computes in binary64; its binary32 steps are those of an
    # integer division.
    for name, (ops, scratch) in kernels.items():
        assert scratch == 0, name
        assert not any(re.match(r"v_pk_(fma|add|mul)_f32", op) for op in ops), name
        assert not any(op.startswith(("flat_", "scratch_")) for op in ops), name
        fused = sum(bool(re.match(r"v_(fma|fmac|mac|mad)_f32|v_(fma|mad)_mix", op)) for op in ops)
        allowed = 5 * (ops.count("v_div_fixup_f32") + ops.count("v_rsq_f32_e32"))
        assert fused <= allowed or "k_rope_table" in name, (name, fused, allowed)


def test_whole_vectors_move_in_sixteen_bytes(kernels):
    for name, (ops, _) in kernels.items():
        if re.search(r"k_heads(_grad)?ILi(1ELi8|0ELi4)E|k_list_(squares|scale)", name):
            assert ops.count("global_load_dwordx4") >= 4, name
        if re.search(r"k_heads(_grad)?ILi(1ELi8|0ELi4)E|k_list_scale", name):
            assert ops.count("global_store_dwordx4") >= 4, name
