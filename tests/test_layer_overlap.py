"""Outputs of the layer operators that share memory with anything else of the call are refused (CPU only).

Every call here is refused before a kernel is launched.
"""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

import bitwise_reproducible_amd as br

CSRC = os.path.join(os.path.dirname(br.__file__), "csrc")
SHIM = """
#include "views.h"
using repro::View;
static View view(uintptr_t first, int64_t run, int dims, const int64_t* size, const int64_t* stride) {
  View v((const void*)first, run);
  for (int d = 0; d < dims; ++d) v.dimension(size[d], stride[d]);
  return v;
}
extern "C" int share(uintptr_t a, int64_t an, int ad, const int64_t* as, const int64_t* at, uintptr_t b, int64_t bn,
                     int bd, const int64_t* bs, const int64_t* bt) {
  return repro::share_memory(view(a, an, ad, as, at), view(b, bn, bd, bs, bt));
}
"""


@pytest.fixture(scope="module")
def share(tmp_path_factory):
    d = tmp_path_factory.mktemp("views")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o",
                    str(lib)], check=True)
    f = ctypes.CDLL(str(lib)).share
    word = ctypes.c_int64
    row = [ctypes.c_uint64, word, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    f.argtypes = row + row

    def call(a, b):
        flat = []
        for first, run, dims in (a, b):
            flat += [first, run, len(dims), (word * 3)(*(n for n, _ in dims)), (word * 3)(*(s for _, s in dims))]
        return bool(f(*flat))

    return call


def _bytes(view):
    first, run, dims = view
    at = {first + sum(i * s for i, (_, s) in zip(index, dims))
          for index in itertools.product(*(range(n) for n, _ in dims))}
    return {x + k for x in at for k in range(run)}


def test_sharing_is_found_exactly(share):
    # Against the sets of bytes themselves: small random views, among them
    # ones with equal, nested, crossing and zero strides, and empty ones.
    rng = random.Random(7)
    seen = {True: 0, False: 0}
    for _ in range(20000):
        common = [rng.choice([1, 2, 3, 4, 6, 8, 12, 24, 40]) for _ in range(3)]
        views = []
        for _ in range(2):
            dims = [(rng.choice([1, 2, 2, 3, 4, 5, 0 if rng.random() < 0.05 else 3]),
                     rng.choice([s, s, s, rng.randint(0, 50)])) for s in common]
            views.append((1000 + rng.randint(0, 60), rng.choice([1, 2, 2, 3, 4, 8]), dims))
        want = bool(_bytes(views[0]) & _bytes(views[1]))
        seen[want] += 1
        assert share(*views) == want, views
        assert share(*views[::-1]) == want, views
    assert min(seen.values()) > 2000, seen


def test_sides_of_one_projection(share):
    # Queries and keys beside each other in every token, in a whole batch:
    # apart, and one element further into each other.
    for size, d, hq, hk, s, b in ((2, 128, 16, 4, 4096, 4), (4, 80, 12, 4, 1037, 3), (2, 2, 1, 1, 70000, 64)):
        row = (hq + hk) * d * size
        dims = lambda h: [(b, s * row), (s, row), (h, d * size)]  # noqa: E731
        q = (1 << 40, d * size, dims(hq))
        assert not share(q, ((1 << 40) + hq * d * size, d * size, dims(hk)))
        assert share(q, ((1 << 40) + hq * d * size - size, d * size, dims(hk)))
        # Heads before tokens in the same memory: the same bytes in another order.
        first = (1 << 40, d * size, [(b, s * row), (s, d * size), (hq + hk, s * d * size)])
        assert share(q, first) and share(first, (1 << 40, d * size, dims(hk)))
        # Every other head, and every other token.
        if hq % 2 == 0:
            even, odd = ((1 << 40) + i * d * size for i in (0, 1))
            assert not share((even, d * size, [(b, s * row), (s, row), (hq // 2, 2 * d * size)]),
                             (odd, d * size, [(b, s * row), (s, row), (hq // 2, 2 * d * size)]))
        assert not share((1 << 40, d * size, [(s // 2, 2 * row), (hq, d * size)]),
                         ((1 << 40) + row, d * size, [(s // 2, 2 * row), (hq, d * size)]))


def test_far_strides_do_not_wrap(share):
    far = 1 << 61
    assert share((64, 8, [(3, far)]), (64 + far, 8, [(2, far)]))
    assert not share((64, 8, [(3, far)]), (72 + far, 8, [(2, far)]))


# ------------------------------------------------------------------- the ABI

BLOCK = 1 << 32  # apart from any other address used here


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


BATCH, SEQ, HEADS, DIM = 2, 3, 4, 16  # as many keys as queries, in FP32


def _args(shared):
    """A call whose tensors lie apart, but for `shared`: {(name, side): (name, side, elements further)}."""
    places = {}

    def place(name, side):
        return (1 + sorted(NAMES).index((name, side))) * BLOCK

    for key in NAMES:
        places[key] = place(*key)
    for key, (name, side, further) in shared.items():
        places[key] = place(name, side) + 4 * further
    a = Args(batch=BATCH, seq=SEQ, dim=DIM, rotary=8, cos=places["cos", 0], sin=places["sin", 0], table_rows=SEQ,
             table_stride=4, positions=places["positions", 0], position_bytes=4, pos_batch=SEQ, pos_seq=1, eps=1e-6)
    for k in range(2):
        a.heads[k] = HEADS
        a.gain[k], a.dgain[k] = places["gain", k], places["dgain", k]
        for name in ("x", "out", "dy"):
            getattr(a, name)[k] = View(places[name, k], SEQ * HEADS * DIM, HEADS * DIM, DIM)
    return bytes(a), places["workspace", 0]


NAMES = [(n, k) for n in ("x", "out", "dy", "gain", "dgain") for k in range(2)]
NAMES += [(n, 0) for n in ("cos", "sin", "positions", "workspace")]
HEAD_BYTES = BATCH * SEQ * HEADS * DIM

FORWARD = {  # name: memory that two of the call's tensors share
    "queries out over keys": {("out", 0): ("x", 1, 0)},
    "keys out over queries": {("out", 1): ("x", 0, 0)},
    "one output twice": {("out", 1): ("out", 0, 0)},
    "outputs a token into each other": {("out", 1): ("out", 0, HEADS * DIM)},
    "in place, one head further": {("out", 0): ("x", 0, DIM)},
    "in place over an input of both sides": {("x", 1): ("x", 0, 0), ("out", 0): ("x", 0, 0)},
    "out over the last element of the input": {("out", 0): ("x", 0, HEAD_BYTES - 1)},
    "out over cosines": {("out", 0): ("cos", 0, 0)},
    "out over sines": {("out", 1): ("sin", 0, 11)},
    "out over positions": {("out", 0): ("positions", 0, 5)},
    "out over a gain": {("out", 1): ("gain", 0, 15)},
}
BACKWARD = {
    "gradient over the other side's upstream": {("out", 0): ("dy", 1, 0)},
    "keys' gradient over the queries' upstream": {("out", 1): ("dy", 0, 0)},
    "upstream, one element further": {("out", 1): ("dy", 1, 1)},
    "one gain gradient twice": {("dgain", 1): ("dgain", 0, 0)},
    "gain gradients into each other": {("dgain", 1): ("dgain", 0, 15)},
    "gain gradient over the other's gain": {("dgain", 0): ("gain", 1, 0)},
    "gain gradient over its gain, further": {("dgain", 0): ("gain", 0, 1)},
    "gain gradient in an output": {("dgain", 0): ("out", 1, 40)},
    "gain gradient in an input": {("dgain", 1): ("x", 1, HEAD_BYTES - 1)},
    "gain gradient in the workspace": {("dgain", 0): ("workspace", 0, 3)},
    "output in the workspace": {("out", 0): ("workspace", 0, 0)},
    "input in the workspace": {("x", 0): ("workspace", 0, 8)},
    "cosines in the workspace": {("cos", 0): ("workspace", 0, 0)},
}


@pytest.mark.parametrize("name", sorted(FORWARD) + sorted(BACKWARD))
def test_shared_memory_is_refused(name):
    lib = br.layer._lib()
    buf, workspace = _args({**FORWARD, **BACKWARD}[name])
    if name in FORWARD:
        assert lib.repro_qk_norm_rope(buf, None) == -1
    need = lib.repro_qk_workspace_bytes(buf)
    assert 64 <= need < BLOCK
    assert lib.repro_qk_norm_rope_backward(buf, workspace, need, None) == -1


@pytest.mark.parametrize("cos, sin", [(0, 0), (0, 60), (60, 0), (-BLOCK, 64), (-BLOCK + 28, 64), (64, -BLOCK - 60)])
def test_table_outputs_are_apart(cos, sin):
    # Four frequencies at BLOCK, 4 x 4 entries of 4 bytes at 2 * BLOCK and on.
    assert br.layer._lib().repro_rope_table(BLOCK, 4, 0, 4, 2 * BLOCK + cos, 2 * BLOCK + sin, None) == -1


def test_list_statistics_are_apart_from_the_plan():
    lib = br.layer._lib()
    sizes, kinds, grads = (ctypes.c_int64 * 2)(5000, 3), (ctypes.c_int32 * 2)(0, 1), (ctypes.c_void_p * 2)(BLOCK, BLOCK)
    nbytes = lib.repro_grad_list_bytes(sizes, kinds, 2)
    room = (ctypes.c_char * (nbytes + 16))()
    host = ctypes.addressof(room) + -ctypes.addressof(room) % 16
    assert lib.repro_grad_list_plan(grads, None, sizes, kinds, 2, host, nbytes) == 0
    plan = 2 * BLOCK
    for out3 in (plan, plan - 8, plan + nbytes // 2 // 4 * 4, plan + nbytes - 4):
        assert lib.repro_grad_list_norm(host, plan, out3, None) == -1
        assert lib.repro_clip_grad_list(host, plan, 1.0, out3, None) == -1
