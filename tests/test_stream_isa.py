"""Instruction audit of the residual stream's and the loss's kernels (CPU only: hipcc emits the gfx950 assembly of our
sources, nothing is run).

The norm keeps multiply and add unfused.  The loss's declared formulas have fused steps, in its softmax, and its
products are matrix instructions.  Nothing may hold a packed binary32 instruction, and only the norm's gradients of
rows beyond 4096 elements may spill to scratch memory.
"""
import re

import pytest

import test_kernel_isa as base

SOURCES = ["residual.hip", "loss.hip"]


@pytest.fixture(scope="module")
def audited():
    return {s: base._kernels(base.lib_build.disassemble(s)) for s in SOURCES}


def test_no_packed_binary32_and_no_fused_norm(audited):
    for source, (kernels, _) in audited.items():
        assert len(kernels) >= 20, sorted(kernels)
        for name, ops in kernels.items():
            packed = [op for op in ops if re.match(r"v_pk_(fma|add|mul)_f32", op)]
            assert not packed, (name, packed)
            if source == "residual.hip":
                fused = sum(c for op, c in ops.items() if base.FUSED_OR_PACKED.match(op))
                assert fused <= 5 * (ops["v_div_fixup_f32"] + ops["v_rsq_f32_e32"]), (name, fused)


def test_products_are_matrix_instructions(audited):
    kernels, _ = audited["loss.hip"]
    for name, ops in kernels.items():
        mfma = sum(c for op, c in ops.items() if op.startswith("v_mfma_f32_") and op.endswith("bf16"))
        if re.match(r"k_(logits|dlogits|dx|dw|few_logits|split_logits|few_dx)$", base._short(name)):
            assert mfma >= 4, name
        assert not [op for op in ops if op.startswith("v_mfma") and not op.endswith("bf16")], name


def test_scratch(audited):
    for kernels, scratch in audited.values():
        assert set(scratch) >= set(kernels)
        for name, size in scratch.items():
            wide = re.search(r"k_residual_gradILi\dELi(8|16)ELi2E", name)
            assert size == 0 or wide, (name, size)
