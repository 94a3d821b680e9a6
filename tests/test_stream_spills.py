"""Which kernels of the residual norm may use scratch memory (CPU only: hipcc emits the assembly of our sources).

Only gradients that hold two chunks a lane in rows of the widest forms: with a norm or gate after the block from 4096
elements on, without from 8192 on.  No kernel of the forward pass does.
"""
import re

import test_kernel_isa as base


def test_scratch_of_each_form():
    kernels, scratch = base._kernels(base.lib_build.disassemble("residual.hip"))
    forms = {}
    for name, size in scratch.items():
        grad = re.search(r"k_residual_gradILi(\d)ELi(\d+)ELi(\d)ELi(\d)E", name)
        if grad is None:
            assert size == 0, (name, size)
            continue
        _, waves, chunks, form = (int(g) for g in grad.groups())
        forms[waves, chunks, form] = max(size, forms.get((waves, chunks, form), 0))
    assert len(forms) == 18, sorted(forms)
    block = 2
    may = {(8, 2, block), (16, 2, 0), (16, 2, 1), (16, 2, block)}
    assert {f for f, size in forms.items() if size} <= may, forms
