"""README's Python examples: one block for each part, each marked for the test that runs it.

The example around an attention layer is the one block marked `python`, the one between two blocks and at the end the
one marked `py` (both names are Python's, for whoever shows the page).
"""
import os
import re

import pytest

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def block(mark):
    with open(README) as fh:
        code, = re.findall(rf"```{mark}\n(.*?)```", fh.read(), re.S)
    return code


@pytest.mark.parametrize("mark, call", [("python", "repro_clip_grad_list"), ("py", "repro_vocab_loss_backward")])
def test_one_block_for_each_part(mark, call):
    code = block(mark)
    compile(code, README, "exec")
    assert call in code
