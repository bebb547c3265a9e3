"""What the kernels' sources may not do, where no run would show it."""
import os
import re

import pytest

from weight_quantized_decode_block_amd import build as hip_build

SOURCES = sorted(f for f in os.listdir(hip_build.CSRC) if f.endswith((".hip", ".h", ".cpp")))


def asm_blocks(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(hip_build.CSRC, name)).read())
    for m in re.finditer(r"\basm\s*(?:volatile)?\s*\(", text):
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[end], 0)
            end += 1
        yield text[m.end():end - 1]


@pytest.mark.parametrize("name", SOURCES)
def test_inline_assembly_writes_no_unnamed_m0(name):
    """m0 is no register that a clobber list may name, so assembly that writes it
    does so behind the compiler; as an operand ("{m0}") the compiler sets it."""
    for block in asm_blocks(name):
        template = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', block.split("\n               :")[0]))
        assert not re.search(r"\bs_\w+\s+m0\b", template), template


def test_the_blocks_are_found():
    assert any("buffer_load_dwordx4" in b for b in asm_blocks("mx_tile.hip"))
