"""Inline assembly in the kernels' sources names what it changes: the compiler keeps values in a register that an
asm block writes without saying so."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "geometric_map_reduce_amd", "csrc")


def asm_blocks():
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".h", ".hip", ".cpp")):
            with open(os.path.join(CSRC, f)) as src:
                for m in re.finditer(r"\basm\s+(?:volatile\s*)?\((.*?)\);", src.read(), re.S):
                    yield f, m.group(1)


def test_there_are_some():
    assert any("global_load_lds" in text for _, text in asm_blocks())


@pytest.mark.parametrize("register", ["m0", "vcc", "exec", "scc"])
def test_fixed_registers_are_named_as_clobbers(register):
    for f, text in asm_blocks():
        code, _, rest = text.partition("::") if "::" in text else text.partition(":")
        if re.search(rf"\bs_\w+\s+{register}\b", code):
            clobbers = rest.rsplit(":", 1)[-1]
            assert f'"{register}"' in clobbers, (f, text)
