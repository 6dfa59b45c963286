"""Memory instructions in inline assembly that read scalar registers: the compiler, which
keeps five wait states between a vector instruction that writes a scalar register and a
memory instruction that reads it, does not look into such a block, so the block itself
has to hold them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "spherical_disco_convolution_amd", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".h", ".hip")))


@pytest.mark.parametrize("name", FILES)
def test_scalar_operands_of_memory_instructions_are_waited_for(name):
    with open(os.path.join(CSRC, name)) as f:
        blocks = re.findall(r"asm(?: volatile)?\((.*?)\);", f.read(), re.S)
    for block in blocks:
        text = "".join(re.findall(r'"([^"]*)"', block.split("\n                 :")[0])).split("\\n\\t")
        scalars = set(re.findall(r"%(\d+)", " ".join(re.findall(r'"[^"]*"', block)))) & {
            str(i) for i, c in enumerate(re.findall(r'"([=+&]?[vsin])"\(', block)) if "s" in c}
        states = 0
        for line in text:
            op = line.split()
            if op and re.match(r"(buffer|global|flat|scratch)_", op[0]):
                if scalars & set(re.findall(r"%(\d+)", line)):
                    assert states >= 5, (name, line)
            states += int(op[1]) + 1 if op and op[0] == "s_nop" else 0
