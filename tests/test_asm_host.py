"""Host test of the kernels' inline assembly.  The compiler keeps the chip's software waits between its own instructions but
does not look into an asm statement, so one that loads through scalar registers carries them itself."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_varlen_amd", "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".hip", ".hpp")))


def statements(text):
    """The assembly of every asm statement, its string literals joined."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        body = text[m.end():].split(";", 1)[0].split("::", 1)[0]
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', body)).replace("\\n", "\n").replace("\\t", "\t")


def states_before_the_load(asm):
    """Wait states in the statement ahead of its memory instruction: one each, n + 1 for s_nop n.  None without one."""
    states = 0
    for line in asm.split("\n"):
        if "offen" in line or re.match(r"\s*(buffer|global|flat|scratch)_", line):
            return states
        if line.strip():
            nop = re.match(r"\s*s_nop\s+(\d+)", line)
            states += int(nop.group(1)) + 1 if nop else 1
    return None


@pytest.mark.parametrize("name", SOURCES)
def test_loads_wait_for_scalar_registers(name):
    """A vector memory instruction may read a scalar register five wait states after a vector instruction wrote it (v_readlane,
    which is how the compiler gives back a register that it spilled, or v_readfirstlane)."""
    with open(os.path.join(CSRC, name)) as f:
        found = [(asm, states_before_the_load(asm)) for asm in statements(f.read())]
    short = [(asm, n) for asm, n in found if n is not None and n < 5]
    assert not short, short


def test_the_loads_are_found():
    """The loads to LDS of both attentions are asm statements: the test above has something to look at."""
    for name, at_least in (("gdn_attn.hpp", 2), ("gdn_attn_fp4.hpp", 1)):
        with open(os.path.join(CSRC, name)) as f:
            assert sum(states_before_the_load(asm) is not None for asm in statements(f.read())) >= at_least
