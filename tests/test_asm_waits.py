"""Assembly blocks wait for themselves: the compiler does not look into them for what an instruction
needs before it may read a register (CPU; reads the sources)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_quantized_gemm_amd", "csrc")


def blocks():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        if os.path.isdir(path):
            continue
        with open(path) as f:
            for m in re.finditer(r'asm(?: volatile)?\(((?:\s*"(?:[^"\\]|\\.)*")+)\s*:(.*?)\);', f.read(), re.S):
                text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m[1]))
                yield os.path.basename(path), [i.strip() for i in text.replace("\\t", "").split("\\n")], m[2]


def states_before(code, what):
    """Wait states of a block before its first instruction that begins with `what`."""
    states = 0
    for i in code:
        if re.match(what, i):
            return states
        nop = re.match(r"s_nop (\d+)", i)
        states += int(nop[1]) + 1 if nop else 1
    return None


LOADS = [(f, c, r) for f, c, r in blocks() if any(re.match("(buffer|global)_", i) for i in c)]


def test_there_are_some():
    assert len(LOADS) == 2


@pytest.mark.parametrize("name,code,registers", LOADS)
def test_vector_memory_waits_for_its_scalars(name, code, registers):
    """Five wait states between a vector instruction that writes a scalar register (which may come
    right before the block) and a vector memory instruction that reads it; one between a write of m0
    and a load to LDS."""
    load = next(i for i in code if re.match("(buffer|global)_", i))
    if load.startswith("buffer"):
        assert states_before(code, "buffer_") >= 5, code
    at = next(k for k, i in enumerate(code) if i.startswith("s_mov_b32 m0"))
    assert states_before(code[at + 1:], "(buffer|global)_") >= 1, code
