"""What the compiler has to be told about inline assembly and the order of memory, read from the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_precision_allreduce_amd", "csrc")


def statements(text):
    """The inline-assembly statements of a source: (instructions, all of the statement)."""
    for m in re.finditer(r"\basm volatile\s*\((.*?)\);", text, re.S):
        yield "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(1).split(":")[0])), m.group(1)


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.h*"))), ids=os.path.basename)
def test_overwritten_m0_is_named(path):
    """A register that an instruction here writes and that is not an operand may not carry the compiler's own values."""
    for instructions, whole in statements(open(path).read()):
        if re.search(r"\bm0\s*,", instructions):
            assert re.search(r':\s*"m0"', whole), whole


def test_statements_are_found():
    text = 'asm volatile("s_mov_b32 m0, %0\\n\\tx" ::"s"(a) : "m0"); asm volatile("" ::: "memory");'
    assert [i for i, _ in statements(text)] == ["s_mov_b32 m0, %0\\n\\tx", ""]
    assert sum("m0" in i for i, _ in statements(open(os.path.join(CSRC, "lpc_gemm.hip")).read())) == 2


@pytest.mark.parametrize("name", ["lpc_gemm.hip", "lpc_cols.hip", "lpc_router.hip", "lpc_adamw.hip", "lpc_ops.hpp"])
def test_wave_barriers_order_memory(name):
    """A wave barrier keeps no load or store where it is; where lanes exchange values through LDS a fence has to."""
    fence = r'__builtin_amdgcn_fence\(__ATOMIC_ACQ_REL, "wavefront"\);\s*'
    text = open(os.path.join(CSRC, name)).read()
    assert len(re.findall(r"__builtin_amdgcn_wave_barrier\(\);", text)) == \
        len(re.findall(fence + r"__builtin_amdgcn_wave_barrier\(\);\s*" + fence, text))
