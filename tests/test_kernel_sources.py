"""What the tensor-core kernels' inline PTX has to say for the compiler and the memory model to keep the order that the
kernels rely on.  A schedule that happens to be right shows in no result, so these read the sources."""
import os
import re

import pytest

import quantized_routed_expert_router_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def statements(text):
    """the inline PTX statements of a source, each up to the parenthesis that closes it"""
    out = []
    for m in re.finditer(r"\basm\b(?:\s+volatile)?\s*\(", text):
        depth, quoted, i = 1, False, m.end()
        while depth:
            c = text[i]
            if c == '"':
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        out.append(text[m.start():i])
    return out


TC = ["moe_tc.cuh", "moe_fp8.cu", "moe_matmul.cu"]


@pytest.mark.parametrize("name", TC)
def test_values_from_tmem_come_out_of_the_wait(name):
    """A statement that waits for TMEM loads names the 32 registers that hold their values."""
    for s in statements(source(name)):
        if "tcgen05.wait::ld" in s:
            assert len(re.findall(r'"[=+]r"\(v\[\d+\]\)', s)) == 32, s
        elif "tcgen05.ld." in s:
            assert len(re.findall(r'"=r"\(v\[\d+\]\)', s)) == 32, s


@pytest.mark.parametrize("name", TC[1:])
def test_loads_that_go_on_are_waited_for_by_their_registers(name):
    text = source(name)
    begun = re.findall(r"tmem_ld32_begin\([^;]*,\s*([\w\[\]]+)\);", text)
    landed = re.findall(r"tmem_landed\(([\w\[\]]+)\);", text)
    assert sorted(begun) == sorted(landed)
    assert not re.search(r"tcgen05\.(ld|wait)", text)     # only through the helpers
