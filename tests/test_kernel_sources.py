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


def test_arrivals_at_another_block_release_for_the_cluster():
    """An arrival without a scope is ordered for its own block alone, and so is a wait without one."""
    remote = [s for s in statements(source("moe_tc.cuh")) if re.search(r"mbarrier\.arrive\S*shared::cluster", s)
              and "tcgen05.commit" not in s]
    assert remote
    for s in remote:
        code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', s))
        assert re.search(r"mbarrier\.arrive\.release\.cluster\.", code) or re.search(
            r"fence\.(release\.sync_restrict::shared::cta|acq_rel)\.cluster;.*mbarrier\.arrive\.relaxed\.cluster\.", code), s
    waits = [s for s in statements(source("moe_tc.cuh")) if "mbarrier.try_wait" in s]
    assert any(re.search(r"try_wait\.parity\.(acquire\.cluster|relaxed\.cluster.*fence\.acquire\S*\.cluster)", s, re.S)
               for s in waits)


def test_waits_for_another_block_acquire_for_the_cluster():
    """Of the products' barriers only `full` is signalled by the waiting block alone."""
    waits = re.findall(r"bar_wait(<PAIR>)?\(&c\.(\w+)\[", source("moe_matmul.cu"))
    assert {name for _, name in waits} == {"full", "done", "other", "sums", "read"}
    for cluster, name in waits:
        assert bool(cluster) == (name != "full"), name
