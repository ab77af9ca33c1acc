"""Rules of the instruction set that a run cannot show to be kept, checked in the sources.  No
GPU needed."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "constrained_logits_sampling_gb300",
                    "csrc")


def code_of(name):
    """The source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def test_a_warpgroup_sets_its_registers_at_one_place():
    """setmaxnreg has to be the same instruction for all warps of a warpgroup: one site for the
    two softmax warpgroups, one for the warpgroup of loads and products, before its warps part."""
    code = code_of("attn_chunk.cuh")
    sites = re.findall(r"\bregs_(up|down)<\w+>\(\)", code)
    assert sorted(sites) == ["down", "up"]
    assert re.search(r"if \(warp >= 8\) regs_down<kOtherRegs>\(\);\s*if \(warp < 8\) \{\s*regs_up<kSoftmaxRegs>\(\);",
                     code)
