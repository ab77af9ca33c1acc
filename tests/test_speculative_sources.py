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


def test_verification_writes_no_flag_that_warps_still_read():
    """Every thread reads the request's flag after a barrier, and the next barrier of the block
    comes only after the sums: a warp that is ahead must not write the word that a warp behind it
    has yet to read, or the two would part before a barrier of all."""
    code = code_of("verify.cu")
    read = code.index("bad = sh.bad;")
    assert "sh.bad" in code[:read] and "sh.bad" not in code[read + len("bad = sh.bad;"):]
