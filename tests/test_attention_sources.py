"""What the attention kernels leave for each other, checked in the sources.  No GPU needed."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "constrained_logits_sampling_gb300",
                    "csrc")


def test_cut_units_are_written_whole():
    """An entry without a cut unit says so with all of its fields: the join counts rows by `pair` too, and what an
    earlier call of pairs left there would make it look for work that there is none of."""
    writes = 0
    for name in os.listdir(CSRC):
        if name.startswith("attn_") and name.endswith(".cuh"):
            with open(os.path.join(CSRC, name)) as f:
                code = re.sub(r"//[^\n]*", "", f.read())
            assert not re.search(r"\bcut\[[^\]]*\]\s*(\.|->)\s*\w+\s*=[^=]", code), name
            writes += len(re.findall(r"\bcut\[[^\]]*\]\s*=[^=]", code))
    assert writes >= 4
