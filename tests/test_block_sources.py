"""What the sources have to say to the compiler, where no run shows that it is missing."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_15_gb300", "csrc")


def test_copies_to_a_place_just_read_are_memory_to_the_compiler():
    """The norm of heads reads a unit's place in shared memory and asks for the next unit to the same place, with no barrier
    between: without the clobber the compiler may move the read behind the copy."""
    with open(os.path.join(CSRC, "norm_rope.cu")) as f:
        copies = re.findall(r"asm volatile\(\s*\"cp\.async\.c[ag]\.shared\.global.*?\);", f.read(), re.S)
    assert len(copies) >= 2 and all('"memory"' in c for c in copies), copies
