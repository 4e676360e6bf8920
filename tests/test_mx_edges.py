"""The microscaled 4-bit operators without a GPU: what their sources and host
checks hold at the ends of what the calls allow."""
import glob
import os
import re

from weight_only_int4_02_amd import build


def test_inline_assembly_that_writes_m0_says_so():
    """The compiler may keep a value of its own in M0: a block of assembly that
    writes the register has to name it among what it overwrites."""
    blocks = []
    for path in glob.glob(os.path.join(build.CSRC, "*")):
        blocks += re.findall(r"asm volatile\(.*?\);", open(path).read(), re.S)
    writes = [b for b in blocks if re.search(r"s_\w+ m0,", b)]
    assert writes
    for block in writes:
        assert re.search(r':\s*"m0"', block), block
