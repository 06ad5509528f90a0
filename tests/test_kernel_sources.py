"""What the kernel sources promise of themselves, checked on their text."""
import os
import re

import nvfp4_bit_microscaled_b200 as pkg

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkg.__file__)), "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_abort_flags_are_read():
    # a flag that a wait which gave up sets is of use only where other loops look at it
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            s = _source(name)
            if "abort_flag = 1" in s:
                assert re.search(r"!\s*\*?\s*abort_flag", s), name
