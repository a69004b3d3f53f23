"""CPU-only check of the sources: a launch that may begin while the one in front still
writes reads what that one writes by ordinary loads, behind its wait.  A read-only load
(__ldg) promises that nothing writes there while the kernel runs, and may be moved in
front of the wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_device_gb300", "csrc")
# written by one launch of a call and read by the next: tile table, column sums, sorted tokens, runs, partial rows
HANDED_ON = ["g.tiles", "a.part", "a.terms", "keys", "pos", "cross", "part", "fill.used", "f.used"]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_what_an_earlier_launch_writes_is_not_read_as_constant(path):
    text = open(path).read()
    if "pdl_wait" not in text:
        return
    names = "|".join(re.escape(n) for n in HANDED_ON)
    assert not re.findall(r"__ld(?:g|cs)\(\s*(?:&\s*)?(?:%s)\b" % names, text)
    assert "__restrict__" not in text
