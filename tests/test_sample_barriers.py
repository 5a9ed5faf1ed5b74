"""CPU test of csrc/sample.cu's block sums: the warps' sums lie in shared memory that the next
sum or scan writes again, so a function that reads them ends behind a barrier."""
import re
from pathlib import Path

import pytest

import speculative_decoding_rejection_gb300 as sv

SOURCE = (Path(sv.__file__).parent / "csrc" / "sample.cu").read_text()


def body(name):
    """The text of a function between its outer braces."""
    at = SOURCE.index("{", re.search(r"void " + name + r"\(", SOURCE).end())
    depth = 0
    for i in range(at, len(SOURCE)):
        depth += (SOURCE[i] == "{") - (SOURCE[i] == "}")
        if depth == 0:
            return SOURCE[at + 1:i]


@pytest.mark.parametrize("name", ["block_scan", "block_sums"])
def test_the_warps_sums_are_read_before_a_barrier(name):
    text = body(name)
    last = max(m.start() for m in re.finditer(r"s\.warp_\w+\[lane\]", text))
    assert "__syncthreads();" in text[last:]
    # and written behind one, or where the caller's last barrier allows it
    first_read = min(m.start() for m in re.finditer(r"s\.warp_\w+\[lane\]", text))
    assert "__syncthreads();" in text[text.index("s.warp_"):first_read]
