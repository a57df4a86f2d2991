"""What the CUDA sources may not hold: the library is loaded by runs on several GPUs too, where a copy with a
cluster multicast destination must not appear."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_linear_q8_gb300", "csrc")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_multicast_copies(path):
    with open(path) as f:
        text = re.sub(r'"\s*"', "", f.read())  # strings that go on over several lines
    assert not re.search(r"cp\.async\.bulk[^;\"]*\.multicast", text)
