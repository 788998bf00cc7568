"""The sources of the paged attention's split kernels: what a warp's lanes tell one another through shared memory is not
written over while a lane may still read it."""
import os
import re

import pytest

from lattice_vq_weight_gb300 import build


@pytest.mark.parametrize("name", ["lq_attn_paged.cu", "lq_attn_q4.cu"])
def test_a_segments_request_is_read_before_the_next_ones_is_written(name):
    """The loop's last reads of `asked` and its write in a later turn have a barrier of the warp between them: nothing
    else in the loop brings the lanes together there."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
    writes = [m.start() for m in re.finditer(r"if \(lane == 0\) asked\[warp\] = ", text)]
    reads = [m.start() for m in re.finditer(r"= asked\[warp\]", text)]
    assert len(writes) == 1 and reads and min(reads) > writes[0]
    assert re.search(r"__syncwarp\(\);\s*$", text[:writes[0]])
