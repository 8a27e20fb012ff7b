"""What the sources of the kernels around the attention over the 4-bit cache have
to say because no run can show it (no GPU needed)."""

import re

from mla_decode_query_gb300 import build


def test_aligned_cluster_barriers_follow_a_warp_barrier():
    """PTX wants all threads of a warp at the same .aligned instruction together; a loop or a
    branch by thread may come before it."""
    text = (build.CSRC / "mlaqp_kv4_select.cu").read_text()
    found = list(re.finditer(r"barrier\.cluster\.\w+\.\w+\.aligned", text))
    assert found
    for m in found:
        body = text[text.rindex("__device__", 0, m.start()):m.start()]
        assert "__syncwarp();" in body, body
