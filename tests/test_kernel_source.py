"""Rules on the kernels' sources that no run can show to be broken."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fine_grained_block_token_b200", "csrc")


@pytest.mark.parametrize("name", ["route.cu", "lora.cu", "lora_tiles.cu"])
def test_cluster_barriers_are_met_converged(name):
    """The cluster barrier is the .aligned form, which the lanes of a warp have
    to execute together.  Loops whose trips differ between lanes and branches of
    one lane come before it, so a __syncwarp() stands directly in front."""
    lines = [re.sub(r"//.*", "", line).strip() for line in open(os.path.join(CSRC, name))]
    lines = [line for line in lines if line]
    at = [i for i, line in enumerate(lines) if "cluster_sync()" in line]
    assert at
    for i in at:
        assert lines[i - 1] == "__syncwarp();", f"{name}: {lines[i - 1]} / {lines[i]}"
