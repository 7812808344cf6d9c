"""Properties of the 8-bit layer's kernels that show in their source only (no GPU): what a
give-up may not do."""

import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "post_weight_quantization_24_b200", "csrc", "fp8_linear.cu")


def _code():
    return re.sub(r"//[^\n]*", "", open(SRC).read())


def test_no_lane_skips_a_warp_wide_wait_by_itself():
    """The promotion warps' waits end in a vote of all lanes, so no condition that lanes read one
    by one (the abort flag) may stand around them."""
    code = _code()
    assert len(re.findall(r"f8_warp_wait(?:<true>)?\(", code)) >= 5
    assert not re.findall(r"if\s*\([^;{}]*abort_flag[^;{}]*\)\s*\{?\s*f8_warp_wait(?:<true>)?\(", code)
