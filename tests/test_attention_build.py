"""What the attention kernels rest on at build time (no GPU needed)."""

import os
import re

from lut_binary_gemv_b200 import build as fb_build


def source(name):
    with open(os.path.join(fb_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_registers_move_in_one_place_a_warpgroup():
    # the four warps of a warpgroup have to execute the same instruction: one for each side, before the roles part
    text = source("attn_tiles.cuh")
    gives, takes = ([m.start() for m in re.finditer(rf"{side}_registers<", text)] for side in ("give", "take"))
    assert len(gives) == len(takes) == 1
    role = text.index("if (warp == 8) {\n")
    assert text.index("if (warp >= 8)") < gives[0] < role < text.index("else if (warp == 9)") < takes[0]
