"""What the attention kernels rest on at build time (no GPU needed)."""

import os
import re
import subprocess

import pytest

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


@pytest.mark.parametrize("name,kernels", [("attn_prompt.cu", 8), ("attn_tree_tiles.cu", 4)])
def test_compiler_gives_the_tiles_the_registers_that_their_warps_share_out(name, kernels, tmp_path):
    # with any other number the calls refuse to launch: the warps' shares would not add up
    planned = re.search(r"kLaunchRegisters = (\d+)", source("attn_tiles.cuh")).group(1)
    flags = [f for f in fb_build.NVCC_FLAGS if f not in ("-shared", "--threads", "0")]
    r = subprocess.run([os.environ.get("NVCC", "nvcc"), *flags, "-Xptxas", "-v", "-I", fb_build.INCLUDE, "-I", fb_build.CSRC,
                        "-c", "-o", str(tmp_path / "o"), os.path.join(fb_build.CSRC, name)],
                       capture_output=True, text=True, check=True)
    got = re.findall(r"entry function '\w*tile_kernel\w*'.*?Used (\d+) registers", r.stderr, re.S)
    assert got == [planned] * kernels
    assert not re.search(r"setmaxnreg|[1-9]\d* bytes spill", r.stderr)
