"""What the attention kernels' source has to keep that no run can show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "skinny_gemm_q4_gb300", "csrc")


def test_the_few_row_kernel_gives_up_as_a_warp():
    """A wait that ran out in some lanes only must not let the others go on to
    the warp's shuffles and products: what leaves the loop over the records is a
    vote, and lane 0, which reports it, takes part."""
    with open(os.path.join(CSRC, "qg_attn_decode.cuh")) as f:
        src = re.sub(r"//.*", "", f.read())
    leave = re.findall(r"if \(([^{}]*)\) \{\s*dead = true;\s*break;", src)
    assert len(leave) == 1 and "_sync(~0u" in leave[0]


def test_the_rotations_angles_are_aligned_as_they_are_read():
    """They are read 16 bytes at a time: a float2 array by itself is aligned to
    8 only."""
    with open(os.path.join(CSRC, "qg_rope.cu")) as f:
        src = re.sub(r"//.*", "", f.read())
    arrays = {n: how for how, n in re.findall(r"__shared__ ([^;]*?)(\w+)\[", src)}
    read = re.findall(r"reinterpret_cast<const float4 \*>\((\w+)\)", src)
    assert arrays
    assert all("__align__(16)" in arrays[n] or "float4" in arrays[n] for n in read if n in arrays)
