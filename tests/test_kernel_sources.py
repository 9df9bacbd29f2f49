"""What the kernel sources must not contain, whatever they compute."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp4_expert_gb300", "csrc")


def test_joint_steps_of_a_warp_name_their_lanes():
    """__activemask() is whoever happens to run together: as the mask of a step that all lanes must have reached
    (a copy out of a slot before it is given back, a vote) it lets lanes go ahead of the others."""
    files = glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h"))
    assert len(files) > 10
    for f in files:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        assert "__activemask" not in code, os.path.basename(f)
