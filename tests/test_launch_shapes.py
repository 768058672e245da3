"""Every launch that the attention and group norm entry points make for sizes that their checks
admit is one that a dispatch can hold.  No GPU: a small program under tests/sanitize/ links the
library's host code with a hipLaunchKernel of its own, which records and checks the shapes."""

import os
import subprocess

from deformable_convolution_vision_amd import build as hip_build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_launches_fit_a_dispatch(tmp_path):
    obj = str(tmp_path / "launch_check.o")
    subprocess.run([hip_build.hipcc(), *hip_build.HIPCC_FLAGS, "-c", os.path.join(HERE, "sanitize", "launch_check.cpp"),
                    "-o", obj], check=True, capture_output=True)
    exe = hip_build.build(str(tmp_path / "launch_check"), sources=("dcn_attention.hip", "dcn_attention_grad.hip",
                                                                   "dcn_norm.hip"),
                          extra_objects=(obj,), link_flags=())
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "LAUNCHES OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
