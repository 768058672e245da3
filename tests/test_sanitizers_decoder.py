"""A CPU build with AddressSanitizer and UndefinedBehaviorSanitizer of the host code of rotary positions,
block joins and the paged cache, driven through its entry points by a small program under
tests/sanitize/, which also records every launch and checks that it can be made.  No GPU is used:
hipLaunchKernel is the program's own."""

import os
import subprocess

from deformable_convolution_vision_amd import build as hip_build

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = os.path.join(HERE, "sanitize")
ENV = {**os.environ, "ASAN_OPTIONS": "verify_asan_link_order=0:halt_on_error=1:detect_leaks=0",
       "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}


def test_decoder_host_code_and_launches_under_sanitizers(tmp_path):
    san = ("-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-g")
    obj = str(tmp_path / "decoder_check.o")
    subprocess.run([hip_build.hipcc(), *hip_build.HIPCC_FLAGS, *san, "-c", os.path.join(SAN, "decoder_check.cpp"),
                    "-o", obj], check=True, capture_output=True)
    exe = hip_build.build(str(tmp_path / "decoder_check"), extra_flags=san, extra_objects=(obj,), link_flags=(),
                          sources=("dcn_rotary.hip", "dcn_append.hip", "dcn_residual.hip", "dcn_paged.hip"))
    r = subprocess.run([exe], env=ENV, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "DECODER SANITIZE OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
