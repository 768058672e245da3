"""A CPU build with AddressSanitizer and UndefinedBehaviorSanitizer of the host code of cross
attention and group norm, driven through its entry points (edge cases included) by a small
program under tests/sanitize/.  No GPU is used: every call returns before a kernel launch."""

import os
import subprocess

from deformable_convolution_vision_amd import build as hip_build

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = os.path.join(HERE, "sanitize")
ENV = {**os.environ, "ASAN_OPTIONS": "verify_asan_link_order=0:halt_on_error=1:detect_leaks=0",
       "UBSAN_OPTIONS": "halt_on_error=1:print_stacktrace=1"}


def test_attention_and_norm_host_code_under_sanitizers(tmp_path):
    san = ("-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer", "-g")
    drv_obj = str(tmp_path / "ops_check.o")
    subprocess.run([hip_build.hipcc(), *hip_build.HIPCC_FLAGS, *san, "-c", os.path.join(SAN, "ops_check.cpp"),
                    "-o", drv_obj], check=True, capture_output=True)
    exe = hip_build.build(str(tmp_path / "ops_check"), extra_flags=san, extra_objects=(drv_obj,), link_flags=())
    r = subprocess.run([exe], env=ENV, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "OPS SANITIZE OK" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
