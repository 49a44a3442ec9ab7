"""The host side of the operators around the projections
(gated_deltanet_02_amd/csrc/gdn_layer_api.cpp) under AddressSanitizer and
UndefinedBehaviorSanitizer: built with g++ for the CPU, the launchers replaced
by stand-ins that check what reaches them, and driven by
tests/native/layer_sanitize.cpp with seeded calls.  A sanitizer report makes the
program exit non-zero."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_deltanet_02_amd", "csrc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


def test_layer_api_under_sanitizers(tmp_path):
    if not shutil.which("g++") or not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        pytest.skip("g++ or the HIP headers not found")
    exe = str(tmp_path / "layer_san")
    subprocess.run(["g++", "-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                    "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
                    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(CSRC, "gdn_layer_api.cpp"),
                    os.path.join(ROOT, "tests", "native", "layer_sanitize.cpp"), "-o", exe], check=True, timeout=300)
    env = dict(os.environ, UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], env=env, capture_output=True, text=True, timeout=300)
    print(r.stdout)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert " 0 failure(s)" in r.stdout
