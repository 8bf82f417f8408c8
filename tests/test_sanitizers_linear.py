"""The host code of the 4-bit layers and the gradient norm (qb_linear_api.cpp) under
AddressSanitizer and UndefinedBehaviorSanitizer, CPU only, with
tests/sanitize/linear_driver.cpp, whose launchers check that every array lies inside the
workspace."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="g++ or the ROCm headers not found")
def test_linear_host_code_under_address_and_undefined_behavior_sanitizers(tmp_path):
    exe = str(tmp_path / "linear_san")
    csrc = os.path.join(ROOT, "bit_optimizer_states_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{csrc}",
           os.path.join(csrc, "qb_linear_api.cpp"), os.path.join(ROOT, "tests", "sanitize", "linear_driver.cpp"),
           f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert "every call returned the expected status" in r.stdout
