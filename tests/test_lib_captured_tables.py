"""The calls that upload a table of tensors, or a user code, under capture (CPU only): qb_api.cpp with
tests/sanitize/capture_driver.cpp in place of the HIP runtime and the kernels, under AddressSanitizer and
UndefinedBehaviorSanitizer.  A captured call must not record a copy from host memory, which the graph would
read again at every replay."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "include", "hip")),
                    reason="g++ or the ROCm headers not found")
def test_captured_calls_carry_their_tables(tmp_path):
    exe = str(tmp_path / "capture")
    csrc = os.path.join(ROOT, "bit_optimizer_states_amd", "csrc")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{ROOT}/include", f"-I{csrc}",
           os.path.join(csrc, "qb_tables.cpp"), os.path.join(csrc, "qb_api.cpp"),
           os.path.join(ROOT, "tests", "sanitize", "capture_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=1"))
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert "captured calls carry their tables" in r.stdout
