"""Host sanitizers on the validation of the layer for a few tokens and of the FFN with
8-bit pre-activations (padding_free_expert_amd/csrc/api_few.cpp and api_ckpt8.cpp with
api.cpp), built beside no-op launchers and driven with arguments from the edges of their
ranges."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import ROOT, SAN, _run, _runtime


@pytest.mark.slow
def test_few_and_ckpt8_validation_fuzz_under_sanitizers(tmp_path):
    _runtime("libasan.so")
    if not shutil.which("g++") or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("g++ or the HIP headers not found")
    exe = str(tmp_path / "few_fuzz")
    src = [os.path.join(ROOT, "padding_free_expert_amd", "csrc", f) for f in ("api.cpp", "api_few.cpp", "api_ckpt8.cpp")] + \
          [os.path.join(ROOT, "tests", "sanitize", f) for f in ("launch_stubs.cpp", "few_stubs.cpp", "few_fuzz.cpp")]
    cmd = ["g++", "-std=c++17", "-O1"] + SAN + ["-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"] + src + \
          ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe]
    b = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert b.returncode == 0, b.stderr[-3000:]
    r = _run(exe)
    assert r.returncode == 0 and "fuzz: 0 failures" in r.stdout, (r.stdout + r.stderr)[-3000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
