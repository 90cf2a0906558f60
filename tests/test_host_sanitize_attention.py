"""The attention-side host layer (attention_api.cpp, the rules in kv_attention.hip) built for the CPU with g++ under
AddressSanitizer and UndefinedBehaviorSanitizer and driven by tests/host_sanitize/attention_driver.cpp."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIP_INCLUDE = "/opt/rocm/include"


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(HIP_INCLUDE), reason="needs g++ and the HIP headers")
def test_attention_host_layer_under_sanitizers(tmp_path):
    exe = str(tmp_path / "orbq_attention_driver")
    csrc = os.path.join(ROOT, "calibration_free_w4a4_amd", "csrc")
    here = os.path.join(ROOT, "tests", "host_sanitize")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined",
           "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", f"-I{HIP_INCLUDE}", f"-I{os.path.join(ROOT, 'include')}", "-x", "c++"]
    cmd += [os.path.join(csrc, f) for f in ("api.cpp", "attention_api.cpp", "codebook.cpp", "kv_attention.hip")]
    cmd += [os.path.join(here, f) for f in ("stubs.cpp", "attention_driver.cpp")] + ["-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert r.stdout.strip().startswith("ok "), r.stdout[-2000:]
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr[-3000:]
