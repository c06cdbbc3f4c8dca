"""The host code of the attention and the slot map past its checks, under
AddressSanitizer and UBSan: launchers that take their arguments and launch
nothing (tests/sanitize/attend_host.cpp).  CPU only."""
import importlib.util
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HERE = os.path.join(ROOT, "tests", "sanitize")


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(HERE, "attend_host.cpp")),
                    reason="needs g++ and tests/sanitize")
def test_launches_under_asan_and_ubsan(tmp_path):
    spec = importlib.util.spec_from_file_location("_kvc_sanitize_run", os.path.join(HERE, "run.py"))
    run = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(run)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    exe = str(tmp_path / "attend_host")
    subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include", "-Wall", *run.SAN,
                    os.path.join(ROOT, "fp8_fp4_quantized_amd", "csrc", "kvc_api.cpp"),
                    os.path.join(HERE, "attend_host.cpp"), f"-L{rocm}/lib", "-lamdhip64",
                    f"-Wl,-rpath,{rocm}/lib", "-o", exe], check=True, timeout=300)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
                                UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1"))
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert "all checks passed" in r.stdout
