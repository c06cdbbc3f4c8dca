"""The wait states of the matrix instructions that collect attention weights,
in the assembly as built: those written out in the source, where the compiler
does not see their hazards, and its own."""
import importlib.util
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "fp8_fp4_quantized_amd")


def load(name):
    spec = importlib.util.spec_from_file_location("_" + name, os.path.join(PACKAGE, name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="no hipcc")
def test_weights_kernel(tmp_path):
    out = str(tmp_path / "weigh.s")
    build = load("build")
    assert "weigh.hip" in build.WAITS
    subprocess.run(["hipcc", *build.FLAGS, "-S", "--cuda-device-only",
                    os.path.join(PACKAGE, "csrc", "weigh.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as fh:
        text = fh.read()
    count, found = load("wait_states").offences(text.splitlines(True))
    # (six kernels of many queries, six bodies of 64 products each)
    assert count > 6 * 6 * 60 and not found, (count, found[:5])
    # the loads that bypass the registers set their place in LDS right before
    lines = [l.strip() for l in text.splitlines() if l.startswith("\t") and not l.strip().startswith((";", "."))]
    at = [i for i, l in enumerate(lines) if l.startswith("global_load_lds")]
    assert at and all(lines[i - 1] == "s_nop 0" and " m0" in lines[i - 2] for i in at)
    assert "v_pk_add_f32" not in text and "v_pk_mul_f32" not in text and "v_pk_fma_f32" not in text
