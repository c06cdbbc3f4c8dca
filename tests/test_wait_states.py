"""The build's check of the attention's matrix instructions (wait_states.py):
what it finds in short sequences, that the kernels as built are clean, and
that the build stops where they are not."""
import importlib.util
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "fp8_fp4_quantized_amd")


def load(name):
    spec = importlib.util.spec_from_file_location(f"_kvc_{name}", os.path.join(PACKAGE, name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.fixture(scope="module")
def waits():
    return load("wait_states")


def mfma(d, a, b, c=None):
    return f"\tv_mfma_f32_32x32x16_bf16 {d}, {a}, {b}, {c if c is not None else d}\n"


SC = mfma("v[16:31]", "v[2:5]", "v[6:9]")
O = mfma("a[0:15]", "v[2:5]", "v[6:9]")
MOV7 = "\tv_mov_b32_e32 v7, v1\n"


# sequences with an offence each
BAD = {
    "a write and the product": [MOV7, O],
    "one wait state": [MOV7, "\ts_nop 0\n", O],
    # the nearest instruction that shares a register is the product before
    "a product on the same accumulators between": [MOV7, mfma("v[16:31]", "v[40:43]", "v[44:47]"), SC],
    "a product's accumulators between": [MOV7, mfma("a[0:15]", "v[40:43]", "v[44:47]"), O],
    "first of a swap": ["\tv_permlane32_swap_b32_e32 v7, v60\n", O],
    "second of a swap": ["\tv_permlane32_swap_b32_e32 v60, v7\n", O],
    "second of a plain swap": ["\tv_swap_b32 v60, v7\n", O],
    "an accumulator written": ["\tv_accvgpr_write_b32 a3, v1\n", O],
    "exec, three wait states": ["\tv_cmpx_eq_u32_e32 v1, v2\n", "\ts_nop 2\n", O],
    "a result read": [O, "\tv_accvgpr_read_b32 v1, a3\n"],
    "a result read after eleven": [O, "\ts_nop 10\n", "\tv_accvgpr_read_b32 v1, a3\n"],
    "a result stored": [O, "\tglobal_store_dwordx4 v[50:51], a[4:7], off\n"],
    "a result stored to LDS": [SC, "\tds_write_b64 v60, v[16:17]\n"],
    "a result overwritten": [SC, "\tv_mov_b32_e32 v20, 0\n"],
    "a result overwritten by a load": [SC, "\tds_read_b128 v[20:23], v60\n"],
    "a result as the next one's factor": [SC, mfma("a[0:15]", "v[16:19]", "v[6:9]")],
    "other accumulators, overlapping": [SC, mfma("v[24:39]", "v[2:5]", "v[6:9]")],
    "the earlier of two results": [O, mfma("a[16:31]", "v[2:5]", "v[6:9]"), "\tv_accvgpr_read_b32 v1, a3\n"],
    "over a branch": [MOV7, "\ts_cbranch_scc1 .LBB0_1\n", "\ts_nop 15\n", ".LBB0_1:\n", O],
    "over a loop's edge": [".LBB0_1:\n", O, "\ts_nop 15\n", MOV7, "\ts_cbranch_scc1 .LBB0_1\n"],
}
# and without one
GOOD = {
    "two wait states": [MOV7, "\ts_nop 1\n", O],
    "two instructions": [MOV7, "\ts_mov_b32 s1, 0\n", "\ts_mov_b32 s2, 0\n", O],
    "other registers": ["\tv_mov_b32_e32 v10, v1\n", O],
    "the same accumulators": [O, O, O],
    "a result after twelve": [O, "\ts_nop 11\n", "\tv_accvgpr_read_b32 v1, a3\n"],
    "exec, four wait states": ["\tv_cmpx_eq_u32_e32 v1, v2\n", "\ts_nop 3\n", O],
    "a scalar result": ["\tv_readlane_b32 s7, v1, 3\n", O],
    "a mask": ["\tv_cmp_eq_u32_e32 vcc, v1, v2\n", O],
    "products of others": [O, SC, mfma("a[16:31]", "v[2:5]", "v[6:9]")],
}


@pytest.mark.parametrize("name", BAD)
def test_offences(waits, name):
    count, found = waits.offences(BAD[name])
    assert count == sum("mfma" in l for l in BAD[name]) and found


@pytest.mark.parametrize("name", GOOD)
def test_clean(waits, name):
    assert waits.offences(GOOD[name])[1] == []


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="no hipcc")
def test_the_kernels(waits, tmp_path):
    out = tmp_path / "attend.s"
    subprocess.run(["hipcc", *load("build").FLAGS, "-S", "--cuda-device-only",
                    os.path.join(PACKAGE, "csrc", "attend.hip"), "-o", str(out)],
                   check=True, capture_output=True, timeout=600)
    with open(out) as fh:
        count, found = waits.offences(fh)
    assert count > 500
    assert not found, f"{len(found)} of {count}: {found[:5]}"


KERNEL = """
#include <hip/hip_runtime.h>
extern "C" __global__ void k() {
  asm volatile("v_mov_b32 v12, 0\\n\\t%sv_mfma_f32_32x32x16_bf16 v[32:47], v[12:15], v[12:15], 0\\n\\ts_nop 15"
               ::: "v12", "v47");
}
"""


@pytest.mark.skipif(shutil.which("hipcc") is None, reason="no hipcc")
def test_the_build_stops(tmp_path, monkeypatch):
    """A kernel whose product reads what the instruction before it wrote is not
    built (compiled here, never run); with two wait states it is."""
    build = load("build")
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    for nop, ok in (("", False), ("s_nop 1\\n\\t", True)):
        (tmp_path / "k.hip").write_text(KERNEL % nop)
        call = lambda: build._compile("k.hip", str(tmp_path / "k.o"), False, waits=True)
        if ok:
            call()
        else:
            with pytest.raises(RuntimeError, match="wait state"):
                call()
        assert (tmp_path / "k.o").exists() == ok
