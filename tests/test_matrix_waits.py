"""The wait states that the attention's matrix instructions need, in the
assembly of the kernels as built: they are written out in the source, where
the compiler does not see their hazards.  A vector instruction's result may be
their operand two wait states later; their own result may be read twelve wait
states after an eight-pass instruction (the ones the compiler itself keeps
around its built-in forms)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "fp8_fp4_quantized_amd", "csrc", "attend.hip")
OPERAND, RESULT = 2, 12


def registers(text):
    out = set()
    for m in re.finditer(r"\b([av])\[(\d+):(\d+)\]|\b([av])(\d+)\b", text):
        if m[1]:
            out |= {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
        else:
            out.add((m[4], int(m[5])))
    return out


def run(lines):
    """(matrix instructions, offences) of instructions in the order they stand."""
    count, found, past = 0, [], []            # past: (opcode, written, wait states it takes)
    for line in lines:
        m = re.match(r"\t([a-z]\w+)\s*(.*)", line)
        op, args = m[1], m[2].split(", ")
        vector, matrix = op.startswith("v_"), "mfma" in op
        writes = registers(args[0]) if vector and not op.startswith("v_cmp") else set()
        if matrix:
            count += 1
            reads = registers(", ".join(args[1:]))
        elif vector:
            reads = registers(", ".join(args[1:])) | writes
        elif op.startswith(("ds_write", "global_store", "buffer_store", "scratch_store", "flat_store")):
            reads = registers(", ".join(args))
        else:
            reads = set()
        waited = 0
        for before, wrote, states in reversed(past):
            if waited >= RESULT:
                break
            if wrote & reads:
                was_matrix = "mfma" in before
                if matrix and not was_matrix and waited < OPERAND:
                    found.append((before, op, waited, line.strip()))
                # (a matrix instruction may follow on the same accumulators)
                if not matrix and was_matrix:
                    found.append((before, op, waited, line.strip()))
                break
            waited += states
        past.append((op, writes, int(args[0]) + 1 if op == "s_nop" else 1))
        del past[:-RESULT - 1]
    return count, found


def hazards(lines):
    """The same of assembly text: of each kernel as it stands, and along each
    branch, from the instructions before it to those at its label."""
    count, found = 0, []
    code, labels = [], {}

    def close():
        nonlocal count
        n, f = run(code)
        count += n
        found.extend(f)
        for i, line in enumerate(code):
            m = re.match(r"\ts_c?branch\w*\s+(\S+)", line)
            if m:
                j = labels[m[1]]
                found.extend(run(code[max(0, i - RESULT):i + 1] + code[j:j + RESULT])[1])
        code.clear()
        labels.clear()

    for line in lines:
        line = line.split(";")[0].rstrip()
        m = re.match(r"([.\w$]+):$", line)
        if m and m[1].startswith(".LBB"):
            labels[m[1]] = len(code)
        elif m and m[1].startswith("_Z"):
            close()
        elif re.match(r"\t[a-z]\w+", line):
            code.append(line)
    close()
    return count, found


def test_the_check_itself():
    line = "\tv_mfma_f32_32x32x16_bf16 a[0:15], v[2:5], v[6:9], a[0:15]\n"
    mov = "\tv_mov_b32_e32 v7, v1\n"
    assert hazards([mov, line])[1] and hazards([mov, "\ts_nop 0\n", line])[1]
    assert hazards([mov, "\ts_nop 1\n", line]) == (1, [])
    read = "\tv_accvgpr_read_b32 v1, a3\n"
    assert hazards([line, read])[1] and hazards([line, "\ts_nop 10\n", read])[1]
    assert hazards([line, "\ts_nop 15\n", read]) == (1, [])
    assert hazards([line, line]) == (2, [])
    # a write before a branch, its reader at the label
    there = ["\ts_cbranch_scc1 .LBB0_1\n", "\ts_nop 15\n", ".LBB0_1:\n", line]
    assert hazards([mov] + there)[1] and not hazards([mov, "\ts_nop 0\n"] + there)[1]


def test_operands_and_results_wait(tmp_path):
    if shutil.which("hipcc") is None:
        pytest.skip("no hipcc")
    out = tmp_path / "attend.s"
    subprocess.run(["hipcc", "-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950", "-Xclang", "-target-feature",
                    "-Xclang", "-packed-fp32-ops", "-S", "--cuda-device-only", SOURCE, "-o", str(out)],
                   check=True, capture_output=True, timeout=600)
    with open(out) as fh:
        count, found = hazards(fh)
    assert count > 500
    assert not found, f"{len(found)} of {count}: {found[:5]}"
