"""The wait states that matrix instructions need on gfx950, in assembly text.

The attention's matrix instructions are written out in its source, where the
compiler does not see their hazards; some of them carry no wait states because
their operands come from LDS and from registers that stay.  That rests on the
registers the compiler allocates, so the build reads the assembly it makes and
stops where a wait is missing.

What is needed, in wait states (an instruction counts one, ``s_nop n`` n + 1):
  - 2 between a vector instruction that writes a register and a product that
    reads it; 4 after one that writes the execution mask;
  - 12 between a product of eight passes (the longest used here) and anything
    that touches its result -- reads, stores, overwrites it, takes it as a
    factor -- but a product that goes on accumulating on the same registers.
"""
from __future__ import annotations

import re

OPERAND, EXEC, RESULT = 2, 4, 12

_REGS = re.compile(r"\b([av])\[(\d+):(\d+)\]|\b([av])(\d+)\b")
_LINE = re.compile(r"\t([a-z]\w+)\s*(.*)")
_LABEL = re.compile(r"([.\w$]+):$")
_BRANCH = re.compile(r"\ts_c?branch\w*\s+(\S+)")
# stores have their data and address among all operands, loads their target first
_STORE = ("ds_write", "ds_add", "ds_or", "ds_max", "global_store", "global_atomic", "buffer_store",
          "scratch_store", "flat_store")
_LOAD = ("ds_read", "ds_bpermute", "ds_permute", "global_load", "buffer_load", "scratch_load", "flat_load")


def registers(text: str) -> set:
    out = set()
    for m in _REGS.finditer(text):
        if m[1]:
            out |= {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
        else:
            out.add((m[4], int(m[5])))
    return out


class _Instruction:
    def __init__(self, line: str):
        m = _LINE.match(line)
        self.text, self.op = line.strip(), m[1]
        args = m[2].split(", ")
        self.matrix = "mfma" in self.op
        self.vector = self.op.startswith("v_") and not self.matrix
        self.states = int(args[0]) + 1 if self.op == "s_nop" else 1
        self.writes, self.reads, self.adds = set(), set(), set()
        self.exec = self.op.startswith("v_cmpx")
        if self.matrix:
            self.writes, self.adds = registers(args[0]), registers(args[3])
            self.reads = registers(", ".join(args[1:3]))
        elif self.vector:
            if not self.op.startswith("v_cmp"):
                swap = "swap" in self.op          # both operands are written
                self.writes = registers(", ".join(args[:2]) if swap else args[0])
            self.reads = registers(", ".join(args[1:]))
        elif self.op.startswith(_STORE):
            self.reads = registers(", ".join(args))
        elif self.op.startswith(_LOAD):
            self.writes, self.reads = registers(args[0]), registers(", ".join(args[1:]))


def _offence(before: _Instruction, waited: int, now: _Instruction) -> bool:
    if now.matrix and before.vector:
        return (waited < OPERAND and bool(before.writes & (now.reads | now.adds)) or
                waited < EXEC and before.exec)
    if before.matrix and waited < RESULT:
        if now.matrix:
            # on the same registers, from which it also accumulates or starts anew
            same = now.writes == before.writes and (not now.adds or now.adds == before.writes)
            touched = now.reads if same else now.reads | now.adds | now.writes
        else:
            touched = now.reads | now.writes
        return bool(before.writes & touched)
    return False


def _run(code: list) -> list:
    """Offences among instructions in the order they stand."""
    found = []
    for i, now in enumerate(code):
        waited = 0
        for before in reversed(code[max(0, i - RESULT):i]):
            if waited >= RESULT:
                break
            if _offence(before, waited, now):
                found.append((before.text, waited, now.text))
            waited += before.states
    return found


def offences(lines) -> tuple:
    """(matrix instructions, offences as (text before, wait states, text)) of
    assembly text: of each kernel as it stands, and along each branch, from the
    instructions before it to those at its label."""
    count, found = 0, []
    code, labels = [], {}

    def close():
        nonlocal count
        count += sum(i.matrix for i in code)
        found.extend(_run(code))
        for i, branch in enumerate(code):
            m = _BRANCH.match("\t" + branch.text)
            if m:
                to = labels[m[1]]
                joined = code[max(0, i - RESULT):i + 1]
                joined += code[to:to + RESULT]
                # (what lies on one side of the branch alone was seen above)
                for o in _run(joined):
                    if o not in found:
                        found.append(o)
        code.clear()
        labels.clear()

    for line in lines:
        line = line.split(";")[0].rstrip()
        m = _LABEL.match(line)
        if m and m[1].startswith(".LBB"):
            labels[m[1]] = len(code)
        elif m and not m[1].startswith("."):
            close()
        elif _LINE.match(line):
            code.append(_Instruction(line))
    close()
    return count, found
