"""No kernel reads a matrix instruction's result behind a branch before it is ready.

The result is ready some issue slots after the instruction (at most 20, for those of 16 passes).  The compiler fills in the waits, but counts too few where a branch is
taken in between (it takes the branch and waits for memory, which may be over at once, for
slots), so the kernels put waits of their own before such branches.  This test follows every
path through the built code from each matrix instruction.
"""
import re
import shutil
import subprocess

import pytest

import all_reduce_amd as ar

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
SLOTS = 20


def registers(operand):
    found = set()
    for kind, low, high in re.findall(r"\b([av])\[(\d+):(\d+)\]", operand):
        found.update((kind, i) for i in range(int(low), int(high) + 1))
    found.update((kind, int(i)) for kind, i in re.findall(r"\b([av])(\d+)\b", operand))
    return found


class Instruction:
    __slots__ = ("name", "operands", "target", "text", "_reads")

    def __init__(self, text, target):
        self.text, self.target = text, target
        self.name, _, rest = text.partition(" ")
        self.operands = [o.strip() for o in rest.split(",")] if rest else []
        self._reads = None

    @property
    def matrix(self):
        return self.name.startswith("v_mfma")

    @property
    def reads(self):
        """Registers that it reads; of a matrix instruction without its addend, for which the
        hardware waits."""
        if self._reads is None:
            if self.matrix:
                read = self.operands[1:3]
            elif re.match(r"(ds_write|ds_add|global_store|global_atomic|flat_store|scratch_store|buffer_store)", self.name):
                read = self.operands
            else:
                read = self.operands[1:]
            self._reads = set().union(*map(registers, read)) if read else set()
        return self._reads


def kernels(listing):
    """(name, instructions) of each function of a disassembly with matrix instructions."""
    for part in re.split(r"^[0-9a-f]+ <", listing, flags=re.M)[1:]:
        if "v_mfma" not in part:
            continue
        name, _, body = part.partition(">:")
        start, code, targets = None, [], {}
        for line in body.splitlines():
            m = re.match(r"\t(\S.*?)\s*// ([0-9A-F]+):(.*)$", line)
            if m is None:
                continue
            text, at = m.group(1), int(m.group(2), 16)
            start = at if start is None else start
            to = re.search(r"<[^>]*\+0x([0-9a-f]+)>", m.group(3))
            to = int(to.group(1), 16) if to else 0 if re.search(r"<[^+>]+>", m.group(3)) else None
            targets[at - start] = len(code)
            code.append(Instruction(text, to if "branch" in text.split(" ")[0] else None))
        for i in code:
            i.target = None if i.target is None else targets.get(i.target)
        yield name, code


def early_reads(code):
    """Instructions that may read a matrix instruction's result behind a branch, less than SLOTS
    issue slots after it: (its place, the reader's place, the slots)."""
    bad = set()

    def walk(at, result, slots, branched, from_):
        while at < len(code) and slots < SLOTS:
            i = code[at]
            at += 1
            if i.name == "s_nop":
                slots += int(i.operands[0], 0) + 1
            elif i.name.startswith("s_waitcnt"):
                pass
            elif i.name == "s_endpgm":
                return
            elif i.target is not None:
                walk(i.target, result, slots + 1, True, from_)
                if i.name == "s_branch":
                    return
                slots += 1
            else:
                if i.reads & result:
                    if branched:
                        bad.add((from_, at - 1, slots))
                    return  # (on this path the compiler has waited before it)
                slots += 4 if i.matrix else 1  # (the matrix unit takes no less than four for one)

    for n, i in enumerate(code):
        if i.matrix:
            walk(n + 1, registers(i.operands[0]), 0, False, n)
    return sorted(bad)


def test_the_walk_finds_reads_behind_branches():
    def listing(*lines):
        body = "".join(f"\t{t:<50} // {256 + 4 * n:012X}: 00000000{to}\n" for n, (t, to) in enumerate(lines))
        return f"0000000000000100 <k>:\n{body}"

    mfma = ("v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0", "")
    there, read, end = ("s_cbranch_scc1 1", " <k+0xc>"), ("v_add_f32_e32 v20, v3, v21", ""), ("s_endpgm", "")
    wait = [("s_nop 7", "")] * 3
    other = ("v_mov_b32_e32 v30, v31", "")

    def found(*lines):
        (_, code), = kernels(listing(*lines))
        return early_reads(code)

    assert found(mfma, there, other, read, end) == [(0, 3, 1)]
    assert found(mfma, *wait, ("s_cbranch_scc1 1", " <k+0x18>"), other, read, end) == []
    assert found(mfma, other, read, end) == []
    # the back edge of a loop, to its first instruction
    assert found(read, mfma, ("s_cbranch_scc1 65534", " <k>"), end) == [(1, 0, 1)]
    assert found(read, mfma, *wait, ("s_cbranch_scc1 65534", " <k>"), end) == []
    # operands of another matrix instruction, and a store's data
    assert found(mfma, there, other, ("v_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[12:15], v[4:7]", ""), end)
    assert not found(mfma, there, other, ("v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]", ""), end)
    assert found(mfma, there, other, ("ds_write_b32 v40, v2 offset:16", ""), end)


def test_no_kernel_reads_a_matrix_result_early(tmp_path):
    if not shutil.which(OBJDUMP):
        pytest.skip("no llvm-objdump")
    copy = tmp_path / "lib.so"
    shutil.copy(ar.LIBRARY, copy)
    subprocess.run([OBJDUMP, "--offloading", str(copy)], check=True, capture_output=True, cwd=tmp_path)
    seen = 0
    for part in sorted(tmp_path.glob("lib.so.*gfx950")):
        listing = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(part)], check=True, capture_output=True,
                                 text=True).stdout
        for name, code in kernels(listing):
            seen += 1
            bad = [(code[a].text, code[b].text, s) for a, b, s in early_reads(code)]
            assert not bad, (name, bad[:5])
    assert seen > 100
