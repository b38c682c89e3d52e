"""No kernel of the built library reads a matrix product's result before it is there.

The matrix instructions write their results some issue slots after they were issued, and on
gfx950 waiting that long is left to the program.  The compiler counts the slots, but across
branches it has been seen to count along the longer of two paths (hipcc 7.2: 4 slots of 18),
which gives wrong sums for some inputs only.  So every path from a product to the first other
instruction that touches its result is walked here, in the disassembly of the library as built.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

ROCM_LLVM = os.environ.get("ROCM_LLVM", "/opt/rocm/llvm/bin")
OBJDUMP = os.path.join(ROCM_LLVM, "llvm-objdump")

# slots between a product and arithmetic, memory or export on its result
NEED = {"v_mfma_f32_32x32x2_f32": 18, "v_mfma_f32_32x32x16_bf16": 11, "v_mfma_f32_32x32x16_f16": 11}
# a product behind another waits for the matrix unit itself, 8 slots at least
PRODUCT = 8

REGISTER = re.compile(r"\b([av])(?:\[(\d+):(\d+)\]|(\d+)\b)")
LINE = re.compile(r"\t([a-z]\w+)\s*([^/]*)")


def registers(text):
    out = set()
    for kind, lo, hi, one in REGISTER.findall(text):
        lo, hi = (int(lo), int(hi)) if lo else (int(one), int(one))
        out.update((kind, i) for i in range(lo, hi + 1))
    return out


def kernels(text):
    """(name, [(opcode, operands)], {label: index}) of each function of a disassembly."""
    name, code, labels = None, [], {}
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(\S+)>:", line)
        if head and not re.fullmatch(r"L\d+", head.group(1)):
            if name:
                yield name, code, labels
            name, code, labels = head.group(1), [], {}
            continue
        label = re.match(r"(?:[0-9a-f]+ )?<(L\d+)>:", line)
        if label:
            labels[label.group(1)] = len(code)
            continue
        ins = LINE.match(line)
        if ins:
            code.append((ins.group(1), ins.group(2).strip()))
    if name:
        yield name, code, labels


def after(code, labels, i):
    op, operands = code[i]
    if op == "s_endpgm":
        return []
    if op == "s_branch":
        return [labels[operands]]
    if op.startswith("s_cbranch"):
        return [i + 1, labels[operands]]
    return [i + 1] if i + 1 < len(code) else []


def early_reads(code, labels):
    """[(slots, needed, product's index, reader's index)] of products that are read too soon."""
    found = []
    for i, (op, operands) in enumerate(code):
        if op not in NEED:
            continue
        result = registers(operands.split(",")[0])
        best, work = {}, [(j, 0) for j in after(code, labels, i)]
        while work:
            j, slots = work.pop()
            if slots >= NEED[op] or best.get(j, 1 << 30) <= slots:
                continue
            best[j] = slots
            other, text = code[j]
            product = other.startswith("v_mfma")
            if registers(text) & result:
                parts = text.split(",")
                # a product that goes on adding to the result is ordered by the hardware
                if not product or (registers(parts[1]) | registers(parts[2])) & result:
                    found.append((slots, NEED[op], i, j))
                continue
            step = PRODUCT if product else int(text, 0) + 1 if other == "s_nop" else 1
            work += [(k, slots + step) for k in after(code, labels, j)]
    return found


def test_the_walk_finds_an_early_read():
    """Planted listings: a read on the short path around an if, and the same after a wait."""
    listing = """
0000000000001900 <planted>:
\tv_mfma_f32_32x32x16_bf16 v[0:15], v[16:19], v[20:23], v[0:15]// 1: 0
\ts_cbranch_execz L0// 2: 0
\ts_nop 15// 3: 0
<L0>:
\tv_add_f32_e32 v30, v3, v31// 4: 0
\ts_endpgm// 5: 0
"""
    (name, code, labels), = kernels(listing)
    assert name == "planted" and early_reads(code, labels) == [(1, 11, 0, 3)]
    (_, code, labels), = kernels(listing.replace("\ts_cbranch", "\ts_nop 9// 0: 0\n\ts_cbranch"))
    assert early_reads(code, labels) == []
    (_, code, labels), = kernels(listing.replace("v_add_f32_e32 v30, v3, v31", "v_add_f32_e32 v30, v33, v31"))
    assert early_reads(code, labels) == []


@pytest.mark.slow
@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler for gfx950")
def test_products_are_awaited(tmp_path):
    from learned_image_compression_amd import build as hip_build
    from learned_image_compression_amd import layers as L
    if not os.path.exists(L.LIBRARY):
        hip_build.build()
    copy = tmp_path / "layers.so"
    shutil.copy(L.LIBRARY, copy)
    subprocess.run([OBJDUMP, "--offloading", copy.name], cwd=tmp_path, check=True, capture_output=True)
    objects = sorted(p for p in tmp_path.iterdir() if p.name.endswith("gfx950"))
    assert objects
    with_products = 0
    for obj in objects:
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--symbolize-operands", obj.name], cwd=tmp_path,
                              check=True, capture_output=True, text=True).stdout
        if "v_mfma" not in text:
            continue
        for name, code, labels in kernels(text):
            unknown = {op for op, _ in code if op.startswith("v_mfma")} - set(NEED)
            assert not unknown, (name, unknown)
            with_products += any(op in NEED for op, _ in code)
            assert early_reads(code, labels) == [], name
    assert with_products >= 50  # four widths and the odd one, four kernels, three types
