"""Code-generation checks on the kernels around the GLU (norms, linear products, routing),
compiled here for gfx950 (CPU only): what the results cannot show reliably.
  * no packed-FP32 VALU instruction;
  * no store's data registers written by the instruction after it, and no 16-byte buffer store
    with a scalar offset register (the compiler leaves no wait behind such a store, and its last
    lanes then store what the next instruction wrote);
  * the 256 x 256 product keeps its sums and fragments in registers through the steady loop, and
    copies its operands straight into LDS.
"""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from glu_activation_microscaling_amd import build

SOURCES = ["glu_norm.hip", "glu_linear.hip", "glu_moe.hip"]
PACKED_FP32 = re.compile(r"^\s+v_pk_(fma|mul|add)_f32\b", re.M)
STORE = re.compile(r"(buffer|global|flat)_store_dwordx[34] ")

pytestmark = pytest.mark.skipif(
    shutil.which(os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc")) is None,
    reason="hipcc not available")


@pytest.fixture(scope="module")
def asm():
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(build.device_asm, SOURCES)))


def instructions(text):
    lines = (l.strip() for l in text.split("\n") if l.startswith("\t"))
    return [l.split(";")[0].strip() for l in lines if not l.startswith((".", ";"))]


def registers(operand):
    """(first, last) vector register of an operand, or None."""
    m = re.fullmatch(r"v\[(\d+):(\d+)\]", operand) or re.fullmatch(r"v(\d+)", operand)
    return None if m is None else (int(m.group(1)), int(m.group(m.lastindex)))


def hazards(code):
    """Wide stores whose registers the next instruction writes, or with a scalar offset register."""
    out = []
    for at, op in enumerate(code):
        m = STORE.match(op)
        if m is None:
            continue
        args = op.split(None, 1)[1].split(", ")
        if m.group(1) == "buffer" and re.match(r"s\d", args[3]):
            out.append(op)
        data = registers(args[0] if m.group(1) == "buffer" else args[1])
        after = code[at + 1].split(None, 1) if at + 1 < len(code) else [""]
        written = registers(after[1].split(",")[0]) if after[0].startswith("v_") and len(after) > 1 else None
        if data and written and written[0] <= data[1] and written[1] >= data[0]:
            out.append(op + " | " + " ".join(after))
    return out


def test_the_hazard_check_sees_one():
    assert hazards(["buffer_store_dwordx4 v[6:9], v37, s[8:11], s4 offen", "v_or_b32_e32 v1, 64, v34"])
    assert hazards(["buffer_store_dwordx4 v[6:9], v37, s[8:11], 0 offen", "v_or_b32_e32 v6, 64, v34"])
    assert hazards(["global_store_dwordx4 v0, v[6:9], s[2:3]", "v_mov_b64_e32 v[8:9], 0"])
    assert not hazards(["buffer_store_dwordx4 v[6:9], v37, s[8:11], 0 offen", "s_nop 0", "v_or_b32_e32 v6, 64, v34"])


@pytest.mark.parametrize("src", SOURCES)
def test_no_packed_fp32_instructions(asm, src):
    found = PACKED_FP32.findall(asm[src])
    assert not found, f"{src}: {len(found)} packed-FP32 instructions"


@pytest.mark.parametrize("src", SOURCES)
def test_stores_keep_their_registers(asm, src):
    found = hazards(instructions(asm[src]))
    assert not found, f"{src}: {found[:5]}"


@pytest.mark.parametrize("mode", [0, 1, 2])
def test_the_large_product_s_steady_loop(asm, mode):
    """The innermost loop with two steps' 128 matrix instructions: 16 copies into LDS, no scratch."""
    m = re.search(r"^(_Z\S*k_productILi%dELi0ELi2ELi4ELi8ELi4ELi2E\S*):" % mode, asm["glu_linear.hip"], re.M)
    body = asm["glu_linear.hip"][m.end():]
    body = body[:body.index(".Lfunc_end")].split("\n")
    labels, loops = {}, []
    for at, line in enumerate(body):
        label = re.match(r"(\.LBB\S+):", line)
        if label:
            labels[label.group(1)] = at
        branch = re.search(r"s_cbranch\S*\s+(\.LBB\S+)", line)
        if branch and branch.group(1) in labels:
            loop = body[labels[branch.group(1)]:at]
            if sum("v_mfma" in l for l in loop) >= 128:
                loops.append(loop)
    steady = min(loops, key=len)
    assert sum("v_mfma_f32_16x16x32_bf16" in l for l in steady) == 128
    assert sum(re.search(r"buffer_load_dwordx4 .* lds", l) is not None for l in steady) == 16
    assert not any("scratch_" in l for l in steady)
