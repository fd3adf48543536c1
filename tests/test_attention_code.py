"""The attention kernels' generated code (CPU only: hipcc writes the assembly).

A matrix product's registers may not be touched, or multiplied, until it has
ended: eight wait states after a 16x16x32 bf16 product (four passes, four more
on gfx950).  The hardware does not wait by itself, and the compiler was seen to
leave the wait out behind a branch that directly follows the product; the
kernels put one there by hand.  Every path from every product is walked here, so
that a new branch, or another compiler, cannot bring that back unnoticed.
Scratch memory and spilled vector registers are refused as well.  (Scalar
registers may spill: they go to lanes of vector registers.)
"""

import os
import re
import subprocess

import pytest

build = pytest.importorskip("mqa_logits_amd.build")

WAIT_STATES = 8
PRODUCT = "v_mfma_f32_16x16x32_bf16"


def registers(operand):
    """Vector and accumulator registers that an operand text names."""
    found = set()
    for bank, first, last, bank1, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", operand):
        if bank:
            found |= {(bank, i) for i in range(int(first), int(last) + 1)}
        else:
            found.add((bank1, int(one)))
    return found


def kernels(assembly):
    """(name, [(opcode, operands)], {label: index}) of every function."""
    parts = re.split(r"^(_Z\w+):", assembly, flags=re.M)
    for name, body in zip(parts[1::2], parts[2::2]):
        code, labels = [], {}
        for line in body.splitlines():
            line = line.split(";")[0].strip()
            label = re.match(r"(\.LBB\w+):", line)
            if label:
                labels[label.group(1)] = len(code)
            elif line and not line.startswith(".") and not line.endswith(":"):
                op, _, operands = line.partition(" ")
                code.append((op, operands))
        yield name, code, labels


def early_uses(code, labels, need=WAIT_STATES):
    """(product, use) index pairs where some path leaves fewer wait states between them."""
    bad = []
    for start, (op, operands) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        assert op == PRODUCT, f"wait states of {op} are not known here"
        result = registers(operands.split(",")[0])
        paths, most = [(start + 1, need)], {}
        while paths:
            i, left = paths.pop()
            while left > 0 and i < len(code) and most.get(i, 0) < left:
                most[i] = left
                op, operands = code[i]
                if op.startswith("v_mfma"):
                    into, a, b, _ = [registers(x) for x in re.split(r",\s*(?![^\[]*\])", operands)[:4]]
                    if (a | b) & result:
                        bad.append((start, i))
                        break
                    if into & result:        # an accumulation, which the hardware chains, starts anew
                        break
                    left -= 4
                elif op == "s_nop":
                    left -= int(operands, 0) + 1
                elif op == "s_endpgm":
                    break
                elif op == "s_branch":
                    i, left = labels[operands.strip()], left - 1
                    continue
                elif op.startswith("s_"):
                    left -= 1
                    if op.startswith("s_cbranch"):
                        paths.append((labels[operands.strip()], left))
                    assert not op.startswith(("s_setpc", "s_swappc", "s_call")), op
                elif registers(operands) & result:
                    bad.append((start, i))
                    break
                else:
                    left -= 1
                i += 1
    return bad


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = str(tmp_path_factory.mktemp("asm") / "attention.s")
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "-S", "--cuda-device-only",
                    os.path.join(build.CSRC, "attention.hip"), "-o", out], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


def test_products_end_before_their_registers_are_used(assembly):
    products = 0
    for name, code, labels in kernels(assembly):
        products += sum(op == PRODUCT for op, _ in code)
        bad = early_uses(code, labels)
        assert not bad, f"{name}: {[(code[i], code[j]) for i, j in bad[:5]]}"
    assert products > 1000


def test_no_scratch_and_no_spilled_vector_registers(assembly):
    found = re.findall(r"\.name:\s*(\S+)\s.*?\.private_segment_fixed_size:\s*(\d+)"
                       r".*?\.vgpr_spill_count:\s*(\d+)", assembly, re.S)
    assert sum("attention" in name for name, _, _ in found) >= 32
    assert [f for f in found if f[1:] != ("0", "0")] == []
    assert "scratch_" not in assembly


HEAD = "_Z1k:\n v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]\n"


@pytest.mark.parametrize("body,early", [
    (" s_nop 7\n v_add_f32 v5, v0, v1\n s_endpgm", False),
    (" s_nop 6\n v_add_f32 v5, v0, v1\n s_endpgm", True),
    (" s_nop 6\n v_mov_b32 v3, 0\n s_endpgm", True),                       # a write
    (" s_nop 6\n global_load_dwordx4 v[2:5], v9, s[0:1]\n s_endpgm", True),
    (" s_nop 6\n v_add_f32 v5, v4, v6\n v_add_f32 v5, v0, v1\n s_endpgm", False),
    (" s_cbranch_vccz .LBB0_1\n s_nop 6\n v_add_f32 v5, v0, v1\n s_endpgm\n.LBB0_1:\n s_endpgm", False),
    (" s_cbranch_vccz .LBB0_1\n s_endpgm\n.LBB0_1:\n v_add_f32 v5, v0, v1\n s_endpgm", True),
    (" s_branch .LBB0_2\n.LBB0_1:\n v_add_f32 v5, v0, v1\n s_endpgm\n.LBB0_2:\n s_branch .LBB0_1", True),
    (" v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], v[0:3]\n s_nop 7\n v_add_f32 v5, v0, v1\n s_endpgm", False),
    (" v_mfma_f32_16x16x32_bf16 v[4:7], v[0:3], v[12:15], 0\n s_endpgm", True),
    (" v_mfma_f32_16x16x32_bf16 v[4:7], v[8:11], v[12:15], 0\n s_nop 3\n v_add_f32 v9, v0, v1\n s_endpgm", False),
    (".LBB0_1:\n s_cbranch_scc1 .LBB0_1\n s_endpgm", False),
])
def test_the_walk_itself(body, early):
    (_, code, labels), = kernels(HEAD + body)
    assert bool(early_uses(code, labels)) == early
