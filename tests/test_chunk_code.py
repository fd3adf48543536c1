"""The generated code of chunk attention, gathered weights and eviction (CPU only).

As for the attention kernels: a matrix product's registers may not be touched until it
has ended, which is twelve wait states after a 32x32x16 product (eight passes, four
more on gfx950); the compiler was seen to leave the wait out behind a branch.  A
product may not write over its operands either, which the compiler was seen to let one
do whose sum starts from a constant.  Scratch memory and spilled vector registers
are refused.
"""

import os
import re
import subprocess

import pytest

from tests.test_attention_code import kernels, registers

build = pytest.importorskip("mqa_logits_amd.build")

WAIT_STATES = 12
PASSES = 8                                   # until the next product starts
PRODUCTS = ("v_mfma_f32_32x32x16_f16", "v_mfma_f32_32x32x16_bf16")


def operands_of(text):
    return [registers(x) for x in re.split(r",\s*(?![^\[]*\])", text)[:4]]


def early_uses(code, labels, need=WAIT_STATES):
    """(product, use) index pairs where some path leaves fewer wait states between them."""
    bad = []
    for start, (op, text) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        assert op in PRODUCTS, f"wait states of {op} are not known here"
        result = operands_of(text)[0]
        paths, most = [(start + 1, need)], {}
        while paths:
            i, left = paths.pop()
            while left > 0 and i < len(code) and most.get(i, 0) < left:
                most[i] = left
                op, text = code[i]
                if op.startswith("v_mfma"):
                    into, a, b, _ = operands_of(text)
                    if (a | b) & result:
                        bad.append((start, i))
                        break
                    if into & result:        # an accumulation, which the hardware chains, starts anew
                        break
                    left -= PASSES
                elif op == "s_nop":
                    left -= int(text, 0) + 1
                elif op == "s_endpgm":
                    break
                elif op == "s_branch":
                    i, left = labels[text.strip()], left - 1
                    continue
                elif op.startswith("s_"):
                    left -= 1
                    if op.startswith("s_cbranch"):
                        paths.append((labels[text.strip()], left))
                    assert not op.startswith(("s_setpc", "s_swappc", "s_call")), op
                elif registers(text) & result:
                    bad.append((start, i))
                    break
                else:
                    left -= 1
                i += 1
    return bad


@pytest.fixture(scope="module", params=["chunk", "weights", "evict"])
def assembly(request, tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    source = os.path.join(build.CSRC, request.param + ".hip")
    out = str(tmp_path_factory.mktemp("asm") / (request.param + ".s"))
    subprocess.run([build.HIPCC, *build.COMMON_FLAGS, "-S", "--cuda-device-only", source, "-o", out], check=True,
                   capture_output=True)
    with open(out) as f:
        return request.param, f.read()


def test_products_end_before_their_registers_are_used(assembly):
    which, text = assembly
    products = 0
    for name, code, labels in kernels(text):
        products += sum(op in PRODUCTS for op, _ in code)
        bad = early_uses(code, labels)
        assert not bad, f"{name}: {[(code[i], code[j]) for i, j in bad[:5]]}"
    assert products > {"chunk": 400, "weights": 300, "evict": -1}[which]


def test_products_leave_their_operands(assembly):
    for name, code, _ in kernels(assembly[1]):
        for op, text in code:
            if op in PRODUCTS:
                d, a, b, c = operands_of(text)
                assert not d & (a | b) and (c == d or not c & d), f"{name}: {op} {text}"


def test_no_scratch_and_no_spilled_vector_registers(assembly):
    which, text = assembly
    found = re.findall(r"\.name:\s*(\S+)\s.*?\.private_segment_fixed_size:\s*(\d+)"
                       r".*?\.vgpr_spill_count:\s*(\d+)", text, re.S)
    assert len(found) >= {"chunk": 8, "weights": 9, "evict": 8}[which]
    assert [f for f in found if f[1:] != ("0", "0")] == []
    assert "scratch_" not in text


HEAD = "_Z1k:\n v_mfma_f32_32x32x16_f16 v[0:15], v[20:23], v[24:27], v[0:15]\n"


@pytest.mark.parametrize("body,early", [
    (" s_nop 11\n v_add_f32 v35, v0, v1\n s_endpgm", False),
    (" s_nop 10\n v_add_f32 v35, v0, v1\n s_endpgm", True),
    (" v_mfma_f32_32x32x16_f16 v[40:55], v[20:23], v[24:27], 0\n s_nop 3\n v_add_f32 v35, v0, v1\n s_endpgm", False),
    (" v_mfma_f32_32x32x16_f16 v[40:55], v[20:23], v[24:27], 0\n s_nop 2\n v_add_f32 v35, v0, v1\n s_endpgm", True),
    (" s_cbranch_vccz .LBB0_1\n s_endpgm\n.LBB0_1:\n v_add_f32 v35, v15, v40\n s_endpgm", True),
])
def test_the_walk_itself(body, early):
    (_, code, labels), = kernels(HEAD + body)
    assert bool(early_uses(code, labels)) == early
