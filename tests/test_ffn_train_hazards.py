"""The experts' training kernels write their matrix instructions as inline
assembly, whose hazards the compiler does not see.  This compiles them to
assembly and checks that around each one no other instruction comes too close:
a vector instruction that writes one of its operands needs 2 wait states before
it, and one that touches its result 18 after it."""
import importlib.util
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_moe_layer_route_amd")


def registers(text):
    out = set()
    for bank, lo, hi, one, n in re.findall(r"\b([av])\[(\d+):(\d+)\]|\b([av])(\d+)\b", text):
        out |= {(bank, i) for i in range(int(lo), int(hi) + 1)} if bank else {(one, int(n))}
    return out


def instructions(body):
    for line in body.split("\n"):
        text = line.split(";")[0].strip()
        if text and not text.startswith((".", "#")):
            yield text


def before(code, i, states):
    """Instructions within so many wait states before code[i], in textual order."""
    while i > 0 and states > 0:
        i -= 1
        if code[i].startswith("s_nop"):
            states -= int(code[i].split()[1]) + 1
        else:
            yield code[i]
            states -= 1


def hazards(code):
    bad = []
    for i, text in enumerate(code):
        op, _, args = text.partition(" ")
        if op.startswith("v_mfma"):
            used = set().union(*map(registers, args.split(",")[1:]))
            for other in before(code, i, 2):
                o, _, a = other.partition(" ")
                if o.startswith("v_") and not o.startswith("v_mfma") and registers(a.split(",")[0]) & used:
                    bad.append((other, text))
        else:
            used = {r for r in registers(args) if r[0] == "a"}
            for other in before(code, i, 18) if used else ():
                o, _, a = other.partition(" ")
                if o.startswith("v_mfma") and registers(a.split(",")[0]) & used:
                    bad.append((other, text))
    return bad


def test_the_reading_sees_both_kinds():
    assert hazards(["v_accvgpr_write_b32 a7, v4", "v_mfma_f32_16x16x32_bf16 a[4:7], v[8:11], v[0:3], a[4:7]"])
    assert hazards(["v_mfma_f32_16x16x32_bf16 a[4:7], v[8:11], v[0:3], a[4:7]", "s_nop 15",
                    "v_accvgpr_read_b32 v1, a5"])
    assert not hazards(["v_mov_b32_e32 v9, 0", "s_nop 1", "v_mfma_f32_16x16x4_f32 a[0:3], v9, v2, a[0:3]",
                        "s_nop 15", "s_nop 15", "v_accvgpr_read_b32 v1, a0"])


def test_no_instruction_too_close_to_a_matrix_instruction(tmp_path):
    spec = importlib.util.spec_from_file_location("_build_flags", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    out = tmp_path / "ffn_train.s"
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    subprocess.run([hipcc, *build.CFLAGS, "--offload-device-only", "-S",
                    os.path.join(PKG, "csrc", "ffn_train_gemm.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    kernels = re.findall(r"^(\S*train_gemm_kernel\S*?):[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(), re.S | re.M)
    assert len(kernels) > 20
    for name, body in kernels:
        code = list(instructions(body))
        assert any(c.startswith("v_mfma") for c in code)
        bad = hazards(code)
        assert not bad, (name, bad[:3])
