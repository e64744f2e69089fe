"""The experts' training kernels as they are compiled: which there are, and that
nothing comes between what their inline assembly counts on."""
import importlib.util
import os
import random
import re
import subprocess

import pytest

from test_ffn_train_hazards import registers
from test_ffn_train_shapes import DACT, DOWN, DW, DX, GATE_UP, NAMES, ask  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_moe_layer_route_amd")
MODES = ["GATE_UP", "GATE_UP8", "DOWN", "DACT", "DACT8", "DX", "DW", "DW_ANY"]
SHAPES = {("2", "2", "8", "8"): "256x256", ("2", "2", "8", "4"): "256x128", ("1", "4", "8", "1"): "128x64",
          ("1", "4", "4", "1"): "64x64"}


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """The assembly of each kernel by (mode, type, shape)."""
    spec = importlib.util.spec_from_file_location("_build_flags", os.path.join(PKG, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    try:
        hipcc = build._hipcc()
    except RuntimeError:
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("assembly") / "ffn_train.s"
    subprocess.run([hipcc, *build.CFLAGS, "--offload-device-only", "-S",
                    os.path.join(PKG, "csrc", "ffn_train_gemm.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    found = {}
    for name, body in re.findall(r"^(\S*train_gemm_kernel\S*?):[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(),
                                 re.S | re.M):
        mode, ty, *sizes = re.search(r"ILi(\d)ENS0_5ShapeI(NS_4bf16E|f)Li(\d)ELi(\d)ELi(\d)ELi(\d)E", name).groups()
        found[MODES[int(mode)], "f32" if ty == "f" else "bf16", SHAPES[tuple(sizes)]] = body
    return found


def test_every_kernel_is_one_that_a_call_reaches(kernels, ask):  # noqa: F811
    """Those compiled are those that the shape rule chooses over batches of all sizes."""
    modes = {GATE_UP: ["GATE_UP", "GATE_UP8"], DOWN: ["DOWN"], DACT: ["DACT", "DACT8"], DX: ["DX"]}
    rng, queries = random.Random(8), []
    size = lambda most: int(2 ** rng.uniform(0, most))  # noqa: E731
    for _ in range(4000):
        queries.append(("shape", rng.randrange(5), rng.randrange(2), size(17), size(6.02), 64 * size(6), 16 * size(8)))
    queries.append(("shape", DX, 1, 32768, 64, 3584, 2560))
    reached = set()
    for (_, which, bf16, *_sizes), s in zip(queries, ask(queries)):
        ty = "bf16" if bf16 else "f32"
        # fp32 gradients of the weights always take the general form
        for mode in modes.get(which, ["DW", "DW_ANY"] if bf16 else ["DW_ANY"]):
            reached.add((mode, ty, NAMES[s]))
    assert set(kernels) == reached


def by_the_compiler(body):
    """(line, instruction) of all that does not come from inline assembly."""
    ours = False
    for i, line in enumerate(body.split("\n")):
        ours = ours or "ASMSTART" in line
        text = line.split(";")[0].strip()
        if not ours and text and not text.startswith("."):
            yield i, text
        ours = ours and "ASMEND" not in line


@pytest.mark.parametrize("mode", ["DACT", "DACT8"])
def test_stages_of_kept_rows_wait_by_count_alone(kernels, mode):
    """Between the first store of dact's outputs and the last the compiler waits
    for no load of its own: it would drain the stream, which it does not see."""
    code = list(by_the_compiler(kernels[mode, "bf16", "256x128"]))
    stores = [i for i, text in code if text.startswith("global_store")]
    for i, text in code:
        if stores[0] < i < stores[-1]:
            assert "vmcnt" not in text and not text.startswith(("scratch_", "global_load", "flat_", "buffer_")), text


# ---------------------------------------------------- along all branches ----
def flow(body):
    """The instructions and, for each, those that can run right before it."""
    code, labels, jumps = [], {}, []
    for line in body.split("\n"):
        text = line.split(";")[0].strip()
        if text.endswith(":") and not text.startswith("#"):
            labels[text[:-1]] = len(code)
        elif text and not text.startswith((".", "#")):
            code.append(text)
    sources = [[i - 1] if i else [] for i in range(len(code) + 1)]
    for i, text in enumerate(code):
        op, _, to = text.partition(" ")
        if op.startswith(("s_branch", "s_cbranch")):
            jumps.append((i, labels[to.strip()]))
        if op in ("s_branch", "s_endpgm"):
            sources[i + 1].remove(i)
    for i, to in jumps:
        sources[to].append(i)
    return code, sources, jumps


def within(code, sources, i, states):
    """Instructions that may have run within so many wait states before code[i]."""
    seen, todo = {}, [(j, states) for j in sources[i]]
    while todo:
        j, left = todo.pop()
        if seen.get(j, 0) >= left:
            continue
        seen[j] = left
        nop = code[j].startswith("s_nop")
        left -= int(code[j].split()[1]) + 1 if nop else 1
        if left > 0:
            todo += [(k, left) for k in sources[j]]
    return [code[j] for j in seen if not code[j].startswith("s_nop")]


def too_close(body):
    """As in test_ffn_train_hazards: a vector instruction that writes a matrix
    instruction's operand within 2 wait states before it, and any that touches its
    result within 18 after it."""
    code, sources, _ = flow(body)
    bad = []
    for i, text in enumerate(code):
        op, _, args = text.partition(" ")
        if op.startswith("v_mfma"):
            used = set().union(*map(registers, args.split(",")[1:]))
            for other in within(code, sources, i, 2):
                o, _, a = other.partition(" ")
                if o.startswith("v_") and not o.startswith("v_mfma") and registers(a.split(",")[0]) & used:
                    bad.append((other, text))
        else:
            used = {r for r in registers(args) if r[0] == "a"}
            for other in within(code, sources, i, 18) if used else ():
                o, _, a = other.partition(" ")
                if o.startswith("v_mfma") and registers(a.split(",")[0]) & used:
                    bad.append((other, text))
    return bad


MFMA = "v_mfma_f32_16x16x32_bf16 a[0:3], v[8:11], v[0:3], a[0:3]"


def test_the_reading_follows_branches():
    # a result read at the head of a loop that a matrix instruction ends
    assert too_close("\n".join([".L0:", "v_accvgpr_read_b32 v20, a1", "s_nop 15", "s_nop 15", MFMA,
                                "s_cbranch_scc1 .L0", "s_endpgm"]))
    assert not too_close("\n".join([".L0:", "v_accvgpr_read_b32 v20, a1", "s_nop 15", "s_nop 15", MFMA,
                                    "s_nop 15", "s_nop 15", "s_cbranch_scc1 .L0", "s_endpgm"]))
    # an operand written on one of two ways, with the other in between in the text
    ways = ["s_cbranch_scc1 .L1", "v_mov_b32_e32 v9, 0", "s_branch .L2", ".L1:", "s_nop 7", ".L2:", MFMA, "s_endpgm"]
    assert too_close("\n".join(ways))
    assert not too_close("\n".join(ways[:2] + ["s_nop 1"] + ways[2:]))
    # what an unconditional branch ends does not run into the next line
    assert not too_close("\n".join(["v_mov_b32_e32 v9, 0", "s_branch .L3", ".L2:", MFMA, ".L3:", "s_endpgm"]))


def test_no_instruction_is_too_close_along_any_branch(kernels):
    for name, body in kernels.items():
        bad = too_close(body)
        assert not bad, (name, bad[:3])


@pytest.mark.parametrize("mode,stages,stores", [("DACT", 8, 6), ("DACT8", 4, 12)])
def test_a_stage_of_kept_rows_has_the_stores_its_waits_count(kernels, mode, stages, stores):
    """ST in the kernel: fewer stores a stage than it says would let a wait pass
    before the loads that it is for."""
    code, _, _ = flow(kernels[mode, "bf16", "256x128"])
    runs, n = [], 0
    for text in code:
        if text == "s_barrier":
            runs.append(n)
            n = 0
        n += text.startswith("global_store")
    assert [r for r in runs + [n] if r] == [stores] * stages


def stage_loops(body):
    """First and last lines of the innermost loops around matrix instructions."""
    lines = body.split("\n")
    at = {line.split(":")[0]: i for i, line in enumerate(lines) if re.match(r"\.L\w+:", line)}
    loops = []
    for i, line in enumerate(lines):
        m = re.match(r"\s*s_c?branch\w* (\.L\w+)", line)
        if m and at[m[1]] < i and "v_mfma" in "\n".join(lines[at[m[1]]:i]):
            loops.append((at[m[1]], i))
    return [(a, b) for a, b in loops if not any((a, b) != (c, d) and a <= c and d <= b for c, d in loops)]


def test_stage_loops_wait_by_count_alone(kernels):
    """The innermost loops of the products hold no scratch access and no wait of
    the compiler's for a load (but for the rows that gate/up looks up for its next
    tile: two or three loads once a tile)."""
    for name, body in kernels.items():
        loops = stage_loops(body)
        assert loops, name
        mine, lines = dict(by_the_compiler(body)), body.split("\n")
        for a, b in loops:
            assert any("s_barrier" in line for line in lines[a:b]), name
            for i in range(a, b):
                text = mine.get(i, "")
                assert not text.startswith("scratch_"), (name, text)
                assert "vmcnt" not in text or name[0].startswith("GATE_UP"), (name, text)


def test_the_lds_address_register_is_the_loads_alone(kernels):
    """M0 is written by the inline assembly without a word to the compiler."""
    for name, body in kernels.items():
        assert not [text for _, text in by_the_compiler(body) if re.search(r"\bm0\b", text)], name
