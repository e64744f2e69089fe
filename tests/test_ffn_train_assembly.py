"""The experts' training kernels as they are compiled: which there are."""
import importlib.util
import os
import random
import re
import subprocess

import pytest

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
