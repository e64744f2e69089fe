"""Which block shape the experts' training takes, on the host: the rule's header
compiled by itself, its count of tiles against counting them, and its choices on
both sides of each crossing."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_moe_layer_route_amd", "csrc")
GATE_UP, DOWN, DACT, DX, DW = range(5)
NAMES = ["256x256", "256x128", "128x64", "64x64"]

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include "ffn_train_shapes.h"
int main() {
  char what[8];
  long long v[6];
  while (std::scanf("%7s %lld %lld %lld %lld %lld %lld", what, v, v + 1, v + 2, v + 3, v + 4, v + 5) == 7)
    if (!std::strcmp(what, "tiles"))
      std::printf("%lld\n", (long long)moe::train_row_tiles(v[0], v[1], v[2], v[3], v[4]));
    else
      std::printf("%d\n", (int)moe::train_shape_of((moe::train_launch)v[0], v[1] != 0, v[2], v[3], v[4], v[5]));
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("shapes")
    (at / "p.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(at / "p.cpp"), "-o", str(at / "p")],
                   check=True)

    def run(lines):
        text = "\n".join(" ".join(map(str, q)) for q in lines) + "\n"
        r = subprocess.run([str(at / "p")], input=text, check=True, capture_output=True, text=True)
        return [int(v) for v in r.stdout.split()]
    return run


def shape(ask, which, dtype, P, E, H, I):
    return NAMES[ask([("shape", which, int(dtype == "bf16"), P, E, H, I)])[0]]


def test_tiles_are_counted(ask):
    rng = random.Random(5)
    cases = []
    for _ in range(400):
        E, n, m = rng.randint(1, 64), rng.choice([64, 128, 256]), rng.choice([64, 128, 256])
        cases.append((rng.randint(1, 1 << rng.randint(1, 25)), E, 16 * rng.randint(1, 300), n, m))
    cases += [(P, 1, w, 128, 256) for P in (128, 10400) for w in (16, 240, 256, 272, 512, 2048)]
    got = ask([("tiles", *c, 0) for c in cases])
    for (P, E, width, n, m), tiles in zip(cases, got):
        across = len(range(0, width, m))
        assert tiles % across == 0
        # as many parts of tiles as there can be: an expert's last row begins one
        ones = min(E, P)
        counts = [1] * ones
        counts[0] += (P - ones) // n * n
        counts[-1] += (P - ones) % n
        need = sum(-(-c // n) for c in counts) * across
        assert need <= tiles <= need + across * 2
        for _ in range(5):                     # any other way of sharing the rows out
            cuts = sorted(rng.randint(0, P) for _ in range(E - 1))
            parts = [b - a for a, b in zip([0] + cuts, cuts + [P])]
            assert sum(-(-c // n) for c in parts) * across <= tiles


def test_narrow_outputs_are_not_counted_twice(ask):
    """One expert, 10400 rows: 82 tiles of 256 outputs leave most CUs without one."""
    for which in (DOWN, DX):
        assert shape(ask, which, "bf16", 10400, 1, 256, 1024) == "128x64"
    assert shape(ask, DACT, "bf16", 10400, 1, 1024, 256) == "128x64"
    assert shape(ask, GATE_UP, "bf16", 16384 - 128, 1, 512, 128) == "128x64"
    # width 64: one tile across, not 1.25
    assert shape(ask, DOWN, "bf16", 128 * 170, 1, 64, 512) == "128x64"


def test_few_tiles_take_no_blocks_that_fill_a_cu(ask):
    """A shared expert's dx, 256 to 4096 rows: 16 to 136 tiles of 256x256 for 256 CUs."""
    for rows in (256, 1024):
        assert shape(ask, DX, "bf16", rows, 1, 2048, 2048) == "128x64"
    assert shape(ask, DX, "bf16", 4096, 1, 2048, 2048) == "256x128"


def test_both_sides_of_each_crossing(ask):
    # tiles of 256x128: rows / 128 + 1 for one expert, times the tiles across
    for which, H, I, last in ((DOWN, 256, 512, 192), (DX, 256, 512, 192), (DACT, 512, 256, 192),
                              (GATE_UP, 512, 128, 176)):
        assert shape(ask, which, "bf16", (last - 1) * 128, 1, H, I) == "128x64"
        assert shape(ask, which, "bf16", last * 128, 1, H, I) == "256x128"
    for E, want in ((16, "128x64"), (17, "256x128")):              # 12 tiles of dW an expert
        assert shape(ask, DW, "bf16", 4096, E, 256, 512) == want
    # dx of matrices past an XCD's L2: 256 rows an expert and four rounds of tiles
    assert shape(ask, DX, "bf16", 256 * 124, 4, 2048, 2048) == "256x256"          # 128 by 8
    assert shape(ask, DX, "bf16", 256 * 124 - 1, 4, 2048, 2048) == "256x128"
    assert shape(ask, DX, "bf16", 256 * 124, 4, 2048, 2032) == "256x128"
    assert shape(ask, DX, "bf16", 256 * 64, 64, 4096, 2048) == "256x256"
    assert shape(ask, DX, "bf16", 256 * 64 - 1, 64, 4096, 2048) == "256x128"
    # few rows an expert
    assert shape(ask, DOWN, "bf16", 64 * 8 - 1, 8, 2048, 512) == "64x64"
    assert shape(ask, DOWN, "bf16", 64 * 8, 8, 2048, 512) == "128x64"
    assert shape(ask, DX, "bf16", 64, 64, 2048, 512) == "256x128"   # 64 experts, 8 tiles each: 512
    assert shape(ask, DX, "bf16", 63, 64, 2048, 512) == "128x64"
    assert {shape(ask, w, "bf16", 64, 64, 4096, 4096) for w in (GATE_UP, DACT)} == {"128x64"}
    # fp32: tiles of 128x64
    for which, H, I in ((DOWN, 128, 512), (DX, 128, 512), (DACT, 512, 128)):
        assert shape(ask, which, "f32", 766 * 64, 1, H, I) == "64x64"
        assert shape(ask, which, "f32", 767 * 64, 1, H, I) == "128x64"
    assert shape(ask, GATE_UP, "f32", 1, 1, 64, 16) == "128x64"
    for E, want in ((21, "64x64"), (22, "128x64")):                 # 12 tiles of 256x128 an expert
        assert shape(ask, DW, "f32", 4096, E, 256, 512) == want
