"""The experts' training operators where the block shapes change and where experts
share the rows unevenly, against their formulas in 64 bits; the tolerances are
those of test_gpu_ffn_train.py, element by element."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_ffn_train import Case, say  # noqa: E402
from test_gpu_ffn_train_large import check_backward, check_forward  # noqa: E402

CASES = [  # T, H, I, E, k, dtype, keep, missing
    (3000, 320, 1296, 5, 2, "bf16", "rows", 0.2),      # dact by 256 x 128, its neighbours by 128 x 64
    (10400, 256, 272, 1, 1, "bf16", "rows", 0.0),      # 82 tiles: 128 x 64
    (24576, 256, 272, 1, 1, "bf16", "int8", 0.0),      # 193: down and dx by 256 x 128
    (64, 2048, 48, 64, 6, "bf16", "rows", 0.1),        # dx of few rows by 256 x 128
    (63, 2048, 48, 64, 4, "bf16", "int8", 0.1),        # and by 128 x 64
    (4000, 8192, 528, 2, 2, "bf16", "rows", 0.1),      # dx by 256 x 256
    (9001, 8256, 512, 1, 1, "bf16", "int8", 0.0),      # the same with ragged ends
    (1500, 128, 2064, 6, 2, "f32", "rows", 0.1),       # fp32 dact and dw by 128 x 64
    (1500, 2112, 144, 6, 2, "f32", "int8", 0.1),       # fp32 down and dx
]


@pytest.mark.parametrize("T,H,I,E,k,dtype,keep,miss", CASES)
def test_forward_and_backward(T, H, I, E, k, dtype, keep, miss):
    say(f"[ffn shapes] T={T} H={H} I={I} E={E} k={k} {dtype} {keep} miss={miss}")
    c = Case(T, H, I, E, k, dtype, keep, miss, pack=False)
    check_forward(c, *c.train())
    check_backward(c, c.backward())


@pytest.mark.parametrize("dtype,keep", [("bf16", "rows"), ("bf16", "int8"), ("f32", "rows")])
@pytest.mark.parametrize("counts", [[3800, 0, 1, 129], [0, 3999, 0, 0], [1, 127, 2000, 1500]])
def test_uneven_experts_by_large_shapes(counts, dtype, keep):
    say(f"[ffn shapes uneven] {counts} {dtype} {keep}")
    c = Case(2000, 1536, 1552, 4, 2, dtype, keep, counts=counts, pack=False)
    check_forward(c, *c.train())
    got = c.backward()
    check_backward(c, got)
    for e, n in enumerate(counts):
        if n == 0:
            assert not any(bool(v[e].any()) for v in got[1:])


@pytest.mark.parametrize("T,H,I,E,dtype,dw", [(1500, 128, 2064, 6, "f32", "same"), (3000, 320, 1296, 5, "bf16", "same"),
                                               (3000, 320, 1296, 5, "bf16", "f32"), (900, 128, 144, 5, "bf16", "f32")])
def test_gradients_added_twice(T, H, I, E, dtype, dw):
    """Added to zeros they are what is overwritten; added again, exactly twice that."""
    c = Case(T, H, I, E, 2, dtype, "rows", 0.1, pack=False)
    once, twice = c.backward(c.grads(dw)), c.grads(dw)
    for v in twice[1:]:
        v.zero_()
    c.backward(twice, accumulate_dw=True)
    assert all(torch.equal(a, b) for a, b in zip(once, twice))
    c.backward(twice, accumulate_dw=True)
    assert all(torch.equal(2 * a, b) for a, b in zip(once[1:], twice[1:]))
