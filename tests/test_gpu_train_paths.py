"""Training operators on the GPU: kernel paths that the sizes of
test_gpu_train leave out, held against the same fp64 forms with the same
bounds, and rows of infinities and NaN in every kind of distillation block."""
import numpy as np
import pytest
import torch

import test_gpu_train as base      # skips this module, too, where there is no GPU
from gpu_harness import say
from oracle import train_oracle as TO
from test_gpu_train import TT, f64, gen, make_dims, near, randn

import sparse_moe_layer_route_amd as M

pytestmark = pytest.mark.gpu


# ------------------------------------------------- sorted rows and back ----
# every pair of types with every group of lanes (16, 32, 64, a block), for one
# or two slots (four units of a lane at once) and for more
ROWS = [  # T, H, k, dtype, rows, missing
    (50, 64, 2, "f32", "f32", 0.1), (45, 128, 2, "f32", "f32", 0.3), (333, 256, 2, "f32", "f32", 0.25),
    (30, 1088, 2, "f32", "f32", 0.2), (90, 128, 8, "f32", "f32", 0.1), (90, 256, 4, "f32", "f32", 0.1),
    (51, 128, 2, "bf16", "f32", 0.2), (40, 192, 1, "bf16", "f32", 0.2), (70, 512, 2, "bf16", "f32", 0.2),
    (9, 2112, 1, "bf16", "f32", 0.0), (20, 64, 3, "bf16", "f32", 0.1), (20, 256, 3, "bf16", "f32", 0.1),
    (61, 64, 1, "bf16", "bf16", 0.2), (37, 256, 2, "bf16", "bf16", 0.2), (2000, 1088, 2, "bf16", "bf16", 0.1),
    (40, 512, 8, "bf16", "bf16", 0.1),
]


@pytest.mark.parametrize("want_dy,want_dw", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("T,H,k,dtype,rows,miss", ROWS)
def test_undispatch_backward_groups(T, H, k, dtype, rows, miss, want_dy, want_dw):
    base.test_undispatch_backward(T, H, k, dtype, rows, miss, want_dy, want_dw)


@pytest.mark.parametrize("T,H,k,dtype,rows", [(10007, 2048, 2, "bf16", "bf16"), (20001, 1088, 2, "bf16", "bf16"),
                                              (10007, 1024, 2, "f32", "f32"), (20001, 1088, 1, "bf16", "f32")])
def test_undispatch_many_rows_of_few_slots(T, H, k, dtype, rows):
    say(f"[many rows] T={T} H={H} k={k} {dtype} rows={rows}")
    base.test_undispatch_many_rows(T, H, k, dtype, rows)


# -------------------------------------------------------- router gradient --
ROUTE = [  # T, H, E, k, dtype, renorm
    # one launch: one step of 32 tokens and two, one to four expert tiles
    (20, 192, 12, 2, "bf16", True), (50, 128, 12, 2, "bf16", False), (31, 64, 20, 3, "bf16", False),
    (50, 192, 30, 3, "bf16", True), (12, 320, 48, 4, "bf16", True), (30, 128, 64, 8, "bf16", True),
    (64, 2048, 64, 6, "bf16", False), (20, 128, 10, 2, "f32", True), (40, 128, 16, 2, "f32", False),
    (20, 192, 30, 2, "f32", True), (50, 192, 20, 4, "f32", True), (9, 192, 40, 3, "f32", False),
    # more tokens: two tiles of a bf16 layer (two waves a tile), three of an fp32 one
    (700, 192, 24, 4, "bf16", True), (300, 256, 40, 4, "f32", True), (150, 256, 24, 4, "f32", False),
    # fp32, a launch each for dW and dx
    (4200, 1344, 40, 2, "f32", True), (4200, 2048, 30, 2, "f32", False),
]


@pytest.mark.parametrize("T,H,E,k,dtype,renorm", ROUTE)
@pytest.mark.parametrize("form", ["weights", "both", "logits"])
def test_route_backward_paths(T, H, E, k, dtype, renorm, form):
    base.test_route_backward(T, H, E, k, dtype, renorm, form)


@pytest.mark.parametrize("T", [20, 60, 300])
def test_route_backward_of_the_largest_logit_gradients(T):
    """fp32's largest values, which no bf16 part can round to, are finite, and so
    are the products; infinite and NaN ones give NaN."""
    H, E = 192, 20
    g = gen(71 + T)
    say(f"[route_backward] T={T} largest logit gradients")
    x, w = randn(g, T, H, dtype="bf16", std=1e-3), randn(g, E, H, dtype="bf16", std=1e-3)
    add = randn(g, T, E)
    most = torch.finfo(torch.float32).max
    at = torch.arange(T, device="cuda")
    add[at, at % 7] = torch.where(at % 2 == 0, most, -most)
    add[at, 7 + at % 3] = torch.where(at % 3 == 0, 3.39e38, -3.3961e38)   # below and past half a step
    d = make_dims(H, E, 2, "bf16")
    dl, dx, dw = torch.empty_like(add), torch.empty_like(x), torch.empty(E, H, device="cuda")
    ws = torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, device="cuda")
    run = lambda: M.moe_route_backward(d, T, x, w, None, None, None, dl, dx, dw, ws, dlogits_add=add)
    run()
    rdx, rdw = TO.router_linear_backward(f64(add), f64(x), f64(w))
    mx, mw = TO.router_linear_backward(np.abs(f64(add)), np.abs(f64(x)), np.abs(f64(w)))
    near(dx, rdx, ((2 * E + 2) * base.U + 2.0 ** -16) * mx + base.HALF["bf16"] * 1.01 * np.abs(rdx), "dx")
    near(dw, rdw, (T + 8) * base.U * mw, "dw_router")
    add[3, 2], add[5, 4] = float("inf"), float("nan")
    run()
    assert torch.isnan(dx[3]).all() and torch.isnan(dx[5]).all()
    assert torch.isnan(dw[2]).all() and torch.isnan(dw[4]).all()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[[3, 5]] = False
    assert torch.isfinite(dx[rest]).all()
    assert torch.isfinite(dw[[e for e in range(E) if e not in (2, 4)]]).all()


@pytest.mark.parametrize("T,H,dtype", [((1 << 20) + 45, 2112, "bf16"), ((1 << 19) + 45, 4160, "f32")])
def test_route_backward_past_2_31_elements(T, H, dtype):
    """x and dx of more than 2^31 elements each.  Small whole numbers: every sum
    is below 2^24 (dx below 2^8) and exact."""
    E, k = 9, 4
    assert T * H > 1 << 31 and T < 1 << 24
    say(f"[route_backward] T={T} H={H} {dtype} whole numbers")
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    whole = lambda m, *shape: torch.randint(-m, m + 1, shape, generator=g, device="cuda", dtype=torch.int8)
    x, w = whole(1, T, H).to(TT[dtype]), whole(8, E, H).to(TT[dtype])
    add = whole(1, T, E).float()
    add[T // 2:T // 2 + 7] = 0.0
    d = make_dims(H, E, k, dtype)
    dl, dx, dw = torch.empty_like(add), torch.empty_like(x), torch.empty(E, H, device="cuda")
    ws = torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, device="cuda")
    M.moe_route_backward(d, T, x, w, None, None, None, dl, dx, dw, ws, dlogits_add=add)
    assert torch.equal(dl, add)
    want = torch.zeros(E, H, device="cuda")
    at = add.t().contiguous()
    for t0 in range(0, T, 65536):
        t1 = min(T, t0 + 65536)
        assert torch.equal(dx[t0:t1].float(), add[t0:t1] @ w.float()), t0
        want += at[:, t0:t1].contiguous() @ x[t0:t1].float()
    assert torch.equal(dw, want)


# ------------------------------------------------------------ distillation --
LONG = [  # T, V, K, dtype: about the longest rows of one block, odd lengths
    (66, 40001, 20, "f32"), (65, 128257, 64, "bf16"),
    (64, 65529, 9, "bf16"), (64, 65530, 9, "bf16"),        # 8192 and 8193 units
    (64, 131065, 9, "bf16"), (64, 131066, 9, "bf16"),      # 16384, and 16385: cut
    (64, 32765, 9, "f32"), (64, 32766, 9, "f32"), (64, 65533, 9, "f32"), (64, 65534, 9, "f32"),
    (63, 32771, 9, "bf16"), (64, 32771, 9, "bf16"),        # cut only below 64 rows
]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,V,K,dtype", LONG)
def test_distill_long_rows(T, V, K, dtype, tail):
    base.test_distill(T, V, K, dtype, False, 1.5, tail)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(12, 60), (12, 300), (12, 5000), (12, 40003), (70, 66001 // 2)])
def test_distill_infinities_and_nan(T, V, dtype, tail):
    """Rows in registers of a group, of a block, and cut into segments: a NaN of
    either sign and +inf end in NaN wherever they stand, -inf is a class with
    q = 0."""
    K, inf, nan = 6, float("inf"), float("nan")
    say(f"[distill] infinities T={T} V={V} {dtype} tail={tail}")
    s, ids, u, lse = base.distill_case(61 + V, T, V, K, dtype, False, 1.0, tail)
    head = torch.zeros(T, V, dtype=torch.bool).scatter_(1, ids.long(), True).cuda()
    free = [int((~head[t]).nonzero()[V // 3]) for t in range(T)]      # a class outside the K
    bits = {"bf16": (torch.int16, -64), "f32": (torch.int32, -(1 << 22))}[dtype]
    minus_nan = torch.tensor([bits[1]], dtype=bits[0]).view(TT[dtype]).cuda()
    assert torch.isnan(minus_nan).all() and torch.signbit(minus_nan).all()
    s[0, ids[0, 1].item()] = -inf                      # the teacher wants a masked class
    s[1, free[1]] = nan
    s[2] = -inf
    s[3, free[3]] = minus_nan[0]
    s[4] = -s[4].abs() - 1.0                           # a NaN of either sign beside negative values
    s[4, free[4]] = minus_nan[0]
    s[5] = -s[5].abs() - 1.0
    s[5, free[5]] = nan
    s[6, ids[6, 2].item()] = nan
    s[7, free[7]] = inf
    s[8, ids[8, 0].item()] = inf
    s[9][~head[9]] = -inf                              # no mass outside the K
    mask = (torch.arange(V) % 3 == 0).cuda() & ~head[10]
    s[10][mask] = -inf
    s[11] = torch.finfo(TT[dtype]).min
    ids, u = ids.cuda(), u.cuda()
    lse = None if lse is None else lse.cuda()
    want = s.clone()
    loss, ds = torch.full((T,), 3.0, device="cuda"), torch.full_like(s, 3.0)
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, s, ids, u, loss, ds, ws, teacher_lse=lse)
    for t in (1, 3, 4, 5, 6, 7, 8):
        assert torch.isnan(loss[t]) and torch.isnan(ds[t]).all(), t
    assert torch.isnan(loss[2])
    assert loss[0] == inf and torch.isfinite(ds[0]).all()
    assert torch.isfinite(ds[9:]).all() and torch.isfinite(loss[10:]).all()
    assert not ds[9][~head[9]].any() and not ds[10][mask].any()
    assert float(loss[9]) == inf if tail else torch.isfinite(loss[9])
    part = lambda t: None if t is None else t[10:]
    base.distill_check(s[10:], ids[10:], u[10:], part(lse), V, 1.0, None, 1.0, dtype, loss[10:], ds[10:])
    # Rows 0 and 9 have finite gradients: of a class with q = 0 it is -p.  A q is off by
    # the sum's delta and by 4 spread u of its own exponent: delta (1 + spread) covers
    # both, as delta >= 32 u; the joins and the rounding add to the value itself.
    for t in (0, 9):
        l = None if lse is None else f64(lse)[t:t + 1]
        _, rg = TO.distill(f64(s)[t:t + 1], ids[t:t + 1].cpu().numpy(), f64(u)[t:t + 1], 1.0, l)
        z = f64(s)[t]
        q = np.exp(z - z.max())
        spread = np.minimum(np.abs(z - z.max()), 110.0)
        delta = ((q / q.sum() * spread).sum() * 4 + V / 64 + 32) * base.U
        near(ds[t], rg[0], 4 * delta * (q / q.sum() + np.abs(rg[0])) * (1 + spread)
             + (base.HALF[dtype] + 4 * base.U) * np.abs(rg[0]) + 1e-37, f"dstudent of row {t}")
    assert torch.equal(s.view(bits[0]), want.view(bits[0]))          # the student is left alone
