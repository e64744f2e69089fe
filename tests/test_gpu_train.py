"""Training operators on the GPU against their fp64 forms (oracle.train_oracle).

Tolerances are rounding bounds, element by element: u = 2^-24 is half a step of
fp32, and a result stored in a type with half step h adds h relative to itself.
A sum of n fp32 products in any order is off by at most n u (sum of |products|)
to first order, each product or fused multiply-add by u of its own.
"""
import dataclasses

import numpy as np
import pytest
import torch

import workloads as W
from oracle import train_oracle as TO
from workloads.device import dims_dict, tensor, upload

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import sparse_moe_layer_route_amd as M  # noqa: E402
from gpu_harness import say  # noqa: E402

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return t.detach().cpu().double().numpy()


def randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(TT[dtype]).cuda()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def random_inv(g, T, k, miss):
    """Positions of a random order of the slots; a share of them missing."""
    P = T * k
    inv = torch.randperm(P, generator=g).to(torch.int32)
    inv[torch.rand(P, generator=g) < miss] = -1
    return inv.cuda()


def near(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} values off, first at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, allowed {np.broadcast_to(tol, got.shape)[i]!r}")


def make_dims(H, E, k, dtype, renorm=False):
    return M.Dims(hidden=H, n_experts=E, top_k=k, inter=64, dtype=dtype, renormalize=renorm)


# ------------------------------------------------- sorted rows and back ----
ROWS = [  # T, H, k, dtype, rows, missing
    (1, 64, 1, "bf16", "bf16", 0.0), (1, 2048, 6, "bf16", "f32", 0.0),
    (7, 64, 8, "f32", "f32", 0.3), (33, 192, 3, "bf16", "bf16", 0.5),
    (130, 320, 5, "bf16", "f32", 0.2), (64, 576, 8, "f32", "f32", 1.0),
    (513, 1536, 8, "bf16", "bf16", 0.1), (19, 4160, 2, "bf16", "bf16", 0.0),
    (300, 128, 7, "bf16", "bf16", 0.9),
]


@pytest.mark.parametrize("T,H,k,dtype,rows,miss", ROWS)
def test_dispatch(T, H, k, dtype, rows, miss):
    g = gen(T * 31 + H)
    say(f"[dispatch] T={T} H={H} k={k} {dtype}")
    x, inv = randn(g, T, H, dtype=dtype), random_inv(g, T, k, miss)
    out = torch.full((T * k, H), 7.0, dtype=TT[dtype], device="cuda")   # rows no slot names stay
    M.moe_dispatch(make_dims(H, 8, k, dtype), T, x, inv, out)
    want = TO.dispatch(f64(x), inv.cpu().numpy(), k, np.full((T * k, H), 7.0))
    assert np.array_equal(f64(out), want)


def undispatch_tol(y, inv, k, w, add, out, dtype):
    # k fused multiply-adds on top of add
    mag = TO.undispatch(np.abs(y), inv, k, None if w is None else np.abs(w),
                        None if add is None else np.abs(add))
    return (k + 1) * U * mag * 1.01 + HALF[dtype] * np.abs(out) * 1.01


@pytest.mark.parametrize("weighted,added", [(True, True), (False, False), (True, False), (False, True)])
@pytest.mark.parametrize("T,H,k,dtype,rows,miss", ROWS)
def test_undispatch(T, H, k, dtype, rows, miss, weighted, added):
    g = gen(T * 37 + H)
    say(f"[undispatch] T={T} H={H} k={k} {dtype} rows={rows} w={weighted} add={added}")
    y, inv = randn(g, T * k, H, dtype=rows), random_inv(g, T, k, miss)
    # a row that no slot names may hold anything
    named = torch.zeros(T * k, dtype=torch.bool, device="cuda")
    named[inv[inv >= 0].long()] = True
    y[~named] = float("nan")
    w = randn(g, T, k) if weighted else None
    add = randn(g, T, H, dtype=dtype) if added else None
    d = make_dims(H, 8, k, dtype)
    out = torch.empty(T, H, dtype=TT[dtype], device="cuda")
    M.moe_undispatch(d, T, y, inv, w, out, add=add)
    y64 = np.nan_to_num(f64(y))
    iv, w64 = inv.cpu().numpy(), None if w is None else f64(w)
    a64 = None if add is None else f64(add)
    want = TO.undispatch(y64, iv, k, w64, a64)
    near(out, want, undispatch_tol(y64, iv, k, w64, a64, want, dtype), "out")
    if added:                                            # in place
        M.moe_undispatch(d, T, y, inv, w, add, add=add)
        assert torch.equal(add, out)


@pytest.mark.parametrize("T,H,k,dtype,rows", [(6001, 1024, 8, "bf16", "bf16"), (4501, 1024, 8, "bf16", "f32"),
                                              (4501, 640, 8, "f32", "f32")])
def test_undispatch_many_rows(T, H, k, dtype, rows):
    """More bytes than the rows that stay in the caches; in 64 bits on the GPU."""
    g = gen(T + H)
    inv, y, w = random_inv(g, T, k, 0.2), randn(g, T * k, H, dtype=rows), torch.rand(T, k, generator=g).cuda()
    add, out = randn(g, T, H, dtype=dtype), torch.full((T, H), 3.0, dtype=TT[dtype], device="cuda")
    M.moe_undispatch(make_dims(H, 16, k, dtype), T, y, inv, w, out, add=add)
    at, want, size = inv.view(T, k).long(), add.double(), add.double().abs()
    for j in range(k):
        p = torch.where(at[:, j:j + 1] >= 0, w[:, j:j + 1].double() * y[at[:, j].clamp(min=0)].double(), 0.0)
        want += p
        size += p.abs()
    tol = (k + 1) * U * size + HALF[dtype] * 1.01 * want.abs()
    assert bool(((out.double() - want).abs() <= tol).all())
    # and back
    dy, dw = torch.zeros_like(y), torch.empty(T, k, device="cuda")
    M.moe_undispatch_backward(make_dims(H, 16, k, dtype), T, out, y, inv, w, dy, dw)
    for j in range(k):
        on, row = at[:, j] >= 0, at[:, j].clamp(min=0)
        p = out.double() * y[row].double()
        want, tol = p.sum(1), (H + 1) * U * p.abs().sum(1)
        assert bool(torch.where(on, (dw[:, j].double() - want).abs() <= tol, dw[:, j] == 0).all())
        want = w[:, j:j + 1].double() * out.double()
        ok = (dy[row].double() - want).abs() <= HALF[rows] * 1.01 * want.abs()
        assert bool((ok | ~on[:, None]).all())


@pytest.mark.parametrize("want_dy,want_dw", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("T,H,k,dtype,rows,miss", ROWS)
def test_undispatch_backward(T, H, k, dtype, rows, miss, want_dy, want_dw):
    g = gen(T * 41 + H)
    say(f"[undispatch_backward] T={T} H={H} k={k} {dtype} rows={rows} dy={want_dy} dw={want_dw}")
    y, inv = randn(g, T * k, H, dtype=rows), random_inv(g, T, k, miss)
    dout, w = randn(g, T, H, dtype=dtype), randn(g, T, k)
    dy = torch.full((T * k, H), 5.0, dtype=TT[rows], device="cuda") if want_dy else None
    dw = torch.full((T, k), 9.0, device="cuda") if want_dw else None
    M.moe_undispatch_backward(make_dims(H, 8, k, dtype), T, dout, y if want_dw else None, inv,
                              w if want_dy else None, dy, dw)
    iv, y64, d64, w64 = inv.cpu().numpy(), f64(y), f64(dout), f64(w)
    rdy, rdw = TO.undispatch_backward(d64, y64, iv, k, w64, np.full(y64.shape, 5.0))
    if want_dy:
        near(dy, rdy, (U + HALF[rows]) * 1.01 * np.abs(rdy), "dy_perm")
    if want_dw:
        _, mag = TO.undispatch_backward(np.abs(d64), np.abs(y64), iv, k, w64, np.zeros(y64.shape))
        # a lane's chain of eight products a unit, then the tree over the lanes
        near(dw, rdw, (H / 8 + 16) * U * mag + U * np.abs(rdw), "dtopk_w")


def test_sorted_rows_with_positions_out_of_range():
    T, H, k = 6, 64, 2
    g = gen(3)
    x = randn(g, T, H, dtype="bf16")
    inv = torch.tensor([0, -1, 12, 5, 2 ** 31 - 1, -2 ** 31, 3, 4, 1, 2, 11, 100], dtype=torch.int32).cuda()
    d = make_dims(H, 8, k, "bf16")
    rows = torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda")
    M.moe_dispatch(d, T, x, inv, rows)
    iv = inv.cpu().numpy()
    assert np.array_equal(f64(rows), TO.dispatch(f64(x), iv, k, np.zeros((T * k, H))))
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    M.moe_undispatch(d, T, rows, inv, None, out)
    want = TO.undispatch(f64(rows), iv, k)
    near(out, want, undispatch_tol(f64(rows), iv, k, None, None, want, "bf16"), "out")


# -------------------------------------------------------- router gradient --
ROUTE = [  # T, H, E, k, dtype, renorm
    (1, 64, 2, 1, "bf16", True), (1, 2048, 64, 6, "bf16", False), (5, 64, 64, 8, "f32", True),
    (37, 192, 40, 8, "bf16", True), (300, 576, 17, 3, "f32", False), (129, 1536, 40, 8, "bf16", False),
    (1030, 320, 64, 8, "bf16", True), (64, 4160, 33, 5, "bf16", True), (257, 256, 8, 2, "f32", True),
    (2200, 128, 1, 1, "bf16", False), (32, 640, 24, 4, "bf16", True), (33, 192, 48, 2, "f32", False),
    (64, 128, 64, 8, "f32", True), (65, 2048, 50, 4, "bf16", False), (4200, 1024, 60, 4, "f32", True),
]


def dlogits_bound(l, ids, g, renorm, add):
    """p off by delta relative: the difference l - m rounded once (|l - m| u),
    expf to 2 ulp, the sum over E terms, the division; then p (G - c)."""
    T, E = l.shape
    mass = np.abs(TO.route_weights(l, ids, renorm))
    p = np.zeros((T, E))
    G = np.zeros((T, E))
    n = np.zeros((T, E))
    for t in range(T):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if 0 <= e < E:
                G[t, e] += abs(g[t, j])
                n[t, e] += 1
                if renorm:
                    p[t, e] = mass[t, j]
    if not renorm:
        z = np.exp(l - l.max(1, keepdims=True))
        p = z / z.sum(1, keepdims=True)
    spread = np.abs(l - l.max(1, keepdims=True)).max(1, keepdims=True)
    delta = (spread + E + 16) * U
    c = (G * p).sum(1, keepdims=True)
    b = 2 * delta * p * (G + np.maximum(n, 1) * c)
    if add is not None:
        b = b + U * np.abs(add)
    return b


@pytest.mark.parametrize("T,H,E,k,dtype,renorm", ROUTE)
@pytest.mark.parametrize("form", ["weights", "both", "logits"])
def test_route_backward(T, H, E, k, dtype, renorm, form):
    g = gen(T * 43 + H)
    say(f"[route_backward] T={T} H={H} E={E} k={k} {dtype} renorm={renorm} {form}")
    x, w = randn(g, T, H, dtype=dtype), randn(g, E, H, dtype=dtype, std=0.05)
    logits = randn(g, T, E, std=2.0)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    if T > 4:
        ids[1] = -1                                   # a token without a slot
        ids[2, k // 2] = E                            # one id out of range
        ids[3] = ids[3, 0]                            # an expert named k times
    dtw = randn(g, T, k) if form != "logits" else None
    add = randn(g, T, E, std=0.1) if form != "weights" else None
    dxa = randn(g, T, H, dtype=dtype) if form == "both" else None
    d = make_dims(H, E, k, dtype, renorm)
    ws = torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, device="cuda")
    dl = torch.full((T, E), 3.0, device="cuda")
    dx = torch.full((T, H), 3.0, dtype=TT[dtype], device="cuda")
    dw = torch.full((E, H), 3.0, device="cuda")
    idc = ids.cuda()
    M.moe_route_backward(d, T, x, w, idc if dtw is not None else None,
                         logits if dtw is not None else None, dtw, dl, dx, dw, ws, dlogits_add=add,
                         dx_add=dxa)
    l64, a64 = f64(logits), None if add is None else f64(add)
    if dtw is None:
        assert torch.equal(dl, add)
    else:
        want = TO.route_dlogits(l64, ids.numpy(), f64(dtw), renorm, a64)
        near(dl, want, dlogits_bound(l64, ids.numpy(), f64(dtw), renorm, a64) + U * np.abs(want),
             "dlogits")
    # the products from the logits' gradient as stored
    dl64, w64, x64 = f64(dl), f64(w), f64(x)
    rdx, rdw = TO.router_linear_backward(dl64, x64, w64, None if dxa is None else f64(dxa))
    mx, mw = TO.router_linear_backward(np.abs(dl64), np.abs(x64), np.abs(w64),
                                       None if dxa is None else np.abs(f64(dxa)))
    # dx of a bf16 layer takes dlogits in two bf16 parts: 2^-16 of it at most is left out
    part = 2.0 ** -16 if dtype == "bf16" else 0.0
    near(dx, rdx, ((2 * E + 2) * U + part) * mx + HALF[dtype] * 1.01 * np.abs(rdx), "dx")
    near(dw, rdw, (T + 8) * U * mw, "dw_router")
    # accumulation, in-place addends, and the same bits again
    dl2 = add.clone() if add is not None else torch.empty_like(dl)
    dx2 = dxa.clone() if dxa is not None else torch.empty_like(dx)
    dw2 = torch.full((E, H), 0.5, device="cuda")
    M.moe_route_backward(d, T, x, w, idc if dtw is not None else None,
                         logits if dtw is not None else None, dtw, dl2, dx2, dw2, ws,
                         dlogits_add=dl2 if add is not None else None,
                         dx_add=dx2 if dxa is not None else None, accumulate_dw=True)
    assert torch.equal(dl, dl2) and torch.equal(dx, dx2)
    near(dw2, f64(dw) + 0.5, (T + 8) * U * (mw + 0.5), "accumulated dw")
    # each product alone
    dx3, dw3 = torch.empty_like(dx), torch.empty_like(dw)
    if dxa is None:
        M.moe_route_backward(d, T, None, w, None, None, None, dl2, dx3, None, ws, dlogits_add=dl)
        assert torch.equal(dx3, dx) and torch.equal(dl2, dl)
    M.moe_route_backward(d, T, x, None, None, None, None, dl2, None, dw3, ws, dlogits_add=dl)
    assert torch.equal(dw3, dw)


@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_with_masked_experts(renorm):
    """Experts masked by -inf or the type's lowest value, a token whose chosen
    logits are all the lowest, one without slots."""
    T, H, E, k = 5, 64, 20, 3
    g = gen(51)
    logits = torch.randn(T, E, generator=g)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    mask = torch.ones(T, E, dtype=torch.bool).scatter_(1, ids.long(), False)
    low = torch.finfo(torch.float32).min
    logits[0][mask[0]] = -float("inf")
    logits[1][mask[1]] = low
    logits[2] = low
    ids[3] = -1
    dtw = torch.randn(T, k, generator=g)
    d = make_dims(H, E, k, "f32", renorm)
    dl = torch.empty(T, E, device="cuda")
    M.moe_route_backward(d, T, None, None, ids.cuda(), logits.cuda(), dtw.cuda(), dl, None, None, None)
    want = TO.route_dlogits(f64(logits), ids.numpy(), f64(dtw), renorm)
    assert torch.isfinite(dl).all() and not dl[3].any()
    # p off by at most (4 + E + 16) u where |l - m| counts (below it p is 0)
    near(dl, want, 2 * 64 * U * np.abs(f64(dtw)).sum(1, keepdims=True), "dlogits")


def test_route_backward_of_an_empty_batch():
    d = make_dims(128, 8, 2, "bf16")
    dw = torch.full((8, 128), 3.0, device="cuda")
    e = torch.empty(0, device="cuda")
    M.moe_route_backward(d, 0, None, None, None, None, e, e, None, dw, None, accumulate_dw=True)
    assert torch.all(dw == 3.0)
    M.moe_route_backward(d, 0, None, None, None, None, e, e, None, dw, None)
    assert torch.all(dw == 0.0)


@pytest.mark.parametrize("T,H,E,dtype", [(20, 256, 40, "bf16"), (64, 2048, 64, "bf16"), (900, 192, 20, "bf16"),
                                         (41, 320, 9, "f32"), (4200, 1024, 64, "f32")])
@pytest.mark.parametrize("in_place", [False, True])
def test_route_backward_in_a_graph(T, H, E, dtype, in_place):
    """Replayed over new logits and a workspace full of what was there; the
    eager call goes to a stream of its own."""
    g, k = gen(T + E), 3
    x, w = randn(g, T, H, dtype=dtype), randn(g, E, H, dtype=dtype, std=0.05)
    logits, dtw = randn(g, T, E), randn(g, T, k)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    d = make_dims(H, E, k, dtype, True)
    side = torch.cuda.Stream()

    def bufs():
        return dict(dl=torch.zeros(T, E, device="cuda"), dx=torch.zeros(T, H, dtype=TT[dtype], device="cuda"),
                    dw=torch.zeros(E, H, device="cuda"),
                    ws=torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, device="cuda"))

    def run(b, stream=None):
        M.moe_route_backward(d, T, x, w, ids, logits, dtw, b["dl"], b["dx"], b["dw"], b["ws"],
                             dlogits_add=b["dl"] if in_place else None,
                             dx_add=b["dx"] if in_place else None, accumulate_dw=in_place, stream=stream)

    got, want = bufs(), bufs()
    run(bufs())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(got)
    for i in range(4):
        logits.copy_(randn(gen(i), T, E))
        got["ws"].fill_(255)
        torch.cuda.synchronize()
        run(want, side)
        graph.replay()
        torch.cuda.synchronize()
        for n in ("dl", "dx", "dw"):
            assert torch.equal(got[n], want[n]) and torch.isfinite(got[n]).all(), (i, n)


# ------------------------------------------------------------ distillation --
DISTILL = [  # T, V, K, dtype, padded, tau
    (1, 2, 1, "f32", False, 1.0), (3, 1, 1, "bf16", False, 0.5), (4096, 40, 8, "f32", False, 1.0),
    (5, 64, 64, "f32", False, 2.0), (37, 65, 8, "bf16", True, 1.0), (9, 1000, 100, "bf16", False, 0.7),
    (17, 4099, 33, "bf16", False, 1.0), (17, 4099, 33, "f32", True, 3.0), (6, 32000, 64, "bf16", False, 2.0),
    (2, 131072, 1024, "bf16", False, 1.0), (3, 100003, 32, "f32", True, 1.5), (300, 2047, 5, "f32", False, 1.0),
    (19, 4095, 20, "bf16", False, 1.0), (5, 4088, 20, "f32", True, 1.0), (7, 8185, 70, "bf16", False, 1.0),
    (4, 16377, 3, "bf16", False, 1.0), (2, 12000, 3, "f32", True, 2.0), (130, 300, 17, "f32", False, 1.0),
    (33, 500, 16, "bf16", False, 1.0), (257, 20001, 7, "f32", False, 1.0), (256, 40003, 7, "bf16", False, 1.0),
    (260, 66001, 9, "f32", False, 1.0), (64, 511, 65, "bf16", False, 1.0), (9, 512, 64, "f32", True, 1.0),
    (1, 262144, 1, "f32", False, 4.0), (1, 262144, 16, "bf16", False, 1.0), (700, 513, 3, "bf16", False, 1.0),
]


def distill_case(seed, T, V, K, dtype, pad, tau, tail):
    g = gen(seed)
    ld = -(-V // 8) * 8 + 8 if pad else V
    s = randn(g, T, ld, dtype=dtype, std=2.0)
    teacher = s[:, :V].float().cpu() + torch.randn(T, V, generator=g)
    top = torch.topk(teacher, K, dim=1)
    ids, u = top.indices.to(torch.int32), top.values.clone()
    lse = torch.logsumexp(teacher.double() / tau, dim=1).float() if tail else None
    return s, ids, u, lse


def distill_check(s, ids, u, lse, V, tau, w, scale, dtype, loss, ds):
    s64, u64 = f64(s)[:, :V], f64(u)
    l64 = None if lse is None else f64(lse)
    w64 = None if w is None else f64(w)
    idn = ids.cpu().numpy()
    rl, rg = TO.distill(s64, idn, u64, float(np.float32(tau)), l64, w64, float(np.float32(scale)))
    s64 = np.where(w64[:, None] == 0.0, 0.0, s64) if w64 is not None else s64   # masked: c = 0
    c = np.abs(np.float32(scale) * (np.ones(len(s64)) if w64 is None else w64))
    # The tail's sum: each term's exponent is rounded to u of its size (the
    # difference and two products) and exp2 to 1 ulp, weighted by the term
    # itself, and a sum of V terms runs in at least 64 chains.
    z = s64 / tau
    q = np.exp(z - z.max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    spread = np.minimum(np.abs(z - z.max(1, keepdims=True)), 110.0)
    delta = ((q * spread).sum(1) * 4 + spread.min(1) + V / 64 + 32) * U
    near(loss, rl, c * delta * 2 + 2 * U * np.abs(rl), "loss")
    if ds is not None:
        p = np.zeros_like(q)
        for t in range(len(q)):
            ok = [k for k in range(idn.shape[1]) if 0 <= idn[t, k] < V]
            np.add.at(p[t], idn[t, ok], np.abs(rg[t, idn[t, ok]]))
        b = (c / tau)[:, None] * (delta[:, None] + 4 * spread * U) * q
        # a tail class's value carries q_T - p_T, off by delta of q_T
        near(ds[:, :V], rg, 2 * b + (HALF[dtype] + 4 * U + 4 * spread * U + delta[:, None]) * np.abs(rg)
             + 1e-37, "dstudent")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T,V,K,dtype,pad,tau", DISTILL)
def test_distill(T, V, K, dtype, pad, tau, tail):
    say(f"[distill] T={T} V={V} K={K} {dtype} pad={pad} tau={tau} tail={tail}")
    s, ids, u, lse = distill_case(T * 47 + V, T, V, K, dtype, pad, tau, tail)
    w = torch.rand(T, generator=gen(1)) + 0.5
    if T > 2:
        w[1] = 0.0
        s[1, :V] = float("nan")                       # a masked row is not read
    w, ids, u = w.cuda(), ids.cuda(), u.cuda()
    lse = None if lse is None else lse.cuda()
    loss = torch.full((T,), 3.0, device="cuda")
    ds = torch.full_like(s, 3.0)
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    kw = dict(teacher_lse=lse, token_w=w, temperature=tau, scale=0.3)
    M.moe_distill_topk(T, V, K, s, ids, u, loss, ds, ws, **kw)
    distill_check(s, ids, u, lse, V, tau, w, 0.3, dtype, loss, ds)
    assert torch.all(ds[:, V:] == 3.0)                # the padding is left as it was
    l2, l3 = torch.empty_like(loss), torch.empty_like(loss)
    M.moe_distill_topk(T, V, K, s, ids, u, l2, None, ws, **kw)       # the loss alone
    assert torch.equal(l2, loss)
    s2 = s.clone()
    M.moe_distill_topk(T, V, K, s2, ids, u, l3, s2, ws, **kw)        # onto the student
    assert torch.equal(l3, loss) and torch.equal(s2[:, :V], ds[:, :V])


MANY = [  # T, V, K, dtype: more rows than the GPU holds at once, odd row lengths
    (2101, 2401, 20, "bf16"), (4103, 1201, 3, "f32"), (1101, 6001, 70, "bf16"), (521, 12001, 9, "bf16"),
    (1030, 3001, 5, "f32"), (301, 30001, 65, "bf16"), (353, 12001, 30, "f32"), (71, 50001, 17, "bf16"),
    (70, 32001, 17, "f32"), (4200, 301, 16, "bf16"),
]


@pytest.mark.parametrize("T,V,K,dtype", MANY)
def test_distill_many_rows(T, V, K, dtype):
    say(f"[distill] T={T} V={V} K={K} {dtype}")
    s, ids, u, lse = distill_case(T + V, T, V, K, dtype, False, 1.5, True)
    ids, u, lse = ids.cuda(), u.cuda(), lse.cuda()
    loss, ds = torch.full((T,), 3.0, device="cuda"), torch.full_like(s, 3.0)
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, s, ids, u, loss, ds, ws, teacher_lse=lse, temperature=1.5)
    distill_check(s, ids, u, lse, V, 1.5, None, 1.0, dtype, loss, ds)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,ld", [(1, 1, 1), (2, 1, 1), (5, 3, 3), (4, 7, 9), (3, 9, 9)])
def test_distill_more_entries_than_classes(T, V, ld, dtype):
    """Each class named by many entries, rows shorter than a 16-byte load."""
    K = 150
    g = gen(37 * V + T)
    flat = randn(g, (T - 1) * ld + V, dtype=dtype)
    s = flat.as_strided((T, V), (ld, 1)).contiguous()
    ids = torch.randint(-1, V + 1, (T, K), generator=g).to(torch.int32)
    ids[:, :V] = torch.arange(V)
    u = torch.randn(T, K, generator=g)
    # of the mass, nine tenths are the entries'
    lse = torch.stack([torch.logsumexp(u[t][(ids[t] >= 0) & (ids[t] < V)], 0) for t in range(T)]) + 0.1
    for l in (None, lse.cuda()):
        loss, ds = torch.empty(T, device="cuda"), torch.full_like(flat, 3.0)
        M.moe_distill_topk(T, V, K, flat, ids.cuda(), u.cuda(), loss, ds, None, teacher_lse=l, ld=ld)
        got = ds.as_strided((T, V), (ld, 1)).contiguous()
        distill_check(s, ids, u, None if l is None else lse, V, 1.0, None, 1.0, dtype, loss, got)
        for t in range(T - 1):
            assert torch.all(ds[t * ld + V:(t + 1) * ld] == 3.0)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V", [40, 5000])
def test_distill_skipped_doubled_and_masked(V, tail):
    """Skipped and doubled entries, rows without any, -inf and lowest logits
    on both sides."""
    T, K, tau = 10, 6, 1.5
    s, ids, u, lse = distill_case(11 + V, T, V, K, "f32", False, tau, tail)
    ids[0] = -1                                        # no entry
    ids[1, ::2] = V                                    # every other one out of range
    ids[2, 1:] = ids[2, 0]                             # one class, K times
    ids[3, 4] = ids[3, 1]
    u[4, 2:] = -float("inf")                           # teacher masses of zero
    u[5] = -float("inf")                               # a teacher row of them only
    s[6, torch.arange(V) % 3 == 0] = -float("inf")     # masked student classes
    s[6, ids[6].long()] = 1.0
    s[7] = torch.finfo(torch.float32).min              # a row of the lowest value
    s[8, ids[8, 0].long()] = 60.0                      # a teacher class takes all of q
    s[9, (ids[9, 0].item() + 1) % V] += 40.0
    ids, u = ids.cuda(), u.cuda()
    lse = None if lse is None else lse.cuda()
    loss, ds = torch.empty(T, device="cuda"), torch.empty_like(s)
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, s, ids, u, loss, ds, ws, teacher_lse=lse, temperature=tau)
    assert torch.isfinite(loss).all() and torch.isfinite(ds).all()
    distill_check(s, ids, u, lse, V, tau, None, 1.0, "f32", loss, ds)
    if not tail:
        assert loss[0] == 0 and not ds[0].any() and loss[5] == 0 and not ds[5].any()


@pytest.mark.parametrize("V,T", [(40, 5), (400, 5), (5000, 5), (300000 // 2, 2)])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_lowest_teacher_logits_on_masked_classes(V, T, tail):
    """A teacher entry of the type's lowest value has p = 0 (it underflows): a
    student that masks the class with -inf loses nothing by it."""
    K, low = 7, torch.finfo(torch.float32).min
    s, ids, u, lse = distill_case(21 + V, T, V, K, "f32", False, 1.0, tail)
    u[:, 3:] = low
    rows = torch.arange(T)[:, None]
    s[rows.cuda(), ids[:, 3:].long().cuda()] = -float("inf")
    u[1, 1] = -1e4                                     # and one that underflows by itself
    s[1, ids[1, 1].item()] = -float("inf")
    ids, u = ids.cuda(), u.cuda()
    lse = None if lse is None else lse.cuda()
    loss, ds = torch.empty(T, device="cuda"), torch.empty_like(s)
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, s, ids, u, loss, ds, ws, teacher_lse=lse)
    assert torch.isfinite(loss).all() and torch.isfinite(ds).all()
    distill_check(s, ids, u, lse, V, 1.0, None, 1.0, "f32", loss, ds)


def test_distill_infinite_and_nan_rows():
    T, V, K = 4, 300, 3
    s, ids, u, _ = distill_case(5, T, V, K, "f32", False, 1.0, False)
    s[0, ids[0, 1].long()] = -float("inf")             # the teacher wants a masked class
    s[1, 7] = float("nan")
    s[2] = -float("inf")
    loss, ds = torch.empty(T, device="cuda"), torch.empty_like(s)
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, s, ids.cuda(), u.cuda(), loss, ds, ws)
    assert loss[0] == float("inf") and torch.isfinite(ds[0]).all()
    assert torch.isnan(loss[1]) and torch.isnan(ds[1]).all()
    assert torch.isnan(loss[2])
    rl, rg = TO.distill(f64(s)[3:], ids[3:].numpy(), f64(u)[3:], 1.0)
    assert abs(float(loss[3]) - rl[0]) < 1e-5 and np.abs(f64(ds)[3] - rg[0]).max() < 1e-6


def test_distill_rows_past_2_31_elements():
    """A row stride that puts the last rows behind 2^31 elements, onto the student."""
    T, V, K, ld = 3, 5001, 9, (1 << 30) + 5001
    s, ids, u, _ = distill_case(31, T, V, K, "bf16", False, 1.0, False)
    far = torch.empty((T - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    for t in range(T):
        far[t * ld:t * ld + V] = s[t]
    loss = torch.empty(T, device="cuda")
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, far, ids.cuda(), u.cuda(), loss, far, ws, ld=ld)
    ds = torch.stack([far[t * ld:t * ld + V] for t in range(T)])
    distill_check(s, ids, u, None, V, 1.0, None, 1.0, "bf16", loss, ds)


def test_distill_many_rows_in_segments():
    """More rows than one launch of segments takes; the rows repeat, so each
    must equal its first copy."""
    R, T, V, K = 48, 32768 + 48, 66000, 2
    s, ids, u, lse = distill_case(33, R, V, K, "f32", False, 1.0, True)
    n = -(-T // R)
    big = s.repeat(n, 1)[:T].contiguous()
    ids, u, lse = ids.repeat(n, 1)[:T].cuda(), u.repeat(n, 1)[:T].cuda(), lse.repeat(n)[:T].cuda()
    loss = torch.empty(T, device="cuda")
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    M.moe_distill_topk(T, V, K, big, ids, u, loss, big, ws, teacher_lse=lse)
    distill_check(s[:3], ids[:3], u[:3], lse[:3], V, 1.0, None, 1.0, "f32", loss[:3], big[:3])
    at = torch.arange(T, device="cuda") % R
    assert torch.equal(loss, loss[:R][at])
    for t0 in range(0, T, 4096):
        assert torch.equal(big[t0:t0 + 4096], big[:R][at[t0:t0 + 4096]])


@pytest.mark.parametrize("T,V,K,dtype", [(5, 40, 8, "f32"), (300, 500, 12, "bf16"), (7, 5001, 70, "bf16"),
                                         (2100, 2401, 5, "bf16"), (66, 40001, 20, "f32"),
                                         (1100, 12001, 3, "f32")])
def test_distill_in_a_graph(T, V, K, dtype):
    """Onto the student, replayed over new students."""
    s, ids, u, lse = distill_case(T + K, T, V, K, dtype, False, 1.0, True)
    ids, u, lse = ids.cuda(), u.cuda(), lse.cuda()
    loss, eager, l0, side = torch.empty(T, device="cuda"), s.clone(), torch.empty(T, device="cuda"), torch.cuda.Stream()
    ws = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
    run = lambda st, lo, stream=None: M.moe_distill_topk(T, V, K, st, ids, u, lo, st, ws, teacher_lse=lse,
                                                         scale=0.5, stream=stream)
    run(s.clone(), l0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(s, loss)
    for i in range(4):
        new = randn(gen(i), T, V, dtype=dtype)
        s.copy_(new)
        eager.copy_(new)
        torch.cuda.synchronize()
        run(eager, l0, side)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, eager) and torch.equal(loss, l0) and torch.isfinite(s).all(), i


def test_distill_segments_in_a_graph():
    T, V, K = 5, 100003, 12
    s, ids, u, lse = distill_case(35, T, V, K, "f32", False, 1.0, True)
    ids, u, lse = ids.cuda(), u.cuda(), lse.cuda()
    bufs = [(torch.empty(T, device="cuda"), torch.empty_like(s),
             torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    run = lambda b: M.moe_distill_topk(T, V, K, s, ids, u, b[0], b[1], b[2], teacher_lse=lse)
    run(bufs[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(bufs[0])
    for i in range(4):
        s.copy_(randn(gen(90 + i), T, V, std=2.0))
        run(bufs[1])
        torch.cuda.synchronize()
        bufs[0][0].fill_(float("nan"))
        bufs[0][1].fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bufs[0][0], bufs[1][0]) and torch.equal(bufs[0][1], bufs[1][1])


def test_sorted_rows_near_the_element_limit():
    """T * k * hidden just below 2^31: 4 GiB of sorted rows."""
    T, H, k = 65528, 4096, 8
    assert (1 << 31) - (1 << 19) < T * k * H < 1 << 31
    d = make_dims(H, 8, k, "bf16")
    g = gen(77)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    inv = torch.randperm(T * k, generator=g).to(torch.int32).cuda()
    rows = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda")
    M.moe_dispatch(d, T, x, inv, rows)
    iv = inv.view(T, k).long()
    for j in range(k):
        for t0 in range(0, T, 8192):
            assert torch.equal(rows[iv[t0:t0 + 8192, j]], x[t0:t0 + 8192])
    w = torch.rand(T, k, device="cuda")
    w[:, 4:] = 0.0
    out = torch.empty_like(x)
    M.moe_undispatch(d, T, rows, inv, None, out)
    assert torch.equal(out, (x.float() * 8).to(torch.bfloat16))      # eight times itself: exact
    dw = torch.empty(T, k, device="cuda")
    M.moe_undispatch_backward(d, T, x, rows, inv, None, None, dw)
    some = torch.tensor([0, 1, T // 2, T - 1], device="cuda")
    want = (x[some].double() ** 2).sum(1, keepdim=True).expand(-1, k)
    assert torch.allclose(dw[some].double(), want, rtol=(H / 8 + 17) * U, atol=0)
    M.moe_undispatch_backward(d, T, x, None, inv, w, rows, None)
    some_rows = (w[some][..., None] * x[some].float()[:, None]).to(torch.bfloat16)
    assert torch.equal(rows[iv[some]], some_rows)


def test_route_backward_of_many_tokens():
    """A long batch of a narrow layer: many token ranges and long ones."""
    T, H, E, k = 300007, 64, 5, 2
    g = gen(41)
    d = make_dims(H, E, k, "bf16", True)
    x, w = randn(g, T, H, dtype="bf16"), randn(g, E, H, dtype="bf16")
    add = randn(g, T, E)
    dl, dx, dw = torch.empty_like(add), torch.empty_like(x), torch.empty(E, H, device="cuda")
    ws = torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, device="cuda")
    M.moe_route_backward(d, T, x, w, None, None, None, dl, dx, dw, ws, dlogits_add=add)
    assert torch.equal(dl, add)
    rdx, rdw = TO.router_linear_backward(f64(add), f64(x), f64(w))
    mx, mw = TO.router_linear_backward(np.abs(f64(add)), np.abs(f64(x)), np.abs(f64(w)))
    near(dx, rdx, ((2 * E + 2) * U + 2.0 ** -16) * mx + HALF["bf16"] * 1.01 * np.abs(rdx), "dx")
    # a wave sums at most T / 256 tokens before the ranges meet
    near(dw, rdw, (T / 256 + 300) * U * mw, "dw_router")


# ------------------------------------------------------ the operators as one --
def train_step(layer, T, x, w, wdev, bufs):
    """Router and prefetch router of a layer with the caller's experts (one
    matrix each, rows sorted by expert): forward, then every gradient."""
    cfg, d = layer.cfg, M.Dims(**dims_dict(layer.cfg))
    E, k, H = cfg.n_experts, cfg.top_k, cfg.hidden
    b = bufs
    M.moe_route(d, T, x, wdev["w_router"], None, 0, "standard", b["ids"], b["topk_w"], b["exact"],
                b["flags"], b["logits"])
    M.moe_permute(T, k, E, b["ids"], b["exact"], b["offsets"], b["perm"], b["inv"], b["pws"])
    M.moe_dispatch(d, T, x, b["inv"], b["xs"])
    torch.mul(b["xs"], w, out=b["ys"])                 # the experts: a diagonal map
    M.moe_undispatch(d, T, b["ys"], b["inv"], b["topk_w"], b["out"], add=x)
    M.moe_undispatch_backward(d, T, b["dout"], b["ys"], b["inv"], b["topk_w"], b["dys"], b["dtw"])
    torch.mul(b["dys"], w, out=b["dxs"])
    M.moe_undispatch(d, T, b["dxs"], b["inv"], None, b["dx"], add=b["dout"])
    M.moe_route_backward(d, T, x, wdev["w_router"], b["ids"], b["logits"], b["dtw"], b["dl"],
                         b["dx"], b["dw"], b["ws"], dx_add=b["dx"])
    # the prefetch router toward the router's choices
    M.moe_route(d, T, x, wdev["w_prefetch"], None, 0, "standard", b["pids"], b["ptw"], b["exact"],
                b["flags"], b["plogits"])
    b["tl"].copy_(torch.gather(b["logits"], 1, b["ids"].long()))
    M.moe_distill_topk(T, E, k, b["plogits"], b["ids"], b["tl"], b["loss"], b["dpl"], b["dws"],
                       scale=1.0 / T)
    M.moe_route_backward(d, T, x, None, None, None, None, b["dpl"], None, b["dwp"], b["ws"],
                         dlogits_add=b["dpl"])


def train_bufs(cfg, T, seed):
    d = M.Dims(**dims_dict(cfg))
    H, E, k = cfg.hidden, cfg.n_experts, cfg.top_k
    dt, P = TT[cfg.dtype], T * k
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
    f = lambda *s: torch.empty(*s, device="cuda")
    x = lambda *s: torch.zeros(*s, dtype=dt, device="cuda")
    b = dict(ids=i32(T, k), pids=i32(T, k), topk_w=f(T, k), ptw=f(T, k), flags=i32(T), logits=f(T, E),
             plogits=f(T, E), exact=torch.empty(T * k, dtype=torch.uint8, device="cuda"),
             offsets=i32(E + 1), perm=i32(P), inv=i32(P), xs=x(P, H), ys=x(P, H), dys=x(P, H),
             dxs=x(P, H), out=x(T, H), dx=x(T, H), dtw=f(T, k), dl=f(T, E), dw=f(E, H), tl=f(T, k),
             loss=f(T), dpl=f(T, E), dwp=f(E, H))
    b["dout"] = randn(gen(seed), T, H, dtype=cfg.dtype)
    size = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
    b["pws"] = size(M.moe_workspace_size(d, T, "standard"))
    b["ws"], b["dws"] = size(M.moe_route_backward_size(d, T)), size(M.moe_distill_topk_size(T, E))
    return b


def small_layer(dtype, renorm):
    cfg = dataclasses.replace(W.CONFIGS["granite_prefill"], name=f"train_{dtype}_{renorm}", hidden=192,
                              n_experts=12, top_k=3, inter=64, dtype=dtype, renormalize=renorm,
                              token_counts=(45,), seed=301)
    return W.Layer(cfg)


@pytest.mark.parametrize("dtype,renorm", [("f32", True), ("f32", False), ("bf16", True)])
def test_train_step_gradients(dtype, renorm):
    """All operators in a row: the gradients of sum(out * dout) and of the
    distillation loss, against the fp64 chain and against differences."""
    layer = small_layer(dtype, renorm)
    cfg, T = layer.cfg, 45
    E, k, H = cfg.n_experts, cfg.top_k, cfg.hidden
    wdev = upload(layer, "cuda", names=[])
    x = tensor(layer.x(T), dtype, "cuda")
    w = randn(gen(9), H, dtype=dtype)
    b = train_bufs(cfg, T, 12)
    train_step(layer, T, x, w, wdev, b)
    torch.cuda.synchronize()
    x64, wr, wp, w64, do = (f64(v) for v in (x, wdev["w_router"], wdev["w_prefetch"], w, b["dout"]))
    ids, inv = b["ids"].cpu().numpy(), b["inv"].cpu().numpy()

    def forward(xv, wrv):
        tw = TO.route_weights(xv @ wrv.T, ids, renorm)
        return float(((xv + tw.sum(1, keepdims=True) * xv * w64) * do).sum())

    logits = x64 @ wr.T
    tw = TO.route_weights(logits, ids, renorm)
    dtw = np.stack([((x64 * w64) * do).sum(1)] * k, 1)
    dl = TO.route_dlogits(logits, ids, dtw, renorm)
    dx, dw = TO.router_linear_backward(dl, x64, wr, do + tw.sum(1, keepdims=True) * w64 * do)
    if dtype == "f32":
        # differences of the fp64 forward along random directions
        rng = np.random.default_rng(3)
        for _ in range(3):
            vx, vw, h = rng.normal(size=x64.shape), rng.normal(size=wr.shape), 1e-5
            num = (forward(x64 + h * vx, wr + h * vw) - forward(x64 - h * vx, wr - h * vw)) / (2 * h)
            ana = (dx * vx).sum() + (dw * vw).sum()
            assert abs(num - ana) < 1e-6 * (1 + abs(ana))
    rel = lambda a, r: np.linalg.norm(f64(a) - r) / max(np.linalg.norm(r), 1e-30)
    # fp32: sums of H and T terms, each 2^-24; bf16: rows rounded four times on the way (2^-8
    # each), and the weights' gradients cancel where renormalised, so they are held in norm
    tol = 2e-5 if dtype == "f32" else 5 * 2.0 ** -8
    assert rel(b["dx"], dx) < tol
    assert np.linalg.norm(f64(b["dl"]) - dl) <= tol * np.linalg.norm(dtw)
    assert np.linalg.norm(f64(b["dw"]) - dw) <= tol * np.linalg.norm(dtw) * np.linalg.norm(x64, 2)
    lp = f64(b["plogits"])
    loss, dlp = TO.distill(lp, ids, f64(b["tl"]), 1.0, None, None, 1.0 / T)
    assert np.abs(f64(b["loss"]) - loss).max() < 1e-6 and rel(b["dpl"], dlp) < 1e-5
    _, dwp = TO.router_linear_backward(dlp, x64, wp)
    assert rel(b["dwp"], dwp) < 1e-5


def test_train_step_in_a_graph():
    """Captured once and replayed over new inputs, with eager work and waits
    between; every replay equals the eager step bit for bit."""
    layer = small_layer("bf16", True)
    cfg, T = layer.cfg, 45
    wdev = upload(layer, "cuda", names=[])
    x = tensor(layer.x(T), "bf16", "cuda").clone()
    w = randn(gen(9), cfg.hidden, dtype="bf16")
    b, eager = train_bufs(cfg, T, 12), train_bufs(cfg, T, 12)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        train_step(layer, T, x, w, wdev, b)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        train_step(layer, T, x, w, wdev, b)
    for i in range(4):
        x.copy_(randn(gen(50 + i), T, cfg.hidden, dtype="bf16"))
        train_step(layer, T, x, w, wdev, eager)
        torch.cuda.synchronize()
        for v in b.values():
            if v.dtype == torch.float32:
                v.fill_(float("nan"))
        b["dout"].copy_(eager["dout"])
        graph.replay()
        torch.cuda.synchronize()
        for n in ("out", "dx", "dl", "dw", "dtw", "loss", "dpl", "dwp", "xs", "dys"):
            assert torch.equal(b[n], eager[n]), (i, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspaces_of_the_largest_batch(dtype):
    """Made once for the most tokens, they serve every smaller batch."""
    most, H, E, k, V = 2112, 256, 33, 3, 33001 if dtype == "bf16" else 17001
    g, d = gen(83), make_dims(H, E, k, dtype, True)
    x, w = randn(g, most, H, dtype=dtype), randn(g, E, H, dtype=dtype, std=0.05)
    add = randn(g, most, E)
    s, u = randn(g, most, V, dtype=dtype), randn(g, most, 4)
    ids = torch.randint(0, V, (most, 4), generator=g).to(torch.int32).cuda()
    rws = torch.empty(M.moe_route_backward_size(d, most), dtype=torch.uint8, device="cuda")
    dws = torch.empty(M.moe_distill_topk_size(most, V), dtype=torch.uint8, device="cuda")
    for T in (1, 63, 64, 65, 257, 700, 2080, most):
        say(f"[workspaces] {dtype} T={T}")
        got = [torch.zeros(T, E, device="cuda"), torch.zeros_like(x[:T]), torch.zeros(E, H, device="cuda")]
        want = [torch.zeros_like(t) for t in got]
        own = torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, device="cuda")
        for out, ws in ((got, rws), (want, own)):
            M.moe_route_backward(d, T, x, w, None, None, None, *out, ws, dlogits_add=add)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        ref, tol = f64(add[:T]).T @ f64(x[:T]), (T + 8) * U * (np.abs(f64(add[:T])).T @ np.abs(f64(x[:T])))
        near(got[2], ref, tol, "dw_router")
        got = [torch.zeros(T, device="cuda"), torch.zeros_like(s[:T])]
        want = [torch.zeros_like(t) for t in got]
        own = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device="cuda")
        for out, ws in ((got, dws), (want, own)):
            M.moe_distill_topk(T, V, 4, s, ids, u, *out, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.isfinite(got[0]).all()


def test_two_streams_at_once():
    """Two steps with buffers of their own on two streams."""
    layer = small_layer("bf16", False)
    cfg, T = layer.cfg, 45
    wdev = upload(layer, "cuda", names=[])
    w = randn(gen(9), cfg.hidden, dtype="bf16")
    xs = [randn(gen(70 + i), T, cfg.hidden, dtype="bf16") for i in range(2)]
    want = [train_bufs(cfg, T, 12) for _ in range(2)]
    got = [train_bufs(cfg, T, 12) for _ in range(2)]
    for x, b in zip(xs, want):
        train_step(layer, T, x, w, wdev, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for s, x, b in zip(streams, xs, got):
            with torch.cuda.stream(s):
                train_step(layer, T, x, w, wdev, b)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for n in ("out", "dx", "dl", "dw", "loss", "dwp"):
            assert torch.equal(a[n], b[n]), n


def test_binding_checks_sizes_and_types():
    d = make_dims(64, 4, 2, "bf16")
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.zeros(8, dtype=torch.int32, device="cuda")
    rows = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        M.moe_dispatch(d, 4, x, inv[:7], rows)
    with pytest.raises(ValueError):
        M.moe_dispatch(d, 4, x, inv, rows[:7])
    with pytest.raises(TypeError):
        M.moe_dispatch(d, 4, x.float(), inv, rows)
    with pytest.raises(TypeError):
        M.moe_dispatch(d, 4, x, inv.long(), rows)
    with pytest.raises(ValueError):
        M.moe_dispatch(d, 4, x, inv, rows.t())
    with pytest.raises(M.MoEError):
        M.moe_undispatch(make_dims(64, 4, 2, "f32"), 4, rows, inv, None, x.float())
    s = torch.zeros(3, 10, device="cuda")
    with pytest.raises(ValueError):
        M.moe_distill_topk(3, 10, 2, s, torch.zeros(3, 1, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, 2, device="cuda"), torch.zeros(3, device="cuda"))
