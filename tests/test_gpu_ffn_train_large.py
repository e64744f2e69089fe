"""The experts' training operators at sizes that take the large block shapes,
against their formulas in 64 bits on the GPU; the tolerances are those of
test_gpu_ffn_train.py, element by element."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from test_gpu_ffn_train import HALF, MARK, Case, say, sum_tol  # noqa: E402

A = torch.abs


def near(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= 1.01 * tol)
    assert not bool(bad.any()), (what, int(bad.sum()), [int(v[0]) for v in bad.nonzero(as_tuple=True)])


def kept_values(c, kept, scale):
    v = kept.double()
    if scale is not None:
        v = v * scale.double().repeat_interleave(64, dim=-1)[..., :c.I]
    return v[:, 0], v[:, 1]


def segments(c):
    off, token = c.offsets.tolist(), torch.div(c.perm.long(), c.k, rounding_mode="floor")
    for e in range(c.E):
        if off[e + 1] > off[e]:
            r = slice(off[e], off[e + 1])
            yield e, r, c.x[token[r]].double()


def check_forward(c, y, kept, scale):
    h = HALF[c.dtype]
    gg, gu = kept_values(c, kept, scale)
    for e, r, x in segments(c):
        wg, wu, wd = (c.w[n][e].double() for n in ("w_gate", "w_up", "w_down"))
        g, u = x @ wg.T, x @ wu.T
        eg, eu = sum_tol(c.H, A(x) @ A(wg).T), sum_tol(c.H, A(x) @ A(wu).T)
        a = A(g * torch.sigmoid(g) * u)
        ea = 1.1 * eg * (A(u) + eu) + A(g) * eu + a * ((A(g) + 5) * 2.0 ** -22 + h)
        want = (g * torch.sigmoid(g) * u) @ wd.T
        near(y[r], want, ea @ A(wd).T + sum_tol(c.I, (a + ea) @ A(wd).T) + h * A(want), f"y of expert {e}")
        for got, v, ev, name in ((gg[r], g, eg, "g"), (gu[r], u, eu, "u")):
            if scale is None:
                near(got, v, ev + h * (A(v) + ev), f"{name} of expert {e}")
                continue
            for b in range(0, c.I, 64):          # half a step, the scale's error over 127 of them
                s = slice(b, b + 64)
                top, et = A(v[:, s]).amax(1, keepdim=True), ev[:, s].amax(1, keepdim=True)
                near(got[:, s], v[:, s], 0.5 * (top + et) / 127 + (top + et) * 2.0 ** -22 + ev[:, s] + et,
                     f"{name} of expert {e} in 8 bits")
    assert bool((y[c.n:] == MARK).all()) and bool((kept[c.n:] == MARK).all())


def check_backward(c, got):
    h, (gall, uall) = HALF[c.dtype], kept_values(c, c.kept, c.scale)
    for e, r, x in segments(c):
        wg, wu, wd = (c.w[n][e].double() for n in ("w_gate", "w_up", "w_down"))
        g, u, dy = gall[r], uall[r], c.dy[r].double()
        G, s, da = A(g), torch.sigmoid(g), dy @ wd
        eda = sum_tol(c.H, A(dy) @ A(wd))
        a, dg, du = g * s * u, da * u * s * (1 + g * (1 - s)), da * g * s
        ea = A(a) * ((G + 5) * 2.0 ** -22 + h)
        edu = (eda + A(da) * (G + 5) * 2.0 ** -22) * A(g * s)
        edu = edu + h * (A(du) + edu)
        ed = s * (1 + 2 * G) * (G + 4) * 2.0 ** -22 + 4 * s * (1 + 2 * G) * 2.0 ** -23
        edg = (A(da) * ed + eda * 1.1) * A(u)
        edg = edg + h * (A(dg) + edg)
        fg, fu = A(dg) + edg, A(du) + edu
        want = dg @ wg + du @ wu
        near(got[0][r], want, edg @ A(wg) + edu @ A(wu) + sum_tol(2 * c.I, fg @ A(wg) + fu @ A(wu)) + h * A(want),
             f"dx of expert {e}")
        n = len(x)
        for i, (d, ed_, f_, o) in enumerate(((dg, edg, fg, x), (du, edu, fu, x))):
            want = d.T @ o
            near(got[1 + i][e], want, ed_.T @ A(o) + sum_tol(n, f_.T @ A(o)) + h * A(want), f"dw {i} of expert {e}")
        want = dy.T @ a
        near(got[3][e], want, A(dy).T @ ea + sum_tol(n, A(dy).T @ (A(a) + ea)) + h * A(want),
             f"dw_down of expert {e}")
    assert bool((got[0][c.n:] == MARK).all())


LARGE = [  # T, H, I, E, k, dtype, keep, missing
    (2000, 1536, 1280, 4, 2, "bf16", "rows", 0.05),      # 256 x 128 everywhere
    (2100, 1600, 1296, 4, 2, "bf16", "int8", 0.0),       # the same with ragged ends
    (8192, 64, 2560, 1, 1, "bf16", "rows", 0.0),         # a single pair of stages before the kept rows
    (8192, 64, 2576, 1, 1, "bf16", "int8", 0.1),
    (600, 2048, 2064, 1, 1, "bf16", "rows", 0.0),        # dx by 256 x 256
    (777, 2112, 2000, 2, 2, "bf16", "int8", 0.1),
    (8100, 4096, 80, 1, 1, "f32", "rows", 0.0),          # fp32, the large ends of its shapes
    (8100, 64, 4096, 1, 1, "f32", "int8", 0.0),    
    (300, 512, 528, 64, 4, "f32", "rows", 0.2),  
]


@pytest.mark.parametrize("T,H,I,E,k,dtype,keep,miss", LARGE)
def test_large_forward(T, H, I, E, k, dtype, keep, miss):
    say(f"[ffn_train large] T={T} H={H} I={I} E={E} k={k} {dtype} {keep} miss={miss}")
    c = Case(T, H, I, E, k, dtype, keep, miss, pack=False)
    check_forward(c, *c.train())


@pytest.mark.parametrize("T,H,I,E,k,dtype,keep,miss", LARGE)
def test_large_backward(T, H, I, E, k, dtype, keep, miss):
    say(f"[ffn_backward large] T={T} H={H} I={I} E={E} k={k} {dtype} {keep} miss={miss}")
    c = Case(T, H, I, E, k, dtype, keep, miss, pack=False)
    first = c.backward()
    check_backward(c, first)
    assert all(torch.equal(a, b) for a, b in zip(first, c.backward()))       # in any order of its blocks


@pytest.mark.parametrize("dtype,dw", [("bf16", "same"), ("bf16", "f32")])
def test_large_gradients_added(dtype, dw):
    c = Case(2000, 1024, 1280, 4, 2, dtype, "rows", 0.0, pack=False)
    once, twice = c.grads(dw), c.grads(dw)
    c.backward(once)
    for v in twice[1:]:
        v.zero_()
    c.backward(twice, accumulate_dw=True)
    assert all(torch.equal(a, b) for a, b in zip(once, twice))
    c.backward(twice, accumulate_dw=True)
    # v + v is exact in either type
    assert all(torch.equal(2 * a, b) for a, b in zip(once[1:], twice[1:]))


# Long fp32 sums are put aside every 512 terms.  With partial sums that wander
# (independent terms of mean zero) n sequential adds, each off by at most 2^-24 of
# the partial sum, give an error of 2^-24 sqrt(n / 2) of the result in the root of
# the mean square; by parts of 512 it is sqrt(512 / 2 + n / 1024).  What stands
# before the sum (64 terms, the activation) adds less than 8 in these units.
def long_bound(n):
    return 2.0 ** -24 * ((256 + n / 1024) ** 0.5 + 8)


@pytest.mark.parametrize("T,H,I", [(16, 64, 32768), (100, 64, 16400)])
def test_long_sums_over_channels(T, H, I):
    c = Case(T, H, I, 1, 1, "f32", "rows", 0.0, pack=False)
    y, kept, _ = c.train()
    e, r, x = next(segments(c))
    wg, wu, wd = (c.w[n][e].double() for n in ("w_gate", "w_up", "w_down"))
    g, u = x @ wg.T, x @ wu.T
    want = (torch.nn.functional.silu(g) * u) @ wd.T
    assert float((y[r].double() - want).norm() / want.norm()) <= long_bound(I)
    g, u = (v[r] for v in kept_values(c, c.kept, c.scale))
    da, s = c.dy[r].double() @ wd, torch.sigmoid(g)
    want = (da * u * s * (1 + g * (1 - s))) @ wg + (da * g * s) @ wu
    got = c.backward()[0][r].double()
    assert float((got - want).norm() / want.norm()) <= long_bound(2 * I)


def test_long_sums_over_rows():
    c = Case(20000, 64, 80, 1, 1, "f32", "rows", 0.0, pack=False)
    got = c.backward()
    e, r, x = next(segments(c))
    g, u = (v[r] for v in kept_values(c, c.kept, c.scale))
    dy, s = c.dy[r].double(), torch.sigmoid(g)
    da = dy @ c.w["w_down"][e].double()
    for v, want in zip(got[1:], ((da * u * s * (1 + g * (1 - s))).T @ x, (da * g * s).T @ x, dy.T @ (g * s * u))):
        assert float((v[e].double() - want).norm() / want.norm()) <= long_bound(c.n)
