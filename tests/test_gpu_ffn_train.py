"""The experts' training operators on the GPU against their fp64 forms
(oracle.ffn_train_oracle).

Tolerances are rounding bounds, element by element, to first order with 1% for
the rest.  u = 2^-24 is half a step of fp32; h half a step of the layer's type.
  - A sum of n products formed in fp32 in any order is off by at most
    2 (n + 1) u times the sum of their magnitudes (2: the matrix cores' adds are
    taken to be off by a whole step rather than half of one).
  - sigmoid(g) from the hardware exponential and reciprocal: the exponent's
    product with log2 e is off by |g| 2^-23 and each of exp2, the sum and the
    reciprocal by 2^-22 at most, so it is off by (|g| + 4) 2^-22 of itself.
  - A value rounded to the layer's type between two products adds h of itself,
    and so does each output.
"""
import dataclasses

import numpy as np
import pytest
import torch

from oracle import ffn_train_oracle as FO

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import sparse_moe_layer_route_amd as M  # noqa: E402
from gpu_harness import say  # noqa: E402

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TT = {"f32": torch.float32, "bf16": torch.bfloat16}
MARK = 7.0                                     # what rows that nothing writes hold


def f64(t):
    return t.detach().cpu().double().numpy()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype="f32", std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(TT[dtype]).cuda()


def near(got, want, tol, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= tol * 1.01)
    if bad.any():
        i = tuple(int(v[0]) for v in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} values off, first at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, allowed {np.broadcast_to(tol, got.shape)[i]!r}")


class Case:
    """Inputs of one batch: pairs sorted by expert, weights, gradients."""

    def __init__(self, T, H, I, E, k, dtype, keep, miss=0.0, seed=0, counts=None, pack=True):
        g = gen(1000 * T + H + I + seed)
        self.T, self.H, self.I, self.E, self.k, self.dtype, self.keep = T, H, I, E, k, dtype, keep
        self.P = P = T * k
        if counts is not None:                 # so many rows for each expert
            key = torch.repeat_interleave(torch.arange(len(counts)), torch.tensor(counts))
            key = torch.cat((key, torch.full((P - len(key),), E)))[torch.randperm(P, generator=g)]
        else:
            ids = torch.topk(torch.randn(T, E, generator=g), k, dim=1).indices
            key = torch.where(torch.rand(T, k, generator=g) < miss, E, ids).flatten()
        self.perm = torch.argsort(key, stable=True).to(torch.int32).cuda()
        n = torch.bincount(key, minlength=E + 1)[:E]
        self.offsets = torch.cat((torch.zeros(1, dtype=torch.int64), n.cumsum(0))).to(torch.int32).cuda()
        self.n = int(self.offsets[-1])
        self.x = randn(g, T, H, dtype=dtype)
        self.w = {"w_gate": randn(g, E, I, H, dtype=dtype, std=H ** -0.5),
                  "w_up": randn(g, E, I, H, dtype=dtype, std=H ** -0.5),
                  "w_down": randn(g, E, H, I, dtype=dtype, std=I ** -0.5)}
        self.dy = randn(g, P, H, dtype=dtype, std=0.1)
        self.dy[self.n:] = float("nan")        # rows behind the last are not read
        self.dims = M.Dims(hidden=H, n_experts=E, top_k=k, inter=I, dtype=dtype)
        self.ws = torch.empty(M.moe_expert_ffn_train_size(self.dims, T), dtype=torch.uint8, device="cuda")
        self.ws.fill_(255)                     # NaN in either type
        # kept rows of the backward pass alone
        kept = randn(g, P, 2, I, dtype=dtype)
        self.blocks = -(-I // 64)
        self.scale = None
        if keep == "int8" and not pack:        # by the library, which test_rows8 checks
            self.kept = torch.empty(P, 2, I, dtype=torch.int8, device="cuda")
            self.scale = torch.empty(P, 2, self.blocks, device="cuda")
            M.moe_rows_pack8(2 * P, I, kept.view(2 * P, I), self.kept.view(2 * P, I), self.scale.view(2 * P, -1))
            self.scale[self.n:] = float("nan")
        elif keep == "int8":
            c, s = FO.pack8(f64(kept).reshape(2 * P, I))
            self.kept = torch.from_numpy(c.reshape(P, 2, I)).to(torch.int8).cuda()
            self.scale = torch.from_numpy(s.reshape(P, 2, self.blocks)).float().cuda()
            self.scale[self.n:] = float("nan")
        else:
            self.kept = kept
            self.kept[self.n:] = float("nan")

    def arrays(self):
        return (f64(self.x), *(f64(self.w[n]) for n in ("w_gate", "w_up", "w_down")),
                self.offsets.cpu().numpy(), self.perm.cpu().numpy(), self.k)

    def values(self, kept, scale):
        """g and u [P][I] that are kept."""
        v = f64(kept).reshape(2 * self.P, self.I)
        if scale is not None:
            v = FO.unpack8(v, f64(scale).reshape(2 * self.P, self.blocks))
        v = v.reshape(self.P, 2, self.I)
        return v[:, 0], v[:, 1]

    def outputs(self, keep=None):
        keep, dev = keep or self.keep, dict(device="cuda")
        y = torch.full((self.P, self.H), MARK, dtype=TT[self.dtype], **dev)
        if keep == "int8":
            return (y, torch.full((self.P, 2, self.I), int(MARK), dtype=torch.int8, **dev),
                    torch.full((self.P, 2, self.blocks), MARK, **dev))
        return y, torch.full((self.P, 2, self.I), MARK, dtype=TT[self.dtype], **dev), None

    def train(self, out=None, **kw):
        y, kept, scale = out or self.outputs()
        M.moe_expert_ffn_train(self.dims, self.T, self.x, self.w, self.offsets, self.perm, y, kept, self.ws,
                               kept_scale=scale, **kw)
        return y, kept, scale

    def grads(self, dw="same"):
        t = TT[self.dtype] if dw == "same" else torch.float32
        return [torch.full((self.P, self.H), MARK, dtype=TT[self.dtype], device="cuda")] + \
               [torch.full(self.w[n].shape, MARK, dtype=t, device="cuda") for n in ("w_gate", "w_up", "w_down")]

    def backward(self, out=None, **kw):
        out = out or self.grads()
        M.moe_expert_ffn_backward(self.dims, self.T, self.x, self.w, self.offsets, self.perm, self.kept,
                                  self.dy, *out, self.ws, kept_scale=self.scale, **kw)
        return out


def sum_tol(n, mag):
    return 2 * (n + 1) * U * mag


def check_forward(c, y, kept, scale):
    x, wg, wu, wd, off, perm, k = c.arrays()
    h = HALF[c.dtype]
    want, g, u = FO.forward(x, wg, wu, wd, off, perm, k, c.P)
    eg, eu, ey = np.zeros_like(g), np.zeros_like(u), np.zeros_like(want)
    for e, r, t in FO.segments(off, perm, k):
        eg[r] = sum_tol(c.H, np.abs(x[t]) @ np.abs(wg[e]).T)
        eu[r] = sum_tol(c.H, np.abs(x[t]) @ np.abs(wu[e]).T)
        a = np.abs(g[r] * FO.sigmoid(g[r]) * u[r])
        # |SiLU'| <= 1.1
        ea = 1.1 * eg[r] * (np.abs(u[r]) + eu[r]) + np.abs(g[r]) * eu[r]
        ea += a * ((np.abs(g[r]) + 5) * 2.0 ** -22 + h)
        ey[r] = ea @ np.abs(wd[e]).T + sum_tol(c.I, (a + ea) @ np.abs(wd[e]).T)
    n = c.n
    near(f64(y)[:n], want[:n], (ey + h * np.abs(want))[:n], "y")
    assert bool((y[n:] == MARK).all()) and bool((kept[n:] == MARK).all())
    gg, gu = c.values(kept, scale)
    if scale is None:
        near(gg[:n], g[:n], (eg + h * (np.abs(g) + eg))[:n], "g")
        near(gu[:n], u[:n], (eu + h * (np.abs(u) + eu))[:n], "u")
        return
    assert bool((scale[n:] == MARK).all())
    assert not bool((kept[:n] == -128).any())
    for got, v, e, j in ((gg, g, eg, 0), (gu, u, eu, 1)):
        for b in range(c.blocks):
            s = slice(64 * b, min(c.I, 64 * b + 64))
            top, etop = np.abs(v[:n, s]).max(1), e[:n, s].max(1)
            near(f64(scale)[:n, j, b], top / 127, (etop + 2 * U * top) / 127, "scale")
            # the nearest step, half a step off; 127 steps off by the scale's error
            half = (0.5 * (top + etop) / 127 + 127 * (top + etop) / 127 * 4 * U)[:, None]
            near(got[:n, s], v[:n, s], half + e[:n, s] + etop[:, None], "8 bits")


def check_backward(c, got, g, u, dy=None, before=None, dw_half=None):
    x, wg, wu, wd, off, perm, k = c.arrays()
    h = HALF[c.dtype]
    dw_half = h if dw_half is None else dw_half
    n = c.n
    dy = np.where(np.arange(c.P)[:, None] < n, f64(c.dy), 0.0) if dy is None else dy
    want = FO.backward(x, wg, wu, wd, off, perm, k, g, u, dy)
    tol = [np.zeros_like(w) for w in want]
    for e, r, t in FO.segments(off, perm, k):
        da, G, A = dy[r] @ wd[e], np.abs(g[r]), np.abs
        eda = sum_tol(c.H, A(dy[r]) @ A(wd[e]))
        s = FO.sigmoid(g[r])
        a, dg, du = FO.gated_grad(g[r], u[r], da)
        ea = A(a) * ((G + 5) * 2.0 ** -22 + h)
        edu = (eda + A(da) * (G + 5) * 2.0 ** -22) * A(g[r] * s)
        edu += h * (A(du) + edu)
        # s (1 + g (1 - s)): s is off by (|g| + 4) 2^-22 of itself wherever it stands, and the
        # steps in between, none larger than s (1 + 2 |g|), by 2^-23 of that each
        ed = s * (1 + 2 * G) * (G + 4) * 2.0 ** -22 + 4 * s * (1 + 2 * G) * 2.0 ** -23
        edg = (A(da) * ed + eda * 1.1) * A(u[r])
        edg += h * (A(dg) + edg)
        tol[0][r] = edg @ A(wg[e]) + edu @ A(wu[e]) + sum_tol(
            2 * c.I, (A(dg) + edg) @ A(wg[e]) + (A(du) + edu) @ A(wu[e]))
        rows = len(t)
        tol[1][e] = edg.T @ A(x[t]) + sum_tol(rows, (A(dg) + edg).T @ A(x[t]))
        tol[2][e] = edu.T @ A(x[t]) + sum_tol(rows, (A(du) + edu).T @ A(x[t]))
        tol[3][e] = A(dy[r]).T @ ea + sum_tol(rows, A(dy[r]).T @ (A(a) + ea))
    for i, (name, v) in enumerate(zip(("dx", "dw_gate", "dw_up", "dw_down"), got)):
        if v is None:
            continue
        if i == 0:
            near(f64(v)[:n], want[0][:n], (tol[0] + h * np.abs(want[0]))[:n], name)
            assert bool((v[n:] == MARK).all())
        else:
            w = want[i] if before is None else want[i] + before[i]
            extra = 0 if before is None else U * np.abs(w)
            near(v, w, tol[i] + extra + dw_half * np.abs(w), name)


CASES = [  # T, H, I, E, k, dtype, keep, missing
    (1, 64, 16, 1, 1, "bf16", "rows", 0.0), (1, 64, 16, 2, 2, "f32", "int8", 0.0),
    (1, 256, 80, 8, 8, "bf16", "int8", 0.0), (3, 128, 48, 64, 6, "bf16", "rows", 0.3),
    (8, 192, 112, 5, 2, "f32", "rows", 0.0), (17, 320, 144, 7, 3, "bf16", "int8", 0.5),
    (64, 512, 256, 64, 6, "bf16", "rows", 0.0), (65, 64, 1040, 3, 2, "bf16", "int8", 0.1),
    (130, 576, 64, 16, 8, "f32", "int8", 0.9), (200, 256, 512, 8, 2, "f32", "rows", 0.2),
    (333, 384, 208, 4, 2, "bf16", "rows", 0.1), (700, 256, 320, 2, 1, "bf16", "int8", 0.0),
    (1025, 128, 192, 1, 1, "bf16", "rows", 0.0), (513, 320, 272, 3, 2, "f32", "rows", 0.0),
    (40, 1536, 512, 40, 8, "bf16", "int8", 0.0), (900, 512, 128, 5, 3, "bf16", "int8", 0.0),
]


@pytest.mark.parametrize("T,H,I,E,k,dtype,keep,miss", CASES)
def test_forward(T, H, I, E, k, dtype, keep, miss):
    say(f"[ffn_train] T={T} H={H} I={I} E={E} k={k} {dtype} {keep} miss={miss}")
    c = Case(T, H, I, E, k, dtype, keep, miss)
    check_forward(c, *c.train())


@pytest.mark.parametrize("T,H,I,E,k,dtype,keep,miss", CASES)
def test_backward(T, H, I, E, k, dtype, keep, miss):
    say(f"[ffn_backward] T={T} H={H} I={I} E={E} k={k} {dtype} {keep} miss={miss}")
    c = Case(T, H, I, E, k, dtype, keep, miss)
    check_backward(c, c.backward(), *clean(c))


def clean(c):
    """Kept values with zeros behind the last row (NaN there, never read)."""
    return [np.where(np.arange(c.P)[:, None] < c.n, v, 0.0) for v in c.values(c.kept, c.scale)]


# rows of single experts: none, one, and around the sizes of tiles
COUNTS = [[0, 0, 5, 0], [300, 0, 0, 1], [0, 1, 63, 64], [65, 127, 128, 129], [255, 256, 257, 0],
          [31, 32, 33, 15], [16, 17, 1, 2], [512, 511, 0, 513], [0, 0, 0, 0]]


@pytest.mark.parametrize("dtype,keep", [("bf16", "rows"), ("bf16", "int8"), ("f32", "rows")])
@pytest.mark.parametrize("counts", COUNTS)
def test_uneven_experts(counts, dtype, keep):
    say(f"[ffn uneven] {counts} {dtype} {keep}")
    T = max(8, -(-sum(counts) // 2) + 3)
    c = Case(T, 192, 208, 4, 2, dtype, keep, counts=counts)
    check_forward(c, *c.train())
    got = c.backward()
    check_backward(c, got, *clean(c))
    for e, n in enumerate(counts):
        if n == 0:                                   # an expert without rows: zeros, written
            assert not any(bool(v[e].any()) for v in got[1:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_then_backward_of_what_it_kept(dtype):
    for keep in ("rows", "int8"):
        c = Case(150, 256, 144, 6, 3, dtype, keep, 0.2)
        _, c.kept, c.scale = c.train()
        check_backward(c, c.backward(), *clean(c))


@pytest.mark.parametrize("T,k,counts", [(90, 2, None), (9, 2, None), (400, 1, [300, 0, 90, 10])])
@pytest.mark.parametrize("dtype,dw", [("bf16", "same"), ("bf16", "f32"), ("f32", "same")])
def test_gradients_added(T, k, counts, dtype, dw):
    c = Case(T, 128, 80, 4, k, dtype, "rows", 0.1, counts=counts)
    g, u = clean(c)
    half = U if dw == "f32" else HALF[dtype]
    out = c.grads(dw)
    c.backward(out)
    check_backward(c, out, g, u, dw_half=half)
    before = [None] + [torch.randn_like(v) for v in out[1:]]
    out = [out[0]] + [b.clone() for b in before[1:]]
    c.backward(out, accumulate_dw=True)
    check_backward(c, out, g, u, before=[None] + [f64(b) for b in before[1:]], dw_half=half)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_some_gradients(dtype, T):
    """Each output alone, and without the inputs that it does not need."""
    c = Case(T, 192, 96, 5, 2, dtype, "int8", 0.1)
    every = c.backward()
    for i in range(4):
        out = [v if i == j else None for j, v in enumerate(c.grads())]
        w = dict(c.w)
        if i != 0:
            w["w_gate"] = w["w_up"] = None
        x, perm = (c.x, c.perm) if i in (1, 2) else (None, None)
        M.moe_expert_ffn_backward(c.dims, c.T, x, w, c.offsets, perm, c.kept, c.dy, *out, c.ws,
                                  kept_scale=c.scale)
        assert torch.equal(out[i], every[i])


@pytest.mark.parametrize("T,dtype,keep", [(300, "bf16", "int8"), (7, "bf16", "rows"), (300, "f32", "rows")])
def test_repeats_are_bitwise_equal(T, dtype, keep):
    c = Case(T, 256, 320, 8, 2, dtype, keep, 0.1)
    first = [v.clone() for v in c.train() if v is not None] + [v.clone() for v in c.backward()]
    c.ws.zero_()
    again = [v for v in c.train() if v is not None] + c.backward()
    assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_a_larger_workspace_and_no_tokens():
    c = Case(50, 128, 48, 4, 2, "bf16", "rows")
    ref = c.train()
    c.ws = torch.empty(M.moe_expert_ffn_train_size(c.dims, 500), dtype=torch.uint8, device="cuda")
    assert all(torch.equal(a, b) for a, b in zip(ref[:2], c.train()[:2]))
    with pytest.raises(M.MoEError, match="orkspace"):
        M.moe_expert_ffn_train(c.dims, c.T, c.x, c.w, c.offsets, c.perm, ref[0], ref[1], c.ws[:1024])
    out = c.grads()
    e = torch.empty(0, device="cuda", dtype=torch.bfloat16)
    M.moe_expert_ffn_backward(c.dims, 0, e, c.w, c.offsets, c.perm, e, e, *out, c.ws)
    assert bool((out[0] == MARK).all()) and not any(bool(v.any()) for v in out[1:])


@pytest.mark.parametrize("T,dtype", [(6, "bf16"), (260, "bf16"), (70, "f32")])
def test_captured_and_replayed(T, dtype):
    """A graph of forward and backward, replayed between eager calls on another
    stream, on inputs that change."""
    c = Case(T, 256, 192, 6, 2, dtype, "int8", 0.1)
    out = c.outputs()
    grads = c.grads()

    def step():
        c.train(out)
        M.moe_expert_ffn_backward(c.dims, c.T, c.x, c.w, c.offsets, c.perm, out[1], c.dy, *grads, c.ws,
                                  kept_scale=out[2])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other, side = Case(T, 256, 192, 6, 2, dtype, "int8", 0.1, seed=5), torch.cuda.Stream()
    ref_side = [v.clone() for v in other.backward()]
    torch.cuda.synchronize()
    for i in range(4):
        c.x.copy_(torch.randn(c.T, c.H, generator=gen(i)).to(c.x.dtype))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            beside = other.backward()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [v.clone() for v in out] + [v.clone() for v in grads]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, list(out) + grads)), i
        assert all(torch.equal(a, b) for a, b in zip(ref_side, beside)), i


def test_layer_trained_through_its_entry_points():
    """route, permute, the experts and the way back, then every gradient of the
    chain, against autograd in 64 bits."""
    T, H, I, E, k = 45, 128, 96, 6, 2
    g = gen(9)
    d = M.Dims(hidden=H, n_experts=E, top_k=k, inter=I, dtype="f32", renormalize=True)
    x, wr = randn(g, T, H), randn(g, E, H, std=H ** -0.5)
    w = {"w_gate": randn(g, E, I, H, std=H ** -0.5), "w_up": randn(g, E, I, H, std=H ** -0.5),
         "w_down": randn(g, E, H, I, std=I ** -0.5)}
    dout, dev, P = randn(g, T, H), dict(device="cuda"), T * k
    i32 = dict(dtype=torch.int32, **dev)
    ids, tw = torch.empty(T, k, **i32), torch.empty(T, k, **dev)
    exact, flags = torch.empty(T, k, dtype=torch.uint8, **dev), torch.empty(T, **i32)
    logits = torch.empty(T, E, **dev)
    M.moe_route(d, T, x, wr, None, 0, "standard", ids, tw, exact, flags, logits)
    off, perm, inv = torch.empty(E + 1, **i32), torch.empty(P, **i32), torch.empty(P, **i32)
    M.moe_permute(T, k, E, ids, exact, off, perm, inv)
    ws = torch.empty(M.moe_expert_ffn_train_size(d, T), dtype=torch.uint8, **dev)
    y, kept, out = torch.empty(P, H, **dev), torch.empty(P, 2, I, **dev), torch.empty(T, H, **dev)
    M.moe_expert_ffn_train(d, T, x, w, off, perm, y, kept, ws)
    M.moe_undispatch(d, T, y, inv, tw, out)
    dy, dtw = torch.empty(P, H, **dev), torch.empty(T, k, **dev)
    M.moe_undispatch_backward(d, T, dout, y, inv, tw, dy, dtw)
    dxp = torch.empty(P, H, **dev)
    dw = [torch.empty_like(w[n]) for n in ("w_gate", "w_up", "w_down")]
    M.moe_expert_ffn_backward(d, T, x, w, off, perm, kept, dy, dxp, *dw, ws)
    dx, dl, dwr = torch.empty(T, H, **dev), torch.empty(T, E, **dev), torch.empty(E, H, **dev)
    M.moe_undispatch(d, T, dxp, inv, None, dx)
    ws2 = torch.empty(M.moe_route_backward_size(d, T), dtype=torch.uint8, **dev)
    M.moe_route_backward(d, T, x, wr, ids, logits, dtw, dl, dx, dwr, ws2, dx_add=dx)

    leaves = [t.cpu().double().requires_grad_() for t in (x, wr, *w.values())]
    xr, wrr, wg, wu, wd = leaves
    at = ids.cpu().long()
    p = torch.softmax((xr @ wrr.T).gather(1, at), 1)
    ref = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        e = at[:, j]
        gate = torch.bmm(wg[e], xr[:, :, None])[:, :, 0]
        up = torch.bmm(wu[e], xr[:, :, None])[:, :, 0]
        ref = ref + p[:, j:j + 1] * torch.bmm(wd[e], (torch.nn.functional.silu(gate) * up)[:, :, None])[:, :, 0]
    ref.backward(dout.cpu().double())
    # chains of up to four fp32 products of a few hundred terms: relative to the
    # 2-norm their roundings stay far below 2 * 400 u = 5e-5
    for name, got, want in zip(("out", "dx", "dw_router", "dw_gate", "dw_up", "dw_down"),
                               (out, dx, dwr, *dw), (ref, *(t.grad for t in leaves))):
        want = want.detach()
        err = float((got.cpu().double() - want).norm() / want.norm())
        assert err < 5e-5, (name, err)


# ------------------------------------------------------- rows in 8 bits ----
ROWS8 = [  # rows, cols, ld, dtype
    (1, 1, 1, "f32"), (1, 64, 64, "bf16"), (3, 63, 63, "bf16"), (5, 65, 70, "f32"), (1, 1000, 1000, "bf16"),
    (7, 16, 16, "f32"), (9, 48, 56, "bf16"), (33, 2048, 2048, "bf16"), (33, 200, 208, "f32"),
    (130, 1411, 1416, "f32"), (129, 1411, 1411, "bf16"), (1000, 80, 80, "bf16"), (64, 4096, 4101, "bf16"),
]


@pytest.mark.parametrize("T,H,I,E,k,dtype,keep", [(70, 128, 96, 4, 2, "bf16", "int8"), (70, 128, 96, 4, 2, "f32", "rows"),
                                                   (1500, 512, 1024, 4, 2, "bf16", "rows")])
def test_values_that_are_not_finite_stay_where_they_belong(T, H, I, E, k, dtype, keep):
    """A token whose pairs are not computed reaches nothing; an infinity in one
    pair's row reaches that row's outputs and its expert's weights alone."""
    c = Case(T, H, I, E, k, dtype, keep, 0.3, pack=False)
    clean, grads = c.train(), c.backward()
    used = torch.zeros(T, dtype=torch.bool)
    used[torch.div(c.perm[:c.n].cpu().long(), k, rounding_mode="floor")] = True
    assert not bool(used.all())
    c.x[~used.cuda()] = float("nan")
    for a, b in zip(clean, c.train()):
        assert a is b or torch.equal(a, b)
    assert all(torch.equal(a, b) for a, b in zip(grads, c.backward()))
    off = c.offsets.tolist()
    p, e = off[2] - 1, 1                  # the last row of expert 1
    token = int(c.perm[p]) // k
    row = c.dy[p, 5].clone()
    c.dy[p, 5] = float("inf")
    got = c.backward()
    keep_rows = torch.arange(c.P, device="cuda") != p
    assert torch.equal(got[0][keep_rows], grads[0][keep_rows]) and not bool(got[0][p].isfinite().any())
    for a, b in zip(got[1:], grads[1:]):
        others = [i for i in range(E) if i != e]
        assert torch.equal(a[others], b[others]) and not bool(a[e].isfinite().all())
    c.dy[p, 5] = row
    c.x[token, 3] = float("inf")
    mine = (torch.div(c.perm[:c.n].long(), k, rounding_mode="floor") == token).nonzero().flatten()
    y, kept, scale = c.train()
    others = torch.ones(c.P, dtype=torch.bool, device="cuda")
    others[mine] = False
    assert torch.equal(y[others], clean[0][others]) and torch.equal(kept[others], clean[1][others])
    assert not bool(y[mine].isfinite().any())
    if scale is not None:                 # comes back as NaN
        assert torch.equal(scale[others], clean[2][others]) and bool(scale[mine].isnan().all())
        assert bool((kept[mine] == 0).all())


@pytest.mark.parametrize("dtype,keep", [("bf16", "int8"), ("f32", "rows")])
def test_two_streams_at_once(dtype, keep):
    cases = [Case(T, 256, 160, 6, 2, dtype, keep, 0.1, seed=s, pack=False) for s, T in enumerate((700, 333))]
    want = [(c.train(), c.backward()) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [(c.outputs(), c.grads()) for c in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for c, s, (out, grads) in zip(cases, streams, outs):
            c.train(out, stream=s)
            c.backward(grads, stream=s)
    torch.cuda.synchronize()
    for (w, wg), (o, og) in zip(want, outs):
        assert all(a is b or torch.equal(a, b) for a, b in zip((*w, *wg), (*o, *og)))


@pytest.mark.parametrize("rows,cols,ld,dtype", ROWS8)
def test_rows8(rows, cols, ld, dtype):
    say(f"[rows8] {rows}x{cols} ld={ld} {dtype}")
    g = gen(rows + cols)
    src = randn(g, rows, ld, dtype=dtype) * randn(g, rows, 1).exp().to(TT[dtype])
    if cols > 2:
        src[0, 2] = 0
        src[rows - 1, :min(cols, 64)] = 0          # a block of zeros
    blocks = -(-cols // 64)
    codes = torch.full((rows, cols), 5, dtype=torch.int8, device="cuda")
    scale = torch.full((rows, blocks), MARK, device="cuda")
    dst = torch.full((rows, ld), MARK, dtype=TT[dtype], device="cuda")
    M.moe_rows_pack8(rows, cols, src, codes, scale)
    M.moe_rows_unpack8(rows, cols, codes, scale, dst)
    v = f64(src)[:, :cols]
    want_c, want_s = FO.pack8(v)
    assert np.array_equal(f64(codes), want_c)      # the nearer code, decided in 64 bits on both sides
    near(scale, want_s, U * want_s, "scale")
    back = FO.unpack8(want_c, f64(scale))
    near(f64(dst)[:, :cols], back, (HALF[dtype] + U) * np.abs(back), "values")
    assert bool((dst[:, cols:] == MARK).all())


@pytest.mark.parametrize("cols,dtype", [(192, "f32"), (192, "bf16"), (191, "f32")])
def test_rows8_special_values(cols, dtype):
    src = torch.randn(6, cols, generator=gen(1)).to(TT[dtype])
    src[0, 3], src[1, 70], src[2, 130] = float("nan"), float("inf"), -float("inf")
    src[3, 64:128] = 1e-36                          # below 2^-100
    src[4, 64:128] *= 2.0 ** -90
    src[5, 0] = torch.finfo(TT[dtype]).max
    src = src.cuda()
    codes = torch.empty(6, cols, dtype=torch.int8, device="cuda")
    scale = torch.empty(6, 3, device="cuda")
    dst = torch.empty_like(src)
    M.moe_rows_pack8(6, cols, src, codes, scale)
    M.moe_rows_unpack8(6, cols, codes, scale, dst)
    want_c, want_s = FO.pack8(f64(src))
    assert np.array_equal(f64(codes), want_c) and np.array_equal(np.isnan(f64(scale)), np.isnan(want_s))
    got, want = f64(dst), FO.unpack8(want_c, want_s)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and not got[3, 64:128].any()
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= (HALF[dtype] + 3 * U) * np.abs(want)[ok]).all()


def test_rows8_many_and_other_strides():
    """More lanes than 2^22 and a given ld, against the GPU's 64 bits."""
    rows, cols, ld = 20001, 333, 400
    src = torch.randn(rows * ld, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda")
    codes = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    scale = torch.empty(rows, 6, device="cuda")
    M.moe_rows_pack8(rows, cols, src, codes, scale, ld=ld)
    v = src.view(rows, ld)[:, :cols].double()
    for b in range(6):
        c = slice(64 * b, min(cols, 64 * b + 64))
        top = v[:, c].abs().amax(1, keepdim=True)
        assert torch.equal(codes[:, c].double(), torch.round(v[:, c] * 127 / top))
    dst = torch.full((rows * ld,), MARK, device="cuda")
    M.moe_rows_unpack8(rows, cols, codes, scale, dst, ld=ld)
    want = codes.float() * scale.repeat_interleave(64, 1)[:, :cols]
    assert torch.equal(dst.view(rows, ld)[:, :cols], want)
    assert bool((dst.view(rows, ld)[:, cols:] == MARK).all())


def test_rows8_the_most_blocks():
    rows = (1 << 28) - 16
    src = (torch.arange(rows, dtype=torch.int32, device="cuda") % 251 - 125).to(torch.bfloat16).view(rows, 1)
    codes = torch.zeros(rows, 1, dtype=torch.int8, device="cuda")
    scale = torch.full((rows, 1), float("nan"), device="cuda")
    M.moe_rows_pack8(rows, 1, src, codes, scale)
    assert torch.equal(codes, (127 * torch.sign(src)).to(torch.int8))
    got = torch.empty_like(src)
    M.moe_rows_unpack8(rows, 1, codes, scale, got)
    assert torch.equal(got, src)         # 127 (top / 127) rounds to top in bf16


def test_refusals_with_gpu_tensors():
    c = Case(4, 64, 32, 2, 1, "bf16", "rows")
    y, kept, _ = c.outputs()
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_expert_ffn_train(c.dims, 4, c.x.t().contiguous().t(), c.w, c.offsets, c.perm, y, kept, c.ws)
    with pytest.raises(TypeError, match="w_gate"):
        M.moe_expert_ffn_train(c.dims, 4, c.x, {**c.w, "w_gate": c.w["w_gate"].float()}, c.offsets, c.perm,
                               y, kept, c.ws)
    with pytest.raises(M.MoEError):                  # the product of what is kept over itself
        M.moe_expert_ffn_train(c.dims, 4, c.x, c.w, c.offsets, c.perm, c.x, kept, c.ws)
    packed = dataclasses.replace(c.dims, weight_layout="mfma16")
    with pytest.raises(M.MoEError):
        M.moe_expert_ffn_train(packed, 4, c.x, c.w, c.offsets, c.perm, y, kept, c.ws)
