"""Training operators, without a GPU: the fp64 oracle against finite
differences and identities, and the entry points' refusals (status codes from
include/moe_route.h, before any HIP call)."""
import copy
import ctypes
import dataclasses
import pathlib
import pickle
import re
import types

import numpy as np
import pytest
import torch

import sparse_moe_layer_route_amd as M
from oracle import train_oracle as TO
from sparse_moe_layer_route_amd import binding as B

L = B._lib
A = 0x100000                      # aligned, never dereferenced: every call below is refused


def dims(**kw):
    d = dict(hidden=256, n_experts=8, top_k=2, inter=512, dtype="bf16")
    d.update(kw)
    return M.Dims(**d)


# ------------------------------------------------------------- oracle pins --
def numeric(f, x, h=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("ids", [[[0, 2], [3, 1], [4, 0]], [[0, -1], [9, -1], [2, 2]]])
def test_route_gradient_matches_differences(renorm, ids):
    rng = np.random.default_rng(5)
    l, g, ids = rng.normal(size=(3, 5)), rng.normal(size=(3, 2)), np.array(ids)
    # central differences of a smooth function: h^2 terms of order 1e-10
    num = numeric(lambda v: float((TO.route_weights(v, ids, renorm) * g).sum()), l)
    got = TO.route_dlogits(l, ids, g, renorm)
    assert np.abs(got - num).max() < 1e-8
    assert np.abs(got.sum(1)).max() < 1e-12       # softmax: a shift of a row changes nothing


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_matches_differences(tail):
    rng = np.random.default_rng(6)
    T, V, K, tau = 4, 7, 3, 1.7
    s, teacher = rng.normal(size=(T, V)), rng.normal(size=(T, V)) * 2
    ids = np.argsort(-teacher, axis=1)[:, :K].copy()
    u = np.take_along_axis(teacher, ids, 1)
    ids[1, 2] = -1                                 # a skipped entry
    ids[2, 1] = ids[2, 0]                          # a class named twice
    lse = np.log(np.exp(teacher / tau).sum(1)) if tail else None
    w = np.array([1.0, 0.5, 2.0, 0.0])
    f = lambda v: float(TO.distill(v, ids, u, tau, lse, w, 0.3)[0].sum())
    loss, grad = TO.distill(s, ids, u, tau, lse, w, 0.3)
    assert np.abs(grad - numeric(f, s)).max() < 1e-8
    assert loss[3] == 0 and not grad[3].any()


def test_distill_of_itself_is_zero():
    rng = np.random.default_rng(7)
    s = rng.normal(size=(3, 9))
    ids = np.argsort(-s, axis=1)[:, :4]
    u = np.take_along_axis(s, ids, 1)
    loss, grad = TO.distill(s, ids, u, 1.0, np.log(np.exp(s).sum(1)))
    assert np.abs(loss).max() < 1e-15 and np.abs(grad).max() < 1e-15
    full = np.argsort(-s, axis=1)                  # all classes named
    loss, grad = TO.distill(s, full, np.take_along_axis(s, full, 1), 1.0)
    assert np.abs(loss).max() < 1e-15 and np.abs(grad).max() < 1e-15


def test_sorted_rows_and_back():
    rng = np.random.default_rng(8)
    T, k, H = 5, 2, 3
    x, dout, w = rng.normal(size=(T, H)), rng.normal(size=(T, H)), rng.normal(size=(T, k))
    inv = rng.permutation(T * k)
    inv[3] = -1
    rows = TO.dispatch(x, inv, k, np.zeros((T * k, H)))
    y = rng.normal(size=rows.shape)
    # <undispatch(y), dout> is linear in y and in w: its gradients are exact adjoints
    dy, dw = TO.undispatch_backward(dout, y, inv, k, w, np.zeros_like(y))
    s = (TO.undispatch(y, inv, k, w) * dout).sum()
    assert abs((dy * y).sum() - s) < 1e-12 and abs((dw * w).sum() - s) < 1e-12
    # dispatch and unweighted undispatch are adjoint
    assert abs((rows * y).sum() - (x * TO.undispatch(y, inv, k)).sum()) < 1e-12


# --------------------------------------------------------------- refusals --
def test_sorted_rows_refusals():
    d = dims()
    c = ctypes.byref(d.c())
    T, P, xb = 16, 32, 16 * 256 * 2
    X, I, R, W, O, G = A, A + (1 << 20), A + (2 << 20), A + (3 << 20), A + (4 << 20), A + (5 << 20)
    dp, un, ub = L.moe_dispatch, L.moe_undispatch, L.moe_undispatch_backward
    for bad in [(None, I, R), (X, None, R), (X, I, None), (X + 8, I, R), (X, I, X + xb - 16),
                (X, R, R)]:
        assert dp(c, T, *bad, None) == B.MOE_EINVAL
    assert dp(None, T, X, I, R, None) == B.MOE_EINVAL
    assert dp(c, -1, X, I, R, None) == B.MOE_EINVAL
    assert dp(c, (1 << 22) + 1, X, I, R, None) == B.MOE_EUNSUPPORTED
    assert dp(c, 1 << 22, X, I, R, None) == B.MOE_EUNSUPPORTED          # T*k*H = 2^31
    assert dp(c, 0, None, None, None, None) == B.MOE_OK
    for bad in [(None, 1, I, W, None, O), (R, 1, None, W, None, O), (R, 1, I, W, None, None),
                (R, 2, I, W, None, O), (R, 1, I, W, O + 16, O), (R, 1, I, W, None, R),
                (R, 1, I, O, None, O), (R, 1, I, W + 4, None, O)]:
        assert un(c, T, *bad, None) == B.MOE_EINVAL
    assert un(c, 0, None, 1, None, None, None, None, None) == B.MOE_OK
    f = dims(dtype="f32")
    assert un(ctypes.byref(f.c()), T, R, 1, I, W, None, O, None) == B.MOE_EUNSUPPORTED
    for bad in [(O, R, 1, I, W, None, None), (O, None, 1, I, W, G, W + 4096), (O, R, 1, I, None, G, None),
                (O, R, 1, I, W, R, None), (O, R, 1, I, W, O, None), (O, R, 1, I, W, G, W),
                (O, R, 1, I, W, G, G), (None, R, 1, I, W, G, None)]:
        assert ub(c, T, *bad, None) == B.MOE_EINVAL


def route_bwd(d, T, **kw):
    names = ["x", "w", "ids", "logits", "dtopk_w", "dl_add", "dl", "dx_add", "dx", "dw", "acc", "ws", "n"]
    base = {n: A + (i << 24) for i, n in enumerate(names)}
    base.update(dl_add=None, dx_add=None, acc=0, n=1 << 24)
    base.update(kw)
    return L.moe_route_backward(ctypes.byref(d.c()), T, *[base[n] for n in names], None)


def test_route_backward_refusals():
    d, T = dims(), 16
    at = lambda i: A + (i << 24)
    assert M.moe_route_backward_size(d, T) > 0
    n = ctypes.c_size_t(0)
    assert L.moe_route_backward_size(ctypes.byref(d.c()), T, None) == B.MOE_EINVAL
    assert L.moe_route_backward_size(ctypes.byref(d.c()), -1, ctypes.byref(n)) == B.MOE_EINVAL
    assert L.moe_route_backward_size(ctypes.byref(dims(n_experts=65).c()), T,
                                     ctypes.byref(n)) == B.MOE_EUNSUPPORTED
    assert L.moe_route_backward_size(ctypes.byref(dims(hidden=1 << 26, n_experts=32, inter=16).c()), 1,
                                     ctypes.byref(n)) == B.MOE_EUNSUPPORTED      # E * H = 2^31
    assert L.moe_route_backward_size(ctypes.byref(dims(hidden=(1 << 24) + 64, inter=16).c()), 1,
                                     ctypes.byref(n)) == B.MOE_EUNSUPPORTED
    for kw in [dict(dl=None), dict(dtopk_w=None), dict(ids=None), dict(logits=None), dict(w=None),
               dict(x=None), dict(acc=2), dict(ws=None), dict(dx=None, dx_add=at(7)),
               dict(dx=at(0)), dict(dl=at(3)), dict(dw=at(6)), dict(dl_add=at(6) + 16),
               dict(dx_add=at(8) + 16), dict(ws=at(9)), dict(x=A + 2), dict(dw=at(9) + 4)]:
        assert route_bwd(d, T, **kw) == B.MOE_EINVAL, kw
    assert route_bwd(d, T, n=M.moe_route_backward_size(d, T) - 1) == B.MOE_EWORKSPACE
    assert route_bwd(d, 0, dw=None) == B.MOE_OK
    assert route_bwd(d, 0, acc=1) == B.MOE_OK
    assert route_bwd(d, 0, dw=at(9) + 4) == B.MOE_EINVAL


def distill(T=16, V=100, ld=100, K=4, **kw):
    names = ["student", "dtype", "ids", "u", "lse", "w", "tau", "scale", "loss", "ds", "ws", "n"]
    base = {n: A + (i << 24) for i, n in enumerate(names)}
    base.update(dtype=0, tau=1.0, scale=1.0, n=1 << 24)
    base.update(kw)
    return L.moe_distill_topk(T, V, ld, K, *[base[n] for n in names], None)


def test_distill_refusals():
    nan, inf = float("nan"), float("inf")
    for kw in [dict(V=0), dict(K=0), dict(ld=99), dict(T=-1), dict(dtype=2), dict(tau=0.0),
               dict(tau=-1.0), dict(tau=nan), dict(tau=inf), dict(scale=nan), dict(scale=inf),
               dict(student=None), dict(ids=None), dict(u=None), dict(loss=None),
               dict(student=A + 4), dict(ds=A + 16), dict(loss=A), dict(ds=A + (2 << 24))]:
        assert distill(**kw) == B.MOE_EINVAL, kw
    for kw in [dict(V=(1 << 18) + 1, ld=1 << 20), dict(K=1025), dict(T=(1 << 22) + 1),
               dict(ld=(1 << 31) + 1), dict(tau=1e-7), dict(tau=2e6)]:
        assert distill(**kw) == B.MOE_EUNSUPPORTED, kw
    assert distill(T=0, student=None) == B.MOE_OK
    n = ctypes.c_size_t(0)
    assert L.moe_distill_topk_size(4, 100, None) == B.MOE_EINVAL
    assert L.moe_distill_topk_size(4, 0, ctypes.byref(n)) == B.MOE_EINVAL
    assert L.moe_distill_topk_size(4, (1 << 18) + 1, ctypes.byref(n)) == B.MOE_EUNSUPPORTED


def test_binding_refuses_host_tensors_and_other_types():
    d = dims()
    x, inv = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(8, dtype=torch.int32)
    rows = torch.zeros(8, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.moe_dispatch(d, 4, x, inv, rows)
    with pytest.raises(TypeError):
        M.moe_undispatch(d, 4, rows.half(), inv, None, x)
    with pytest.raises(TypeError):
        M.moe_undispatch_backward(d, 4, x, None, inv, None, None, None)
    with pytest.raises(TypeError):
        M.moe_dispatch(d, 4, None, inv, rows)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,E", [(64, 2), (64, 17), (1536, 40), (3584, 64), (40000 // 64 * 64, 9)])
def test_route_workspace_serves_fewer_tokens(H, E, dtype):
    """A workspace made for T tokens is no smaller than one for any fewer."""
    d = M.Dims(hidden=H, n_experts=E, top_k=2, inter=64, dtype=dtype)
    sizes = [M.moe_route_backward_size(d, T) for T in range(0, 20000, 13)]
    assert sizes == sorted(sizes) and sizes[0] == 0


@pytest.mark.parametrize("V", [3, 4096, 16380, 33000, 66000, 131080, 262144])
def test_distill_workspace_serves_fewer_rows(V):
    sizes = [M.moe_distill_topk_size(T, V) for T in [*range(300), *range(300, 40000, 997)]]
    assert sizes == sorted(sizes) and sizes[0] == 0


# ----------------------------------------------------------------- sources --
def test_barriers_are_for_whole_blocks():
    """A device function with a barrier in it is never called for some of a
    block's waves or lanes only: a barrier that part of a block does not reach
    has no meaning."""
    csrc = pathlib.Path(M.__file__).parent / "csrc"
    text = "\n".join(re.sub(r"//[^\n]*", "", f.read_text()) for f in sorted(csrc.iterdir())
                     if f.suffix in (".hip", ".h"))
    bodies = re.split(r"\n}", text)                     # functions end in column 0
    names = {re.findall(r"\b(?:void|int|float|bool) (\w+)\(", b)[0] for b in bodies
             if "__syncthreads()" in b and re.search(r"__device__[^;{]*\b(?:void|int|float|bool) \w+\(", b)}
    assert "route_dw" in names
    own = r"\b(?:wv|wave|lane|tid|threadIdx|l)\b"
    for name in names | {"__syncthreads"}:
        for cond in re.findall(r"if \(([^;{}]*?)\)\s*" + name + r"\s*[<(]", text):
            assert not re.search(own, cond), f"{name} under if ({cond})"


# -------------------------------------------------------------------- Dims --
def as_dict(c):
    return {n: getattr(c, n) for n, _ in c._fields_}


def test_dims_hold_their_fields_alone():
    """A call leaves a Dims as it was: its attributes are the fields."""
    d = dims(renormalize=True)
    before = dict(vars(d))
    M.moe_route_backward_size(d, 16)
    M.moe_workspace_size(d, 16, "standard")
    assert vars(d) == before and set(before) == {f.name for f in dataclasses.fields(d)}
    assert M.Dims(**vars(d)) == d
    for e in (copy.copy(d), copy.deepcopy(d), pickle.loads(pickle.dumps(d)), dataclasses.replace(d)):
        assert e == d and vars(e) == before and as_dict(B._dims(e)) == as_dict(d.c())
        e.hidden = 512
        assert B._dims(e).hidden == 512 and B._dims(d).hidden == 256


def test_dims_changed_between_calls():
    """Whatever way a field changes, the next call takes the new value."""
    d = dims()
    steps = [lambda: setattr(d, "hidden", 128), lambda: d.__dict__.update(n_experts=16),
             lambda: object.__setattr__(d, "top_k", 4), lambda: setattr(d, "renormalize", True),
             lambda: setattr(d, "n_shared", 2), lambda: delattr(d, "n_shared"),
             lambda: setattr(d, "dtype", "f32"), lambda: setattr(d, "tie_margin", 0.5),
             lambda: [delattr(d, "lore_rank"), delattr(d, "floe_keep"), setattr(d, "floe_keep", 8),
                      setattr(d, "lore_rank", 16)],
             lambda: [delattr(d, "lore_rank"), delattr(d, "floe_keep"), setattr(d, "lore_rank", 8),
                      setattr(d, "floe_keep", 16)]]
    for step in steps:
        B._dims(d)
        step()
        assert as_dict(B._dims(d)) == as_dict(d.c())

    class Wide(M.Dims):
        scale = 1

        def c(self):
            c = super().c()
            c.hidden *= self.scale
            return c

    w = Wide(hidden=64, n_experts=4, top_k=2, inter=64)
    assert B._dims(w).hidden == 64
    Wide.scale = 2
    assert B._dims(w).hidden == 128


def test_dims_changed_while_converted():
    """A field set while another thread converts the old values is not lost."""
    d = dims()
    convert = M.Dims.c

    def slow(self):
        c = convert(self)
        d.hidden = 1024                      # what another thread does here
        return c
    M.Dims.c = slow
    try:
        B._dims(d)
    finally:
        M.Dims.c = convert
    assert B._dims(d).hidden == 1024


# ------------------------------------------------------------ row lengths --
def test_distill_refuses_rows_of_other_lengths(monkeypatch):
    """The first K of a teacher's longer rows, or a gradient in rows of another
    stride, would be taken from the wrong places: refused, not answered."""
    T, V, K = 6, 20, 4
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    calls = []
    # host tensors for the current GPU's, and a library that only counts
    monkeypatch.setattr(B, "_device", lambda stream: -1)
    monkeypatch.setattr(B, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(B, "_lib", types.SimpleNamespace(
        moe_distill_topk=lambda *a: calls.append(a) or B.MOE_OK))

    def call(ids=(T, K), u=(T, K), ds=(T, V), student=(T, V), T=T, **kw):
        M.moe_distill_topk(T, V, K, z(*student), z(*ids, dtype=torch.int32), z(*u), z(T),
                           None if ds is None else z(*ds), None, **kw)
    for kw in [dict(ids=(T, 2 * K)), dict(u=(T, 2 * K)), dict(ds=(T, V + 4)), dict(ids=(2, 3, K + 1))]:
        with pytest.raises(ValueError, match="rows of"):
            call(**kw)
    assert not calls
    # one row, flat tensors, more rows than the call's, other shapes of as many elements, a
    # stride of the caller's
    fine = [dict(T=1, ids=(1, 2 * K), ds=(1, V + 4)), dict(ids=(2 * T * K,)), dict(ids=(T + 3, K)),
            dict(ids=(2, 3, K)), dict(ids=(T * K, 1)), dict(ds=(T, 2, V // 2)), dict(ds=(2, 3, V)),
            dict(ds=None), dict(student=(T, 2, V), ds=(T, 2, V), ld=2 * V), dict(ds=(T * V + 8,)),
            dict(student=(T, V + 4), ds=(T, V + 4))]
    for kw in fine:
        call(**kw)
    assert len(calls) == len(fine) and calls[-1][2] == V + 4


def test_route_backward_takes_batches_that_sorted_rows_do_not():
    """Its limits are T <= 2^22, E * hidden < 2^31 and hidden <= 2^24 alone."""
    for H, k, T in [(2048, 8, 1 << 17), (2048, 8, (1 << 20) + 3), (2048, 1, 1 << 22), (1 << 20, 8, 1 << 22)]:
        assert T * k * H >= 1 << 31
        d = dims(hidden=H, n_experts=64, top_k=k, inter=64, dtype="f32")
        n = M.moe_route_backward_size(d, T)
        assert n >= T * 64 * 4
        far = lambda i: (1 << 56) + (i << 46)          # buffers of up to 2^44 bytes, never looked at
        names = ["x", "w", "ids", "logits", "dtopk_w", "dl", "dx", "dw", "ws"]
        at = {m: far(i) for i, m in enumerate(names)}
        assert route_bwd(d, T, **at, n=n - 1 - n // 2) == B.MOE_EWORKSPACE
        assert route_bwd(d, T, **{**at, "dx": at["x"] + T * H * 4 - 16}, n=n) == B.MOE_EINVAL
    n = ctypes.c_size_t(0)
    for T in (-1, (1 << 22) + 1):
        st = L.moe_route_backward_size(ctypes.byref(dims().c()), T, ctypes.byref(n))
        assert st == (B.MOE_EINVAL if T < 0 else B.MOE_EUNSUPPORTED)
