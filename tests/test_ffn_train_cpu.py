"""The experts' training operators without a GPU: the fp64 oracle against
finite differences and identities, and the entry points' refusals (status codes
from include/moe_route.h, before any HIP call)."""
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

import sparse_moe_layer_route_amd as M
from oracle import ffn_train_oracle as FO
from sparse_moe_layer_route_amd import binding as B

L = B._lib
A = 0x100000                      # aligned, never dereferenced: every call below is refused
STEP = 1 << 34                    # no two buffers of a call overlap


def dims(**kw):
    d = dict(hidden=256, n_experts=8, top_k=2, inter=512, dtype="bf16")
    d.update(kw)
    return M.Dims(**d)


# ------------------------------------------------------------- oracle pins --
def case(rng, T=5, H=4, I=3, E=3, k=2, here=None):
    ids = np.array([rng.permutation(E)[:k] for _ in range(T)])
    key = np.where(np.ones((T, k), bool) if here is None else here, ids, E).ravel()
    perm = np.argsort(key, kind="stable")
    offsets = np.concatenate(([0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])))
    return (rng.normal(size=(T, H)), rng.normal(size=(E, I, H)), rng.normal(size=(E, I, H)),
            rng.normal(size=(E, H, I)), offsets, perm, k)


def test_ffn_gradient_matches_differences():
    rng = np.random.default_rng(3)
    here = rng.random((5, 2)) < 0.8
    x, wg, wu, wd, off, perm, k = case(rng, here=here)
    P, n = len(perm), off[-1]
    dy = rng.normal(size=(P, x.shape[1]))

    def loss(x, wg, wu, wd):
        return float((FO.forward(x, wg, wu, wd, off, perm, k, P)[0] * dy)[:n].sum())

    _, g, u = FO.forward(x, wg, wu, wd, off, perm, k, P)
    dx, dwg, dwu, dwd = FO.backward(x, wg, wu, wd, off, perm, k, g, u, dy)
    dtok = np.zeros_like(x)                       # a token's gradient: the sum of its rows'
    np.add.at(dtok, perm[:n] // k, dx[:n])
    args = [x, wg, wu, wd]
    for i, want in enumerate((dtok, dwg, dwu, dwd)):
        for at in np.ndindex(*want.shape):
            lo, hi = [a.copy() for a in args], [a.copy() for a in args]
            lo[i][at] -= 1e-5
            hi[i][at] += 1e-5
            # central differences of a smooth function: h^2 terms of order 1e-9
            assert abs((loss(*hi) - loss(*lo)) / 2e-5 - want[at]) < 1e-7 * (1 + abs(want[at]))
    assert not dx[n:].any()


def test_ffn_oracle_by_hand():
    # one row, one channel: g = 2, u = -3, y = silu(2) * -3 * 0.5
    one = lambda v: np.full((1, 1, 1), float(v))
    y, g, u = FO.forward(np.ones((1, 1)), one(2), one(-3), one(0.5), [0, 1], [0], 1, 1)
    s = 1 / (1 + np.exp(-2.0))
    assert g[0, 0] == 2 and u[0, 0] == -3 and abs(y[0, 0] + 3 * s) < 1e-15
    _, dwg, dwu, dwd = FO.backward(np.ones((1, 1)), one(2), one(-3), one(0.5), [0, 1], [0], 1, g, u,
                                   np.ones((1, 1)))
    assert abs(dwd[0, 0, 0] + 6 * s) < 1e-14 and abs(dwu[0, 0, 0] - s) < 1e-15
    assert abs(dwg[0, 0, 0] + 1.5 * (s + 2 * s * (1 - s))) < 1e-15


def test_pack8_oracle():
    rng = np.random.default_rng(4)
    v = rng.normal(size=(3, 150))
    v[1, 64:128] = 0
    v[2, 128:] = 1e-40                            # below 2^-100
    codes, scale = FO.pack8(v)
    back = FO.unpack8(codes, scale)
    assert np.abs(codes).max() == 127 and not codes[1, 64:128].any() and not back[2, 128:].any()
    step = np.repeat(scale, 64, axis=1)[:, :150]
    assert (np.abs(back - v) <= step / 2 * (1 + 1e-12) + 1e-39).all()
    v[0, 3], v[1, 140] = np.nan, -np.inf
    codes, scale = FO.pack8(v)
    back = FO.unpack8(codes, scale)
    assert np.isnan(back[0, :64]).all() and np.isnan(back[1, 128:]).all()
    assert np.isfinite(back[0, 64:]).all() and np.isfinite(back[1, :128]).all()


# ---------------------------------------------------------------- refusals --
def train_args(d, T=4, keep=0, **kw):
    a = dict(x=A, w_gate=A + STEP, w_up=A + 2 * STEP, w_down=A + 3 * STEP, offsets=A + 4 * STEP,
             perm=A + 5 * STEP, keep=keep, kept=A + 6 * STEP, scale=A + 7 * STEP if keep else None,
             y=A + 8 * STEP, ws=A + 9 * STEP, ws_bytes=STEP)
    a.update(kw)
    return a


def train(d, T=4, **kw):
    a = train_args(d, T, **kw)
    w = B.MoeWeights(None, a["w_gate"], a["w_up"], a["w_down"])
    c = d.c() if isinstance(d, M.Dims) else d
    return L.moe_expert_ffn_train(ctypes.byref(c), T, a["x"], ctypes.byref(w), a["offsets"], a["perm"],
                                  a["keep"], a["kept"], a["scale"], a["y"], a["ws"], a["ws_bytes"], None)


def backward(d, T=4, dw_dtype=1, accumulate=0, **kw):
    a = dict(dx=A + 10 * STEP, dwg=A + 11 * STEP, dwu=A + 12 * STEP, dwd=A + 13 * STEP)
    a = {**train_args(d, T, **{n: v for n, v in kw.items() if n not in a}),
         **{n: kw.get(n, v) for n, v in a.items()}}
    w = B.MoeWeights(None, a["w_gate"], a["w_up"], a["w_down"])
    c = d.c() if isinstance(d, M.Dims) else d
    return L.moe_expert_ffn_backward(ctypes.byref(c), T, a["x"], ctypes.byref(w), a["offsets"], a["perm"],
                                     a["keep"], a["kept"], a["scale"], a["y"], a["dx"], a["dwg"],
                                     a["dwu"], a["dwd"], dw_dtype, accumulate, a["ws"], a["ws_bytes"], None)


BAD_DIMS = [(dict(hidden=250), 2), (dict(inter=500), 2), (dict(n_experts=65), 2), (dict(top_k=9, n_experts=16), 2),
            (dict(hidden=0), 1), (dict(weight_layout="mfma16"), 2), (dict(hidden=1 << 21), 2),
            (dict(inter=1 << 21, hidden=64), 2), (dict(dtype="bf16", up_format="int2_g64"), 2)]


@pytest.mark.parametrize("over,status", BAD_DIMS)
def test_dims_refused(over, status):
    n = ctypes.c_size_t(0)
    d = dims(**over)
    assert train(d) == status and backward(d) == status
    assert L.moe_expert_ffn_train_size(ctypes.byref(d.c()), 4, ctypes.byref(n)) == status


@pytest.mark.parametrize("call", [train, backward])
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(T=(1 << 22) + 1), 2), (dict(T=1 << 21), 2), (dict(keep=2), 1),
    (dict(w_down=None), 1), (dict(offsets=None), 1), (dict(kept=None), 1), (dict(y=None), 1),
    (dict(ws=None), 1), (dict(kept=A + 6 * STEP + 8), 1), (dict(x=A + 4), 1),
    (dict(scale=A + 7 * STEP), 1),                       # scales without 8 bits
    (dict(keep=1, scale=None), 1), (dict(ws_bytes=100), 3),
    (dict(ws=A), 1), (dict(ws=A + 6 * STEP), 1), (dict(ws=A + 8 * STEP - 16), 1)])
def test_calls_refused(call, kw, status):
    assert call(dims(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(perm=None), 1), (dict(w_gate=None), 1), (dict(w_up=None), 1),
    (dict(y=A), 1), (dict(kept=A + STEP), 1)])
def test_forward_refused(kw, status):
    assert train(dims(), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dx=None, dwg=None, dwu=None, dwd=None), 1), (dict(dw_dtype=2), 1), (dict(accumulate=2), 1),
    (dict(w_gate=None), 1), (dict(w_up=None), 1), (dict(x=None), 1), (dict(perm=None), 1),
    (dict(dwd=None, dwg=None, x=None), 1), (dict(dwg=A + 4), 1),
    (dict(dx=A), 1), (dict(dx=A + 8 * STEP), 1), (dict(dwu=A + 11 * STEP), 1), (dict(dwd=A + 3 * STEP), 1)])
def test_backward_refused(kw, status):
    assert backward(dims(), **kw) == status


def test_backward_types_refused():
    assert backward(dims(dtype="f32"), dw_dtype=1) == 2
    # an empty batch looks at its gradients' addresses alone
    assert backward(dims(), T=0, dwg=A + 4) == 1
    assert backward(dims(), T=0, dwu=A + 11 * STEP) == 1
    assert backward(dims(), T=0, accumulate=1) == 0
    assert backward(dims(), T=0, dwg=None, dwu=None, dwd=None) == 0
    assert train(dims(), T=0, x=None, w_gate=None, kept=None, y=None, ws=None) == 0


def rows8(fn, rows=4, cols=100, ld=128, src=A, dtype=1, codes=A + STEP, scale=A + 2 * STEP):
    if fn == "pack":
        return L.moe_rows_pack8(rows, cols, ld, src, dtype, codes, scale, None)
    return L.moe_rows_unpack8(rows, cols, ld, codes, scale, src, dtype, None)


@pytest.mark.parametrize("fn", ["pack", "unpack"])
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(ld=99), 1), (dict(dtype=2), 1), (dict(src=None), 1),
    (dict(codes=None), 1), (dict(scale=None), 1), (dict(src=A + 8), 1), (dict(codes=A + STEP + 4), 1),
    (dict(cols=(1 << 24) + 1, ld=1 << 25), 2), (dict(ld=(1 << 31) + 1), 2), (dict(rows=1 << 28), 2),
    (dict(rows=(1 << 28) - 15, cols=1), 2), (dict(rows=1 << 27), 2), (dict(codes=A), 1), (dict(scale=A + 16), 1)])
def test_rows8_refused(fn, kw, status):
    assert rows8(fn, **kw) == status


def test_rows8_empty():
    assert rows8("pack", rows=0, src=None, codes=None) == 0
    assert rows8("unpack", rows=0, src=None, codes=None) == 0


def test_workspace_serves_smaller_batches():
    d = dims()
    sizes = [M.moe_expert_ffn_train_size(d, T) for T in range(0, 300)]
    assert sizes == sorted(sizes)
    f = dataclasses.replace(d, dtype="f32")
    assert M.moe_expert_ffn_train_size(f, 64) >= M.moe_expert_ffn_train_size(d, 64)


def test_binding_refuses_before_any_call():
    d = dims()
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = {n: torch.zeros(8, 512, 256, dtype=torch.bfloat16) for n in ("w_gate", "w_up", "w_down")}
    i = torch.zeros(9, dtype=torch.int32)
    kept = torch.zeros(8, 2, 512, dtype=torch.bfloat16)
    ws = torch.zeros(10, dtype=torch.uint8)
    with pytest.raises(ValueError, match="kept"):        # host tensors
        M.moe_expert_ffn_train(d, 4, t, w, i, i, t, kept, ws)
    with pytest.raises(TypeError, match="int8"):
        M.moe_expert_ffn_train(d, 4, t, w, i, i, t, kept, ws, kept_scale=kept)
    with pytest.raises(ValueError, match="at least"):
        M.moe_expert_ffn_train(d, 5, t, w, i, i, t, kept, ws)
    with pytest.raises(TypeError, match="Tensor"):
        M.moe_expert_ffn_backward(d, 4, t, w, i, i, None, t, None, None, None, None, ws)
    with pytest.raises(TypeError, match="gradients"):
        M.moe_expert_ffn_backward(d, 4, t, w, i, i, kept, t, None, i, None, None, ws)
    with pytest.raises(TypeError, match="rows"):
        M.moe_rows_pack8(1, 9, i, i, i)
