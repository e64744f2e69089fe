"""Measured cases of the experts' training operators.

The gated feed-forward block of the experts over rows sorted by expert, with
what its backward pass needs kept as rows or in 8 bits (moe_expert_ffn_train);
its backward pass (moe_expert_ffn_backward); both as a training step; rows kept
in 8 bits and brought back (moe_rows_pack8, moe_rows_unpack8).

``own`` selects what ``run`` does: False computes each operator in elementary
torch operations in 32 bits, True calls the library.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 64           # columns that share a scale in 8 bits
SMALL = 2.0 ** -100  # a block whose largest value is below this is kept as zeros


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # eight tokens of a DeepSeek-V2-Lite-shaped layer, the forward pass of
        # a step on a handful of tokens: the weights' stream
        dict(name="train_few", op="train", dtype="bf16", T=8, H=2048, I=1408, E=64, k=6, miss=0.0),
        # a Granite-shaped training batch
        dict(name="train_batch", op="train", dtype="bf16", T=4096, H=1536, I=512, E=40, k=8,
             miss=0.0),
        # the small fp32 layer, an odd batch with slots that are not computed
        dict(name="train_f32", op="train", dtype="f32", T=333, H=256, I=512, E=8, k=2, miss=0.2),
        # gradients of a small fine-tuning batch, a few rows an expert
        dict(name="backward_few", op="backward", dtype="bf16", keep="rows", T=64, H=2048, I=1408,
             E=64, k=6, miss=0.0),
        # a ragged training batch, a tenth of the slots not computed
        dict(name="backward_ragged", op="backward", dtype="bf16", keep="rows", T=3001, H=2048,
             I=1408, E=64, k=6, miss=0.1),
        # the largest layer, gate and up rows kept in 8 bits
        dict(name="backward_large", op="backward", dtype="bf16", keep="int8", T=4096, H=3584,
             I=2560, E=64, k=8, miss=0.0),
        # the small fp32 layer's gradients
        dict(name="backward_f32", op="backward", dtype="f32", keep="int8", T=1000, H=256, I=512,
             E=8, k=2, miss=0.2),
        # forward and backward of a Granite-shaped training batch
        dict(name="step_batch", op="step", dtype="bf16", keep="int8", T=4096, H=1536, I=512, E=40,
             k=8, miss=0.0),
        # a shared expert: one expert that takes every token
        dict(name="step_shared", op="step", dtype="bf16", keep="rows", T=2048, H=2048, I=1408,
             E=1, k=1, miss=0.0),
        # a decoding batch's hidden states: launch latency
        dict(name="rows8_few", op="rows8", dtype="bf16", rows=64, cols=2048, pad=0),
        # a training batch's hidden states kept until the backward pass
        dict(name="rows8_batch", op="rows8", dtype="bf16", rows=16384, cols=3584, pad=0),
        # odd fp32 rows inside longer ones
        dict(name="rows8_odd", op="rows8", dtype="f32", rows=3001, cols=1411, pad=5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {w: max(work(c)[w] for c in listed()) for w in ("bytes", "flops")}
    while True:
        op = rng.choice(["train", "backward", "backward", "step", "rows8"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "rows8":
            case = dict(op=op, dtype=dtype, rows=_log_int(rng, 1, 65536),
                        cols=_log_int(rng, 1, 16384), pad=rng.choice([0, 0, 8, 3]))
        else:
            E = rng.randint(1, 64)
            case = dict(op=op, dtype=dtype, T=_log_int(rng, 1, 4096), H=64 * _log_int(rng, 1, 64),
                        I=16 * _log_int(rng, 1, 160), E=E, k=rng.randint(1, min(8, E)),
                        miss=rng.choice([0.0, 0.2, 0.9]))
            if op == "backward":
                case.update(keep=rng.choice(["rows", "int8"]))
            if op == "step":
                # fp32 gradients show where a sum's order moves a value to the next of 8 bits
                case.update(keep="rows" if dtype == "f32" else rng.choice(["rows", "int8"]))
        # fp32 products cost sixteen times bf16's on the matrix cores
        w = work(case)
        cost = w["flops"] * (16 if dtype == "f32" else 1)
        if w["bytes"] <= most["bytes"] and cost <= most["flops"]:
            return case


def work(case):
    b = _size(case["dtype"])
    if case["op"] == "rows8":
        n, blocks = case["rows"] * case["cols"], case["rows"] * -(-case["cols"] // BLOCK)
        return {"bytes": float(2 * (n * b + n + 4 * blocks)), "flops": 8.0 * n}
    H, I, E, k = case["H"], case["I"], case["E"], case["k"]
    P = case["T"] * k * (1.0 - case["miss"])
    weights = 3.0 * min(E, P) * I * H * b     # experts without rows need no weights
    x, rows = min(case["T"], P) * H * b, P * H * b
    kept = P * 2 * I * b
    if case.get("keep") == "int8":
        kept = P * 2 * (I + 4 * -(-I // BLOCK))
    forward = weights + x + kept + rows
    # weights, x, dy and what was kept are read, all gradients written
    backward = weights + x + 2 * rows + kept + 3.0 * E * I * H * b
    product = 2.0 * P * I * H
    return {"train": {"bytes": forward, "flops": 3 * product},
            "backward": {"bytes": backward, "flops": 6 * product},
            "step": {"bytes": forward + backward, "flops": 9 * product}}[case["op"]]


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _torch(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


# ------------------------------------------------------------------ inputs --
def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype).mul_(std)


def _sorted_pairs(g, case):
    """expert_offsets and perm of the stable sort by expert, the experts drawn
    unevenly; perm's entries behind the last computed pair are not read."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = _randn(g, T, E) + _randn(g, E, std=0.3)
    ids = torch.topk(logits, k, dim=1).indices
    here = torch.rand(T, k, generator=g, device=DEVICE) >= case["miss"]
    here[0, 0] = True                    # a pair to compute, however small the batch
    key = torch.where(here, ids, torch.full_like(ids, E)).flatten()
    perm = torch.argsort(key, stable=True).to(torch.int32)
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEVICE)
    offsets[1:] = counts.cumsum(0)
    return offsets, perm


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    dt, st = _torch(case["dtype"]), {"case": case}
    if case["op"] == "rows8":
        n, c, ld = case["rows"], case["cols"], case["cols"] + case["pad"]
        # rows of different sizes, as hidden states have them
        st["src"] = _randn(g, n, ld, dtype=dt) * _randn(g, n, 1).exp().to(dt)
        if own:
            st["codes"] = torch.empty(n, c, dtype=torch.int8, device=DEVICE)
            st["scale"] = torch.empty(n, -(-c // BLOCK), device=DEVICE)
            st["dst"] = torch.empty(n, c, dtype=dt, device=DEVICE)
        return st
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    P = T * k
    st["offsets"], st["perm"] = _sorted_pairs(g, case)
    st["x"] = _randn(g, T, H, dtype=dt)
    std = 0.9 / math.sqrt(H)             # gate and up of about one
    st["w_gate"] = _randn(g, E, I, H, dtype=dt, std=std)
    st["w_up"] = _randn(g, E, I, H, dtype=dt, std=std)
    st["w_down"] = _randn(g, E, H, I, dtype=dt, std=0.5 / math.sqrt(I))
    if case["op"] != "train":
        st["dy"] = _randn(g, P, H, dtype=dt, std=0.02)
    if case["op"] == "backward":
        kept = _randn(g, P, 2, I, dtype=dt, std=0.9)
        if case["keep"] == "int8":
            st["kept"], st["scale"] = _pack(kept)
        else:
            st["kept"], st["scale"] = kept, None
    if own:
        import sparse_moe_layer_route_amd as M
        st["dims"] = M.Dims(hidden=H, n_experts=E, top_k=k, inter=I, dtype=case["dtype"])
        st["ws"] = torch.empty(M.moe_expert_ffn_train_size(st["dims"], T), dtype=torch.uint8,
                               device=DEVICE)
        if case["op"] != "backward":
            int8 = case.get("keep") == "int8"
            st["y"] = torch.zeros(P, H, dtype=dt, device=DEVICE)
            st["kept"] = torch.zeros(P, 2, I, dtype=torch.int8 if int8 else dt, device=DEVICE)
            st["scale"] = torch.zeros(P, 2, -(-I // BLOCK), device=DEVICE) if int8 else None
        if case["op"] != "train":
            st["dx"] = torch.zeros(P, H, dtype=dt, device=DEVICE)
            st["dw"] = [torch.empty_like(st[n]) for n in ("w_gate", "w_up", "w_down")]
    else:
        # the plain form's batched products take the experts' rows side by side
        n = st["offsets"].diff().long()
        at = torch.arange(max(1, int(n.max())), device=DEVICE)
        st["rows"] = torch.where(at < n[:, None], at + st["offsets"][:-1, None].long(), P)
    return st


# -------------------------------------------------------------------- pass --
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import sparse_moe_layer_route_amd as M
    case = st["case"]
    op = case["op"]
    if op == "rows8":
        M.moe_rows_pack8(case["rows"], case["cols"], st["src"], st["codes"], st["scale"])
        M.moe_rows_unpack8(case["rows"], case["cols"], st["codes"], st["scale"], st["dst"])
        return st["dst"]
    if op != "backward":
        M.moe_expert_ffn_train(st["dims"], case["T"], st["x"], st, st["offsets"], st["perm"],
                               st["y"], st["kept"], st["ws"], kept_scale=st["scale"])
        if op == "train":
            return st["y"], st["kept"]
    M.moe_expert_ffn_backward(st["dims"], case["T"], st["x"], st, st["offsets"], st["perm"],
                              st["kept"], st["dy"], st["dx"], *st["dw"], st["ws"],
                              kept_scale=st["scale"])
    return ([st["y"]] if op == "step" else []) + [st["dx"]] + st["dw"]


def _pack(v):
    """8-bit values and scales of rows in blocks of BLOCK columns; which of two
    values is nearer is decided in 64 bits."""
    cols = v.shape[-1]
    blocks = -(-cols // BLOCK)
    f = torch.nn.functional.pad(v.float(), (0, blocks * BLOCK - cols))
    f = f.view(*v.shape[:-1], blocks, BLOCK)
    top = f.abs().amax(-1, keepdim=True)
    live, wide = top >= SMALL, top.double()
    codes = torch.where(live, (f.double() * 127 / wide).round(), 0.0).to(torch.int8)
    scale = torch.where(live, wide / 127, 0.0).float()
    return codes.view(*v.shape[:-1], -1)[..., :cols].contiguous(), scale[..., 0].contiguous()


def _unpack(codes, scale):
    cols = codes.shape[-1]
    return codes.float() * scale.repeat_interleave(BLOCK, dim=-1)[..., :cols]


def _side_by_side(rows, st):
    """[E, most rows, ...] of rows sorted by expert, zeros where one has fewer."""
    rows = torch.cat((rows.float(), torch.zeros_like(rows[:1], dtype=torch.float32)))
    return rows[st["rows"]]


def _back(padded, st, like):
    """Rows sorted by expert again; zeros behind the last."""
    out = torch.zeros(len(st["perm"]) + 1, *padded.shape[2:], dtype=like.dtype, device=DEVICE)
    out[st["rows"]] = padded.to(like.dtype)
    return out[:-1]


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rows8":
        return _unpack(*_pack(st["src"][:, :case["cols"]])).to(st["src"].dtype)
    x, out = st["x"], []
    xe = _side_by_side(x[st["perm"].long() // case["k"]], st)
    wd = st["w_down"].float()
    if op == "backward":
        kept = st["kept"] if st["scale"] is None else _unpack(st["kept"], st["scale"])
        gu = _side_by_side(kept, st)
    else:
        gu = torch.stack((torch.bmm(xe, st["w_gate"].float().transpose(1, 2)),
                          torch.bmm(xe, st["w_up"].float().transpose(1, 2))), dim=2)
        g, u = gu[:, :, 0], gu[:, :, 1]
        y = torch.bmm(g / (1 + (-g).exp()) * u, wd.transpose(1, 2))
        out.append(_back(y, st, x))
        if op == "train":
            return out[0], _back(gu, st, x)
        # what is kept in between
        gu = _unpack(*_pack(gu)) if case["keep"] == "int8" else gu.to(x.dtype).float()
    g, u = gu[:, :, 0], gu[:, :, 1]
    sig = 1 / (1 + (-g).exp())
    dy = _side_by_side(st["dy"], st)
    dh = torch.bmm(dy, wd)
    dg, du = dh * u * sig * (1 + g * (1 - sig)), dh * g * sig
    dx = torch.bmm(dg, st["w_gate"].float()) + torch.bmm(du, st["w_up"].float())
    out.append(_back(dx, st, x))
    out.append(torch.bmm(dg.transpose(1, 2), xe).to(x.dtype))
    out.append(torch.bmm(du.transpose(1, 2), xe).to(x.dtype))
    out.append(torch.bmm(dy.transpose(1, 2), g * sig * u).to(x.dtype))
    return out


# ------------------------------------------------------------- 64-bit truth --
def _exact8(v):
    """Values that v's 8-bit form stands for: steps of a block's largest / 127."""
    out = torch.zeros_like(v)
    for c in range(0, v.shape[-1], BLOCK):
        b = v[..., c:c + BLOCK]
        top = b.abs().amax(-1, keepdim=True)
        live = top >= SMALL
        q = torch.round(b * 127 / torch.where(live, top, torch.ones_like(top)))
        out[..., c:c + BLOCK] = torch.where(live, q * top / 127, torch.zeros_like(b))
    return out


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "rows8":
        return _exact8(st["src"][:, :case["cols"]].double())
    T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
    P, offsets, x = T * k, st["offsets"].tolist(), st["x"]
    y = torch.zeros(P, H, dtype=f64, device=DEVICE)
    kept = torch.zeros(P, 2, I, dtype=f64, device=DEVICE)
    dx = torch.zeros(P, H, dtype=f64, device=DEVICE)
    dw = [torch.zeros(st[n].shape, dtype=f64, device=DEVICE) for n in ("w_gate", "w_up", "w_down")]
    for e in range(E):
        r = slice(offsets[e], offsets[e + 1])
        if r.start == r.stop:
            continue
        xe = x[torch.div(st["perm"][r].long(), k, rounding_mode="floor")].double()
        wg, wu, wd = (st[n][e].double() for n in ("w_gate", "w_up", "w_down"))
        if op == "backward":
            g, u = st["kept"][r].double().unbind(1)
            if st["scale"] is not None:
                s = st["scale"][r].double()
                col = torch.arange(I, device=DEVICE) // BLOCK
                g, u = g * s[:, 0, col], u * s[:, 1, col]
        else:
            g, u = xe @ wg.T, xe @ wu.T
            y[r] = (g * torch.sigmoid(g) * u) @ wd.T
            kept[r, 0], kept[r, 1] = g, u
            if op == "train":
                continue
            if case["keep"] == "int8":
                g, u = _exact8(g), _exact8(u)
        s = torch.sigmoid(g)
        dy = st["dy"][r].double()
        dh = dy @ wd
        # the derivative of g s(g) is s + g s (1 - s)
        dg, du = dh * u * (s + g * s * (1 - s)), dh * (g * s)
        dx[r] = dg @ wg + du @ wu
        dw[0][e], dw[1][e], dw[2][e] = dg.T @ xe, du.T @ xe, dy.T @ (g * s * u)
    if op == "train":
        return y, kept
    return ([y] if op == "step" else []) + [dx] + dw
