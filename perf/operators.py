"""Measured cases of the MoE layer's training operators.

Tokens sorted by expert and back with the slot weights applied, and its
gradient (moe_dispatch, moe_undispatch, moe_undispatch_backward); the router's
gradient (moe_route_backward); distillation from a teacher's top logits with
its gradient (moe_distill_topk).

``own`` selects what ``run`` does: False computes each operator in elementary
torch operations in 32 bits, True calls the library.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
INTER = 512          # routed intermediate size named in Dims; these operators do not read it


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # eight decoding tokens of a DeepSeek-V2-Lite-shaped layer handed to a
        # caller's own experts: launch latency
        dict(name="dispatch_decode", op="dispatch", dtype="bf16", T=8, H=2048, E=64, k=6, miss=0.0),
        # a 4096-token Granite-shaped prefill or training batch
        dict(name="dispatch_prefill", op="dispatch", dtype="bf16", T=4096, H=1536, E=40, k=8,
             miss=0.0),
        # the library's own fp32 expert rows of a 256-token Qwen2-57B-shaped
        # decode batch brought back onto the shared experts' output
        dict(name="undispatch_f32_rows", op="undispatch", dtype="bf16", rows="f32", T=256, H=3584,
             E=64, k=8, miss=0.0, weighted=True, add=True),
        # the gradient of dispatch on a ragged training batch, a tenth of the
        # slots not computed exactly, onto a gradient that is there already
        dict(name="dispatch_grad_ragged", op="undispatch", dtype="bf16", rows="bf16", T=6007,
             H=2048, E=64, k=6, miss=0.1, weighted=False, add=True),
        # gradient of the weighted way back, Granite-shaped training batch
        dict(name="undispatch_grad_train", op="undispatch_backward", dtype="bf16", rows="bf16",
             T=4096, H=1536, E=40, k=8, miss=0.0),
        # the same on a small fp32 layer, odd batch
        dict(name="undispatch_grad_f32", op="undispatch_backward", dtype="f32", rows="f32", T=333,
             H=256, E=8, k=2, miss=0.25),
        # router gradient of a small fine-tuning batch, unnormalised weights
        dict(name="route_grad_small", op="route_backward", dtype="bf16", T=64, H=2048, E=64, k=6,
             renorm=False, aux=False, dx_add=False),
        # router gradient of a training batch with an auxiliary loss, the
        # input gradient added to the dispatch gradient
        dict(name="route_grad_train", op="route_backward", dtype="bf16", T=4096, H=1536, E=40,
             k=8, renorm=True, aux=True, dx_add=True),
        # the largest router batch
        dict(name="route_grad_large", op="route_backward", dtype="bf16", T=16384, H=3584, E=64,
             k=8, renorm=True, aux=False, dx_add=False),
        # prefetch router distilled from the router's top eight of 40 experts
        dict(name="distill_router", op="distill", dtype="f32", T=4096, V=40, K=8, tail=False,
             pad=False, masked=0.0, tau=1.0),
        # a student's logits over a vocabulary, teacher's 64 best and a tail
        # bucket, a tenth of the positions masked
        dict(name="distill_vocab", op="distill", dtype="bf16", T=2048, V=32000, K=64, tail=True,
             pad=False, masked=0.1, tau=2.0),
        # few rows over a long odd axis in padded fp32 rows
        dict(name="distill_few_rows", op="distill", dtype="f32", T=7, V=100003, K=32, tail=True,
             pad=True, masked=0.0, tau=1.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    limit = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["dispatch", "undispatch", "undispatch_backward", "route_backward",
                         "distill"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        if op == "distill":
            V = _log_int(rng, 2, 131072)
            case = dict(op=op, dtype=dtype, T=_log_int(rng, 1, 16384), V=V,
                        K=min(V, _log_int(rng, 1, 256)), tail=rng.random() < 0.5,
                        pad=rng.random() < 0.5, masked=rng.choice([0.0, 0.3]),
                        tau=rng.choice([0.7, 1.0, 3.0]))
        else:
            E = rng.randint(2, 64)
            case = dict(op=op, dtype=dtype, T=_log_int(rng, 1, 16384), H=64 * _log_int(rng, 1, 64),
                        E=E, k=rng.randint(1, min(8, E)))
            if op == "route_backward":
                case.update(renorm=rng.random() < 0.5, aux=rng.random() < 0.5,
                            dx_add=rng.random() < 0.5)
            else:
                case.update(miss=rng.choice([0.0, 0.2, 0.9]))
                if op != "dispatch":
                    case.update(rows="f32" if dtype == "f32" else rng.choice(["bf16", "f32"]))
                if op == "undispatch":
                    case.update(weighted=rng.random() < 0.7, add=rng.random() < 0.5)
        if work(case)["bytes"] <= limit:
            return case


def work(case):
    T, b = case["T"], _size(case["dtype"])
    if case["op"] == "distill":
        V, K = case["V"], case["K"]
        return {"bytes": T * (1.0 - case["masked"]) * (V * b + 8 * K) + T * (V * b + 4),
                "flops": 8.0 * T * V}
    H, E, k = case["H"], case["E"], case["k"]
    x, P = T * H * b, T * k
    if case["op"] == "route_backward":
        n = 2 * x + E * H * (b + 4) + 8 * T * E + 8 * P
        n += 4 * T * E * case["aux"] + x * case["dx_add"]
        return {"bytes": float(n), "flops": 4.0 * T * E * H}
    rows = P * (1.0 - case["miss"]) * H * _size(case.get("rows", case["dtype"]))
    if case["op"] == "dispatch":
        return {"bytes": x + rows + 4 * P, "flops": 0.0}
    if case["op"] == "undispatch":
        return {"bytes": x * (1 + case["add"]) + rows + 4 * P * (1 + case["weighted"]),
                "flops": 2.0 * P * H}
    return {"bytes": x + 2 * rows + 12 * P, "flops": 3.0 * P * H}


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _scale(case):
    """Mean over the positions, with the usual square of the temperature."""
    return case["tau"] ** 2 / case["T"]


def _torch(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


# ------------------------------------------------------------------ inputs --
def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEVICE) * std).to(dtype)


def _sorted_positions(g, case):
    """Slot -> row of the stable sort by expert, -1 for slots not computed."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = torch.topk(_randn(g, T, E), k, dim=1).indices
    here = torch.rand(T, k, generator=g, device=DEVICE) >= case["miss"]
    key = torch.where(here, ids, torch.full_like(ids, E)).flatten()
    order = torch.argsort(key, stable=True)
    inv = torch.empty(T * k, dtype=torch.int32, device=DEVICE)
    inv[order] = torch.arange(T * k, dtype=torch.int32, device=DEVICE)
    inv[~here.flatten()] = -1
    return inv


def _dims(case):
    import sparse_moe_layer_route_amd as M
    return M.Dims(hidden=case["H"], n_experts=case["E"], top_k=case["k"], inter=INTER,
                  renormalize=case.get("renorm", False), dtype=case["dtype"])


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op, T, dt = case["op"], case["T"], _torch(case["dtype"])
    st = {"case": case}
    if op == "distill":
        return _prepare_distill(st, g, case)
    H, E, k = case["H"], case["E"], case["k"]
    if own:
        st["dims"] = _dims(case)
    if op == "route_backward":
        st["x"] = _randn(g, T, H, dtype=dt)
        st["w"] = _randn(g, E, H, dtype=dt, std=0.02)
        st["logits"] = st["x"].float() @ st["w"].float().t()
        st["ids"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
        st["dtopk_w"] = _randn(g, T, k)
        st["aux"] = _randn(g, T, E, std=0.01) if case["aux"] else None
        st["dx_add"] = _randn(g, T, H, dtype=dt, std=0.05) if case["dx_add"] else None
        if own:
            import sparse_moe_layer_route_amd as M
            st["dlogits"] = torch.empty(T, E, device=DEVICE)
            st["dx"] = torch.empty(T, H, dtype=dt, device=DEVICE)
            st["dw"] = torch.empty(E, H, device=DEVICE)
            st["ws"] = torch.empty(M.moe_route_backward_size(st["dims"], T), dtype=torch.uint8,
                                   device=DEVICE)
        return st
    rt = _torch(case.get("rows", case["dtype"]))
    st["inv"] = _sorted_positions(g, case)
    if op == "dispatch":
        st["x"] = _randn(g, T, H, dtype=dt)
        if own:
            st["x_perm"] = torch.zeros(T * k, H, dtype=dt, device=DEVICE)
        return st
    st["y_perm"] = _randn(g, T * k, H, dtype=rt, std=0.3)
    weighted = op == "undispatch_backward" or case["weighted"]
    st["topk_w"] = torch.softmax(_randn(g, T, k), dim=1) if weighted else None
    if op == "undispatch":
        st["add"] = _randn(g, T, H, dtype=dt) if case["add"] else None
        if own:
            st["out"] = torch.empty(T, H, dtype=dt, device=DEVICE)
    else:
        st["dout"] = _randn(g, T, H, dtype=dt)
        if own:
            st["dy_perm"] = torch.zeros(T * k, H, dtype=rt, device=DEVICE)
            st["dtopk_w"] = torch.empty(T, k, device=DEVICE)
    return st


def _prepare_distill(st, g, case):
    T, V, K, dt = case["T"], case["V"], case["K"], _torch(case["dtype"])
    ld = -(-V // 64) * 64 if case["pad"] else V
    student = _randn(g, T, ld, std=2.0)
    teacher = student[:, :V] + _randn(g, T, V)
    top = torch.topk(teacher, K, dim=1)
    st["student"] = student.to(dt)
    st["ids"] = top.indices.to(torch.int32).contiguous()
    st["t_logits"] = top.values.contiguous()
    st["lse"] = torch.logsumexp(teacher / case["tau"], dim=1) if case["tail"] else None
    keep = torch.rand(T, generator=g, device=DEVICE) >= case["masked"]
    st["token_w"] = keep.float() if case["masked"] else None
    st["scale"] = _scale(case)
    if own:
        import sparse_moe_layer_route_amd as M
        st["loss"] = torch.empty(T, device=DEVICE)
        st["dstudent"] = torch.empty(T, ld, dtype=dt, device=DEVICE)
        st["ws"] = torch.empty(M.moe_distill_topk_size(T, V), dtype=torch.uint8, device=DEVICE)
    return st


# -------------------------------------------------------------------- pass --
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import sparse_moe_layer_route_amd as M
    case = st["case"]
    op, T = case["op"], case["T"]
    if op == "dispatch":
        M.moe_dispatch(st["dims"], T, st["x"], st["inv"], st["x_perm"])
        return st["x_perm"]
    if op == "undispatch":
        M.moe_undispatch(st["dims"], T, st["y_perm"], st["inv"], st["topk_w"], st["out"],
                         add=st["add"])
        return st["out"]
    if op == "undispatch_backward":
        M.moe_undispatch_backward(st["dims"], T, st["dout"], st["y_perm"], st["inv"],
                                  st["topk_w"], st["dy_perm"], st["dtopk_w"])
        return st["dy_perm"], st["dtopk_w"]
    if op == "route_backward":
        M.moe_route_backward(st["dims"], T, st["x"], st["w"], st["ids"], st["logits"],
                             st["dtopk_w"], st["dlogits"], st["dx"], st["dw"], st["ws"],
                             dlogits_add=st["aux"], dx_add=st["dx_add"])
        return st["dlogits"], st["dx"], st["dw"]
    M.moe_distill_topk(T, case["V"], case["K"], st["student"], st["ids"], st["t_logits"],
                       st["loss"], st["dstudent"], st["ws"], teacher_lse=st["lse"],
                       token_w=st["token_w"], temperature=case["tau"], scale=st["scale"])
    return st["loss"], st["dstudent"][:, :case["V"]]


def _run_plain(st):
    case = st["case"]
    op, T, dt = case["op"], case["T"], _torch(case["dtype"])
    if op == "distill":
        return _distill_plain(st)
    if op == "route_backward":
        return _route_plain(st)
    k, inv = case["k"], st["inv"]
    here = inv >= 0
    if op == "dispatch":
        out = torch.zeros(T * k, case["H"], dtype=dt, device=DEVICE)
        slot = here.nonzero()[:, 0]
        out[inv[slot].long()] = st["x"][slot // k]
        return out
    row = inv.clamp(min=0).long()
    if op == "undispatch":
        y = st["y_perm"][row].float().view(T, k, -1)
        w = here.view(T, k).float()
        if st["topk_w"] is not None:
            w = w * st["topk_w"]
        out = (w[:, :, None] * y).sum(1)
        if st["add"] is not None:
            out = out + st["add"].float()
        return out.to(dt)
    dout = st["dout"].float()
    y = st["y_perm"][row].float().view(T, k, -1)
    dw = torch.where(here.view(T, k), (dout[:, None, :] * y).sum(2),
                     torch.zeros((), device=DEVICE))
    dy = torch.zeros_like(st["y_perm"])
    slot = here.nonzero()[:, 0]
    grad = st["topk_w"].flatten()[slot, None] * dout[slot // k]
    dy[inv[slot].long()] = grad.to(dy.dtype)
    return dy, dw


def _route_plain(st):
    case, logits = st["case"], st["logits"]
    ids = st["ids"].long()
    if case["renorm"]:
        # the weights are a softmax over the chosen logits alone
        chosen = logits.gather(1, ids)
        e = (chosen - chosen.amax(1, keepdim=True)).exp()
        w = e / e.sum(1, keepdim=True)
        d = w * (st["dtopk_w"] - (w * st["dtopk_w"]).sum(1, keepdim=True))
        dl = torch.zeros_like(logits).scatter_add(1, ids, d)
    else:
        e = (logits - logits.amax(1, keepdim=True)).exp()
        p = e / e.sum(1, keepdim=True)
        grad = torch.zeros_like(logits).scatter_add(1, ids, st["dtopk_w"])
        dl = p * (grad - (p * grad).sum(1, keepdim=True))
    if st["aux"] is not None:
        dl = dl + st["aux"]
    dx = dl @ st["w"].float()
    if st["dx_add"] is not None:
        dx = dx + st["dx_add"].float()
    return dl, dx.to(st["x"].dtype), dl.t() @ st["x"].float()


def _distill_plain(st):
    """The vocabulary's sums and exponentials in 32 bits; the K teacher entries,
    whose differences from the student cancel, in 64."""
    case = st["case"]
    T, V, K, tau = case["T"], case["V"], case["K"], case["tau"]
    ids = st["ids"].long()
    z = st["student"][:, :V].float() / tau
    zk = st["student"][:, :V].gather(1, ids).double() / tau
    t = st["t_logits"].double() / tau
    if st["lse"] is None:
        e = (t - t.amax(1, keepdim=True)).exp()
        logp = t - t.amax(1, keepdim=True) - e.sum(1, keepdim=True).log()
    else:
        logp = t - st["lse"].double()[:, None]
    p = logp.exp()
    mass = p.sum(1, keepdim=True)
    # lse over the classes outside the teacher's K, then joined with the K
    mk = zk.amax(1, keepdim=True)
    lse_head = (zk - mk).exp().sum(1, keepdim=True).log() + mk
    if K < V:
        zt = z.scatter(1, ids, -math.inf)
        mt = zt.amax(1, keepdim=True)
        et = (zt - mt).exp()
        sum_t = et.sum(1, keepdim=True).double()
        lse_tail = sum_t.log() + mt.double()
        top = torch.maximum(lse_head, lse_tail)
        lse = ((lse_head - top).exp() + (lse_tail - top).exp()).log() + top
        qt = (lse_tail - lse).exp()
    else:
        lse = lse_head
    kl = (p * (logp - zk + lse)).sum(1)
    left = mass
    if K < V:
        factor = qt * mass
        if st["lse"] is not None:
            pt = (1.0 - mass).clamp(min=0.0)
            kl = kl + (pt * (pt.clamp(min=1e-300).log() - lse_tail + lse))[:, 0]
            factor, left = qt - pt, mass + pt
    c = torch.full((T,), st["scale"], dtype=torch.float64, device=DEVICE)
    if st["token_w"] is not None:
        c = c * st["token_w"]
    g = (c / tau)[:, None]
    grad = torch.empty_like(z) if K == V else et * (g * factor / sum_t).float()
    grad.scatter_(1, ids, (g * ((zk - lse).exp() * left - p)).float())
    return (c * kl).float(), grad.to(st["student"].dtype)


# ------------------------------------------------------------- 64-bit truth --
def exact(case, seed):
    st = prepare(case, seed)
    f = {n: (v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v)
         for n, v in st.items()}
    op, T = case["op"], case["T"]
    if op == "distill":
        return _distill_exact(case, f)
    if op == "route_backward":
        return _route_exact(case, f)
    H, k = case["H"], case["k"]
    inv = st["inv"].long().view(T, k)
    if op == "dispatch":
        out = torch.zeros(T * k, H, dtype=torch.float64, device=DEVICE)
        for j in range(k):
            t = (inv[:, j] >= 0).nonzero()[:, 0]
            out[inv[t, j]] = f["x"][t]
        return out
    if op == "undispatch":
        out = torch.zeros(T, H, dtype=torch.float64, device=DEVICE)
        if f["add"] is not None:
            out += f["add"]
        for j in range(k):
            t = (inv[:, j] >= 0).nonzero()[:, 0]
            rows = f["y_perm"][inv[t, j]]
            out[t] += rows if f["topk_w"] is None else f["topk_w"][t, j, None] * rows
        return out
    dy = torch.zeros(T * k, H, dtype=torch.float64, device=DEVICE)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEVICE)
    for j in range(k):
        t = (inv[:, j] >= 0).nonzero()[:, 0]
        dy[inv[t, j]] = f["topk_w"][t, j, None] * f["dout"][t]
        dw[t, j] = (f["dout"][t] * f["y_perm"][inv[t, j]]).sum(1)
    return dy, dw


def _route_exact(case, f):
    """Chain rule through the Jacobian of each slot's weight, slot by slot."""
    T, E, k = case["T"], case["E"], case["k"]
    ids = f["ids"].long()
    dl = torch.zeros(T, E, dtype=torch.float64, device=DEVICE)
    p = torch.softmax(f["logits"], dim=1)
    if case["renorm"]:
        member = torch.zeros(T, E, dtype=torch.float64, device=DEVICE)
        member.scatter_(1, ids, 1.0)
        p = p * member / (p * member).sum(1, keepdim=True)
    for j in range(k):
        own_p = p.gather(1, ids[:, j:j + 1])
        # d w_j / d l_v = w_j (delta_{v, e_j} - p_v)
        dl -= f["dtopk_w"][:, j:j + 1] * own_p * p
        dl.scatter_add_(1, ids[:, j:j + 1], f["dtopk_w"][:, j:j + 1] * own_p)
    if f["aux"] is not None:
        dl += f["aux"]
    dx = dl @ f["w"]
    if f["dx_add"] is not None:
        dx += f["dx_add"]
    return dl, dx, dl.t() @ f["x"]


def _distill_exact(case, f):
    """Head classes and, with a tail, one more class joined from the rest."""
    T, V, K, tau = case["T"], case["V"], case["K"], case["tau"]
    ids = f["ids"].long()
    z = f["student"][:, :V] / tau
    logq = torch.log_softmax(z, dim=1)
    t = f["t_logits"] / tau
    logp = torch.log_softmax(t, dim=1) if f["lse"] is None else t - f["lse"][:, None]
    p = logp.exp()
    kl = (p * (logp - logq.gather(1, ids))).sum(1)
    grad = logq.exp() * p.sum(1, keepdim=True)
    if f["lse"] is not None and K < V:
        head = torch.zeros(T, V, dtype=torch.bool, device=DEVICE).scatter_(1, ids, True)
        log_tail = logq.masked_fill(head, -math.inf)
        log_qt = torch.logsumexp(log_tail, dim=1)
        pt = (1.0 - p.sum(1)).clamp(min=0.0)
        kl = kl + torch.xlogy(pt, pt) - pt * log_qt
        grad = grad + pt[:, None] * (logq.exp() - (log_tail - log_qt[:, None]).exp())
    grad.scatter_add_(1, ids, -p)
    c = torch.full((T,), _scale(case), dtype=torch.float64, device=DEVICE)
    if f["token_w"] is not None:
        c = c * f["token_w"]
    return c * kl, grad * (c / tau)[:, None]
