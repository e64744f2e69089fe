"""Plain fp64 NumPy forms of the training operators: tokens sorted by expert
and back with the slot weights applied, their gradients, the router's
gradient, and distillation from a teacher's top logits.

Written from the formulas, slot by slot and class by class; shares no code
with the GPU path.  ``inv`` and teacher ids outside their range are skipped.
"""
from __future__ import annotations

import numpy as np


def _slots(inv, T, k):
    inv = np.asarray(inv).reshape(T, k)
    return inv, (inv >= 0) & (inv < T * k)


def dispatch(x, inv, k, out):
    """Rows of x at their sorted positions; `out` supplies the other rows."""
    T = len(x)
    inv, here = _slots(inv, T, k)
    out = np.array(out, copy=True)
    for t in range(T):
        for j in range(k):
            if here[t, j]:
                out[inv[t, j]] = x[t]
    return out


def undispatch(y_perm, inv, k, w=None, add=None):
    y = np.asarray(y_perm, dtype=np.float64)
    T = len(y) // k
    inv, here = _slots(inv, T, k)
    out = np.zeros((T, y.shape[1])) if add is None else np.array(add, dtype=np.float64)
    for t in range(T):
        for j in range(k):
            if here[t, j]:
                out[t] += (1.0 if w is None else float(w[t, j])) * y[inv[t, j]]
    return out


def undispatch_backward(dout, y_perm, inv, k, w, dy):
    """(dy_perm, dtopk_w); `dy` supplies the rows that no slot names."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y_perm, np.float64)
    T = len(dout)
    inv, here = _slots(inv, T, k)
    dy, dw = np.array(dy, dtype=np.float64), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            if here[t, j]:
                dy[inv[t, j]] = float(w[t, j]) * dout[t]
                dw[t, j] = dout[t] @ y[inv[t, j]]
    return dy, dw


def route_weights(logits, ids, renormalize):
    """The weight of each slot (0 for an id out of range): p_e, or p_e over
    the sum of the slots' p."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids = np.asarray(ids).reshape(T, -1)
    w = np.zeros(ids.shape)
    for t in range(T):
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not slots:
            continue
        if renormalize:
            e = np.array([l[t, ids[t, j]] for j in slots])
            e = np.exp(e - e.max())
            w[t, slots] = e / e.sum()
        else:
            e = np.exp(l[t] - l[t].max())
            w[t, slots] = (e / e.sum())[ids[t, slots]]
    return w


def route_dlogits(logits, ids, dtopk_w, renormalize, add=None):
    """Through each slot's row of the Jacobian d w_j / d l_v."""
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    ids = np.asarray(ids).reshape(T, -1)
    g = np.asarray(dtopk_w, np.float64).reshape(T, -1)
    w = route_weights(l, ids, renormalize)
    dl = np.zeros((T, E)) if add is None else np.array(add, dtype=np.float64)
    for t in range(T):
        slots = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if renormalize:
            q = np.zeros(E)
            for j in slots:
                q[ids[t, j]] += w[t, j]
        else:
            e = np.exp(l[t] - l[t].max())
            q = e / e.sum()
        for j in slots:
            jac = -w[t, j] * q
            jac[ids[t, j]] += w[t, j]
            dl[t] += g[t, j] * jac
    return dl


def router_linear_backward(dlogits, x, w_router, dx_add=None):
    """(dx, dW) of logits = x W^T."""
    dl = np.asarray(dlogits, np.float64)
    dx = dl @ np.asarray(w_router, np.float64)
    if dx_add is not None:
        dx = dx + np.asarray(dx_add, np.float64)
    return dx, dl.T @ np.asarray(x, np.float64)


def distill(student, ids, t_logits, temperature, t_lse=None, token_w=None, scale=1.0):
    """(loss [T], d loss / d student [T][V])."""
    s = np.asarray(student, np.float64)
    T, V = s.shape
    loss, grad = np.zeros(T), np.zeros((T, V))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        for t in range(T):
            c = scale * (1.0 if token_w is None else float(token_w[t]))
            ks = [k for k in range(len(ids[t])) if 0 <= ids[t][k] < V]
            u = np.array([float(t_logits[t][k]) for k in ks]) / temperature
            if c == 0.0 or (t_lse is None and (not ks or u.max() == -np.inf)):
                continue
            if t_lse is None:
                p = np.exp(u - u.max())
                logp = u - u.max() - np.log(p.sum())
            else:
                logp = u - float(t_lse[t])
            p = np.exp(logp)
            z = s[t] / temperature
            logq = z - z.max() - np.log(np.exp(z - z.max()).sum())
            kl, g = 0.0, np.zeros(V)
            for i, k in enumerate(ks):
                if p[i] > 0:
                    kl += p[i] * (logp[i] - logq[ids[t][k]])
                g[ids[t][k]] -= p[i]
            mass = p.sum()
            tail = np.ones(V, bool)
            tail[[ids[t][k] for k in ks]] = False
            if t_lse is not None and tail.any():
                pt = max(0.0, 1.0 - mass)
                lt = logq[tail]
                lqt = lt.max() + np.log(np.exp(lt - lt.max()).sum()) if lt.max() > -np.inf else -np.inf
                if pt > 0:
                    kl += pt * (np.log(pt) - lqt)
                    if lqt > -np.inf:
                        g[tail] -= pt * np.exp(lt - lqt)
                mass += pt
            g += mass * np.exp(logq)
            loss[t], grad[t] = c * kl, c / temperature * g
    return loss, grad
