"""CPU oracle of the routing by expert scores with a selection bias, and of its gradient.

TEST INFRASTRUCTURE ONLY, like moe_oracle (whose slot and row assignment it uses). fp64 numpy:
scores by the sigmoid or the softmax, selection by score + bias with expert groups, weights
from the scores alone; ties rank the lower index (stable sorts of the negated values).

Experts whose logit or bias is not finite are out of the selection; their score is 0. Among
what is left over (a token with fewer than k experts in it) the lower index comes first.
"""

from __future__ import annotations

import numpy as np

from oracle import moe_oracle as O


def scores(logits, kind: str) -> np.ndarray:
    l = np.asarray(logits, np.float64)
    ok = np.isfinite(l)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(ok, 1.0 / (1.0 + np.exp(-np.where(ok, l, 0.0))), 0.0)
    m = np.where(ok, l, -np.inf).max(axis=1, keepdims=True)
    e = np.where(ok, np.exp(np.where(ok, l, 0.0) - np.where(np.isfinite(m), m, 0.0)), 0.0)
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def select(logits, bias, cfg: dict, score: dict) -> np.ndarray:
    """Chosen experts [S, k], best first."""
    S, E, k = cfg["S"], cfg["E"], cfg["k"]
    sel = scores(logits, score["score"])
    out = ~np.isfinite(np.asarray(logits, np.float64))
    if bias is not None:
        b = np.asarray(bias, np.float64)
        out = out | ~np.isfinite(b)[None, :]
        sel = sel + np.where(np.isfinite(b), b, 0.0)[None, :]
    sel = np.where(out, -np.inf, sel)
    ng = int(cfg.get("n_expert_groups", 0) or 0)
    allowed = np.ones((S, E), bool)
    if ng > 1:
        size = E // ng
        best = -np.sort(-sel.reshape(S, ng, size), axis=2)
        gs = best[:, :, 0] + best[:, :, 1] if score["group_top"] == 2 and size > 1 else best[:, :, 0]
        kept = np.argsort(-gs, axis=1, kind="stable")[:, :cfg["topk_groups"]]
        in_group = np.zeros((S, ng), bool)
        np.put_along_axis(in_group, kept, True, axis=1)
        allowed = np.repeat(in_group, size, axis=1)
    # allowed experts first, by selection score, then index
    order = np.lexsort((np.broadcast_to(np.arange(E), (S, E)), -sel, ~allowed), axis=1)
    return order[:, :k].astype(np.int64)


def raw_weights(logits, ids, bias, score: dict) -> np.ndarray:
    """The weights [S, k] before any assignment is dropped. The renormalised sigmoids are formed
    from their logarithms, so that they are right where every sigmoid underflows."""
    l = np.take_along_axis(np.asarray(logits, np.float64), ids, axis=1)
    out = ~np.isfinite(l)
    if bias is not None:
        out |= ~np.isfinite(np.asarray(bias, np.float64))[ids]
    if not score["renorm"]:
        s = np.take_along_axis(scores(logits, score["score"]), ids, axis=1)
        return score["scale"] * np.where(out, 0.0, s)
    safe = np.where(out, 0.0, l)
    log_s = safe if score["score"] == "softmax" else np.minimum(safe, 0.0) - np.log1p(np.exp(-np.abs(safe)))
    log_s = np.where(out, -np.inf, log_s)
    m = log_s.max(axis=1, keepdims=True)
    w = np.exp(log_s - np.where(np.isfinite(m), m, 0.0))
    t = w.sum(axis=1, keepdims=True)
    return score["scale"] * np.divide(w, t, out=np.zeros_like(w), where=t > 0)


def normalised(logits, kind: str) -> np.ndarray:
    """s_e / sum s, the shares of the balance loss."""
    l = np.asarray(logits, np.float64)
    ok = np.isfinite(l)
    if kind == "softmax":
        return scores(l, kind)
    safe = np.where(ok, l, 0.0)
    log_s = np.where(ok, np.minimum(safe, 0.0) - np.log1p(np.exp(-np.abs(safe))), -np.inf)
    m = log_s.max(axis=1, keepdims=True)
    w = np.exp(log_s - np.where(np.isfinite(m), m, 0.0))
    t = w.sum(axis=1, keepdims=True)
    return np.divide(w, t, out=np.zeros_like(w), where=t > 0)


def losses(logits, counts_routed, cfg: dict, score: dict):
    S, G, E, k = cfg["S"], cfg["G"], cfg["E"], cfg["k"]
    q = normalised(logits, score["score"]).reshape(G, S // G, E).mean(axis=1)
    aux = float((E * (counts_routed / float(S // G * k) * q).sum(axis=1)).mean())
    l = np.asarray(logits, np.float64)
    l = np.where(np.isfinite(l), l, -np.inf)
    m = l.max(axis=1)
    any_ = np.isfinite(m)
    lse = np.where(any_, np.where(any_, m, 0.0) +
                   np.log(np.maximum(np.exp(l - np.where(any_, m, 0.0)[:, None]).sum(axis=1), 1e-300)), 0.0)
    return aux, float(np.mean(lse ** 2)), lse


def route(logits, bias, cfg: dict, score: dict, ids=None) -> dict:
    S, G, E, k = cfg["S"], cfg["G"], cfg["E"], cfg["k"]
    C = O.capacity(S, G, E, k, cfg["capacity_factor"])
    if ids is None:
        ids = select(logits, bias, cfg, score)
    w = raw_weights(logits, ids, bias, score)
    pos, reason, counts = O.assign_slots(ids, np.ones((S, k), bool), G, E, C)
    row, offsets, token_of, choice_of = O.compact_rows(ids, pos, G, E, counts)
    routed = np.zeros((G, E), np.int64)
    np.add.at(routed, (np.repeat(np.arange(S) // (S // G), k), ids.ravel()), 1)
    aux, z, _ = losses(logits, routed, cfg, score)
    gate = np.where(pos >= 0, w, 0.0)
    return dict(expert_id=ids, gate=gate, gate_raw=w, pos=pos, drop_reason=reason, counts=counts,
                counts_routed=routed, row=row, expert_offsets=offsets, token_of=token_of,
                w_perm=gate[token_of, choice_of], aux_loss=aux, z_loss=z)


def loss(logits, cfg: dict, score: dict, r: dict, dgate, aux_coef, z_coef) -> float:
    """The scalar whose gradient logit_grad is, the routing decisions of r held fixed."""
    w = raw_weights(logits, r["expert_id"], None, score)
    aux, z, _ = losses(logits, r["counts_routed"], cfg, score)
    return float((w * dgate * (r["pos"] >= 0)).sum() + aux_coef * aux + z_coef * z)


def logit_grad(logits, cfg: dict, score: dict, r: dict, dgate, aux_coef, z_coef) -> np.ndarray:
    """d loss / d logits [S, E]: Jacobians written out as matrices, token by token."""
    S, G, E, k = cfg["S"], cfg["G"], cfg["E"], cfg["k"]
    l = np.asarray(logits, np.float64)
    ids, keep = r["expert_id"], r["pos"] >= 0
    q = normalised(l, score["score"])
    _, _, lse = losses(l, r["counts_routed"], cfg, score)
    p = np.exp(l - lse[:, None])
    f = np.repeat(r["counts_routed"] / float(S // G * k), S // G, axis=0)
    one_minus = 1.0 / (1.0 + np.exp(l)) if score["score"] == "sigmoid" else np.ones_like(l)
    out = np.zeros((S, E))
    for t in range(S):
        d = np.where(keep[t], dgate[t], 0.0) * score["scale"]
        if score["renorm"]:
            w = r["gate_raw"][t] / score["scale"]
            jac = np.diag(w) - np.outer(w, w)           # d w_i / d log s_j
            out[t, ids[t]] += (d @ jac) * one_minus[t, ids[t]]
        elif score["score"] == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l[t, ids[t]]))
            out[t, ids[t]] += d * s * one_minus[t, ids[t]]
        else:
            full = np.zeros(E)
            full[ids[t]] = d
            out[t] += p[t] * (full - p[t] @ full)
        ds = f[t] @ (np.diag(q[t]) - np.outer(q[t], q[t]))
        out[t] += aux_coef * E / (G * (S // G)) * ds * one_minus[t]
        out[t] += z_coef * 2.0 / S * lse[t] * p[t]
    return out
