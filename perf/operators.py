"""The operators around the MoE layer, as cases to time and compare.

A Transformer block with a Mixture-of-Experts (or a dense) feed-forward half runs, besides
the expert GEMMs,

  route      expert scores (sigmoid or softmax) of the router logits, a per-expert bias that
             balances the load and takes part in the selection only, expert groups, top-k,
             renormalised and scaled weights, capacity slots and expert-contiguous rows
  route_bwd  the gradient of those weights (and of the two routing losses) to the logits
  norm       layer norm, with the residual addition in front of it
  norm_bwd   its gradients, the reductions of the weight's and the bias's among them
  linear     y = act(x W^T + b) + residual
  linear_bwd the gradients of x, W and b

``own = False`` computes them from elementary torch operations, ``own = True`` through this
package's entry points.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a serving step, 256 experts in 8 groups of which 4 are kept, top-8: latency
        dict(name="route_token", op="route", S=1, G=1, E=256, k=8, score="sigmoid", bias=1, ng=8, tg=4,
             gtop=2, renorm=1, scale=2.5, cf=0.0),
        # a training batch of the same router, dropless
        dict(name="route_train", op="route", S=16384, G=1, E=256, k=8, score="sigmoid", bias=1, ng=8,
             tg=4, gtop=2, renorm=1, scale=2.5, cf=0.0),
        # the largest batch here: 64 experts, top-2, softmax scores, capacity factor 1.25
        dict(name="route_capacity", op="route", S=65536, G=1, E=64, k=2, score="softmax", bias=1, ng=0,
             tg=0, gtop=1, renorm=0, scale=1.0, cf=1.25),
        # its backward at the training batch, with both losses
        dict(name="route_bwd", op="route_bwd", S=16384, G=1, E=256, k=8, score="sigmoid", bias=1, ng=8,
             tg=4, gtop=2, renorm=1, scale=2.5, cf=0.0),
        # one token before its layer: latency
        dict(name="norm_token", op="norm", T=1, M=4096, dtype="bf16", res=1, beta=1, pad=0),
        # the pre-norm of a batch of 65536 tokens with the residual sum written too
        dict(name="norm_batch", op="norm", T=65536, M=1024, dtype="bf16", res=1, beta=1, pad=0),
        # a training step's norm backward
        dict(name="norm_bwd", op="norm_bwd", T=16384, M=4096, dtype="bf16", res=1, beta=1, pad=0),
        # odd rows and columns, fp32
        dict(name="norm_bwd_odd", op="norm_bwd", T=4097, M=1003, dtype="f32", res=0, beta=1, pad=5),
        # one token through the first layer of a dense feed-forward: the weights' bytes
        dict(name="linear_token", op="linear", T=1, N=14336, K=4096, dtype="bf16", act="silu", bias=1,
             res=0, pre=0, pad=0),
        # the same layer over a training batch, the pre-activation kept for the backward
        dict(name="linear_batch", op="linear", T=8192, N=14336, K=4096, dtype="bf16", act="gelu", bias=1,
             res=0, pre=1, pad=0),
        # sizes that no tile or 16-byte row divides, with the residual in the epilogue
        dict(name="linear_odd", op="linear", T=777, N=1411, K=2049, dtype="bf16", act="none", bias=1,
             res=1, pre=0, pad=0),
        # a dense feed-forward layer's backward over a training batch
        dict(name="linear_bwd", op="linear_bwd", T=16384, N=4096, K=1024, dtype="bf16", act="gelu", bias=1,
             res=0, pre=1, pad=0),
    ]


def _logint(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "norm", "norm_bwd", "linear", "linear", "linear_bwd"])
    if op in ("route", "route_bwd"):
        k = rng.randint(1, 8)
        ng = rng.choice([0, 0, 2, 4, 8, 16, 5])
        gtop = rng.choice([1, 2])
        if ng:
            gsz = _logint(rng, 1, 256 // ng)
            tg = rng.randint(1, ng)
            E = ng * gsz
            k = min(k, tg * gsz)
        else:
            tg, E = 0, _logint(rng, k, 256)
        G = rng.choice([1, 1, 1, 2, 7, 16])
        S = max(1, _logint(rng, 1, min(65536, (1 << 22) // E)) // G) * G
        return dict(op=op, S=S, G=G, E=E, k=k, score=rng.choice(["sigmoid", "sigmoid", "softmax"]),
                    bias=rng.choice([0, 1, 1]), ng=ng, tg=tg, gtop=gtop, renorm=rng.choice([0, 1]),
                    scale=rng.choice([1.0, 2.5]), cf=rng.choice([0.0, 0.0, 1.0, 1.25]))
    if op in ("norm", "norm_bwd"):
        M = _logint(rng, 1, 16384)
        T = _logint(rng, 1, min(65536, (1 << 26) // M))
        if rng.random() < 0.5:
            M = (M + 63) // 64 * 64
        return dict(op=op, T=T, M=M, dtype=rng.choice(["bf16", "bf16", "f32"]), res=rng.choice([0, 1]),
                    beta=rng.choice([0, 1]), pad=rng.choice([0, 0, 8, 3]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    top = 1 << (37 if dtype == "bf16" else 33)
    N, K = _logint(rng, 1, 14336), _logint(rng, 1, 14336)
    if rng.random() < 0.5:
        N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
    T = _logint(rng, 1, max(1, min(16384, top // (N * K))))
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    return dict(op=op, T=T, N=N, K=K, dtype=dtype, act=act, bias=rng.choice([0, 1]),
                res=rng.choice([0, 1]) if op == "linear" else 0,
                pre=rng.choice([0, 1]) if op == "linear" else 1, pad=rng.choice([0, 0, 8, 3]))


# ------------------------------------------------------------------ inputs
def _randn(gen, *shape, dtype=torch.float32, pad=0, scale=1.0):
    """Standard normal values; pad > 0 gives rows that lie `pad` elements further apart."""
    if not pad:
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)
    full = torch.empty((*shape[:-1], shape[-1] + pad), device=DEV, dtype=dtype)
    view = full[..., :shape[-1]]
    view.copy_(torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale))
    return view


def _moe_cfg(case):
    """The MoE layer configuration that the routing calls take (M and H play no part)."""
    return dict(S=case["S"], G=case["G"], E=case["E"], M=64, H=64, k=case["k"],
                capacity_factor=case["cf"], random_routing=0, n_shared=0, H_shared=0, act="relu",
                dtype="bf16", n_expert_groups=case["ng"], topk_groups=case["tg"])


def _score_cfg(case):
    return dict(score=case["score"], group_top=case["gtop"], renorm=case["renorm"], scale=case["scale"])


def _capacity(case):
    if case["cf"] <= 0:
        return -1
    return math.ceil(float(np.float32(case["cf"])) * case["k"] * (case["S"] // case["G"]) / case["E"])


def _rows_max(case):
    C, sk = _capacity(case), case["S"] * case["k"]
    return sk if C < 0 else min(sk, case["G"] * case["E"] * C)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = dict(case=case)
    op = case["op"]
    if op in ("route", "route_bwd"):
        S, E, k = case["S"], case["E"], case["k"]
        # router logits: a common part per expert (a skewed load) and a token's own
        st["logits"] = _randn(gen, S, E) + 0.3 * _randn(gen, E)
        st["bias"] = 0.05 * _randn(gen, E) if case["bias"] else None
        if op == "route_bwd":
            r = _route_plain(case, st["logits"], st["bias"])
            st["fwd"] = r
            st["dgate"] = _randn(gen, S, k)
            st["dlogits"] = torch.empty(S, E, device=DEV)
            st["coef"] = (0.01, 0.001)
        if own:
            from top_gating_expert_gb300 import moe
            st["cfg"] = moe.make_config(_moe_cfg(case))
            st["out"] = moe.RouteOutputs.allocate(st["cfg"], DEV)
            st["score"] = _score_cfg(case)
            st["ws"] = moe.workspace(st["cfg"], 0, DEV)
            if op == "route_bwd":
                for name in ("expert_id", "gate", "pos", "drop_reason", "row", "counts", "counts_routed"):
                    getattr(st["out"], name).copy_(st["fwd"][name])
        return st
    dt = DT[case["dtype"]]
    if op in ("norm", "norm_bwd"):
        T, M, pad = case["T"], case["M"], case["pad"]
        # a residual stream: an offset and a scale of their own for each channel, a few large ones
        ch = torch.exp(0.5 * _randn(gen, M))
        off = 0.3 * _randn(gen, M)
        x = _randn(gen, T, M, pad=pad, dtype=dt)
        x.copy_(x.float() * ch + off)
        st["gamma"] = 1.0 + 0.2 * _randn(gen, M)
        st["beta"] = 0.1 * _randn(gen, M) if case["beta"] else None
        if op == "norm":
            st["x"] = x
            st["res"] = _randn(gen, T, M, pad=pad, dtype=dt) if case["res"] else None
            if own:
                st["y"] = torch.empty(T, M, device=DEV, dtype=dt)
                st["h"] = torch.empty(T, M, device=DEV, dtype=dt) if case["res"] else None
                st["mean"], st["rstd"] = torch.empty(2, T, device=DEV).unbind(0)
        else:
            st["h"] = x
            xf = x.float()
            st["mean"] = xf.mean(1)
            st["rstd"] = torch.rsqrt((xf - st["mean"][:, None]).square().mean(1) + EPS)
            st["dy"] = _randn(gen, T, M, dtype=dt)
            st["dh"] = _randn(gen, T, M, dtype=dt) if case["res"] else None
            if own:
                from top_gating_expert_gb300 import block
                st["ws"] = block.layer_norm_workspace(T, M, dt, DEV)
                st["dx"] = torch.empty(T, M, device=DEV, dtype=dt)
        return st
    T, N, K, pad = case["T"], case["N"], case["K"], case["pad"]
    st["x"] = _randn(gen, T, K, pad=pad, dtype=dt)
    st["W"] = _randn(gen, N, K, dtype=dt, scale=1.0 / math.sqrt(K))
    st["b"] = 0.1 * _randn(gen, N) if case["bias"] else None
    if op == "linear":
        st["res"] = _randn(gen, T, N, pad=pad, dtype=dt) if case["res"] else None
        if own:
            from top_gating_expert_gb300 import block
            st["ws"] = block.linear_workspace(T, N, K, dt, DEV)
            st["y"] = torch.empty(T, N, device=DEV, dtype=dt)
            st["pre"] = torch.empty(T, N, device=DEV, dtype=dt) if case["pre"] else None
    else:
        st["dy"] = _randn(gen, T, N, pad=pad, dtype=dt)
        st["pre"] = _randn(gen, T, N, dtype=dt) if case["act"] != "none" else None
        if own:
            from top_gating_expert_gb300 import block
            st["ws"] = block.linear_workspace(T, N, K, dt, DEV)
            st["dx"] = torch.empty(T, K, device=DEV, dtype=dt)
            st["dW"] = torch.empty(N, K, device=DEV, dtype=dt)
            st["db"] = torch.empty(N, device=DEV) if case["bias"] else None
    return st


# ------------------------------------------------------------------ plain forms
def _scores64(case, logits):
    """The experts' scores, in 64 bits: they decide which experts are chosen."""
    l = logits.double()
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_plain(case, logits, bias):
    S, G, E, k = case["S"], case["G"], case["E"], case["k"]
    Sg = S // G
    score = _scores64(case, logits)
    sel = score + bias.double() if bias is not None else score
    if case["ng"] > 1:
        ng = case["ng"]
        grouped = sel.reshape(S, ng, E // ng)
        n_best = min(case["gtop"], E // ng)
        gscore = grouped.sort(dim=2, descending=True).values[:, :, :n_best].sum(2)
        kept = gscore.sort(dim=1, descending=True, stable=True).indices[:, :case["tg"]]
        allowed = torch.zeros(S, ng, dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        sel = torch.where(allowed[:, :, None], grouped, -math.inf).reshape(S, E)
    ids = sel.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = w * case["scale"]
    # slots: per (group, expert) all first choices in token order, then all second ones, ...
    C = _capacity(case)
    t = torch.arange(S, device=DEV)
    queue = (t // Sg)[:, None] * E + ids                               # (group, expert)
    place = torch.arange(k, device=DEV)[None, :] * S + t[:, None]      # order inside a queue
    order = (queue * (k * S) + place).reshape(-1).argsort()
    size = torch.zeros(G * E, dtype=torch.int64, device=DEV)
    size.scatter_add_(0, queue.reshape(-1), torch.ones_like(order))
    start = size.cumsum(0) - size
    pos = torch.empty_like(order)
    pos[order] = torch.arange(S * k, device=DEV) - start[queue.reshape(-1)[order]]
    pos = pos.reshape(S, k)
    keep = pos < C if C >= 0 else torch.ones_like(pos, dtype=torch.bool)
    counts = (size.clamp(max=C) if C >= 0 else size).reshape(G, E)
    # rows: expert by expert, inside an expert group by group
    per = counts.t().reshape(-1)
    first = (per.cumsum(0) - per).reshape(E, G)
    row = first[ids, (t // Sg)[:, None]] + pos
    rows = int(_rows_max(case))
    token_of = torch.zeros(rows + 1, dtype=torch.int32, device=DEV)
    w_perm = torch.zeros(rows + 1, device=DEV)
    at = torch.where(keep, row, rows).reshape(-1)
    token_of[at] = t[:, None].expand(S, k).reshape(-1).int()
    w_perm[at] = w.float().reshape(-1)
    # losses: E sum_e f_e P_e with P the normalised scores' mean, and the mean logsumexp^2
    q = score / score.sum(1, keepdim=True)
    f = size.reshape(G, E).double() / (Sg * k)
    aux = (E * (f * q.reshape(G, Sg, E).mean(1)).sum(1)).mean()
    z = torch.logsumexp(logits.double(), 1).square().mean()
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.sum(0).cumsum(0)])
    return dict(expert_id=ids.int(), gate=torch.where(keep, w, 0.0).float(),
                pos=torch.where(keep, pos, -1).int(), drop_reason=(~keep).to(torch.uint8),
                row=torch.where(keep, row, -1).int(), counts=counts.int(),
                counts_routed=size.reshape(G, E).int(), expert_offsets=offsets.int(),
                token_of=token_of[:rows], w_perm=w_perm[:rows], aux_loss=aux.float().reshape(1),
                z_loss=z.float().reshape(1))


def _route_bwd_plain(case, st):
    S, G, E, k = case["S"], case["G"], case["E"], case["k"]
    Sg, (ca, cz) = S // G, st["coef"]
    ids = st["fwd"]["expert_id"].long()
    kept = st["fwd"]["row"] >= 0
    dw = torch.where(kept, st["dgate"], 0.0).double() * case["scale"]
    score = _scores64(case, st["logits"])
    # of the weights, to the scores
    s = score.gather(1, ids)
    if case["renorm"]:
        tot = s.sum(1, keepdim=True)
        ds = (dw - (dw * s / tot).sum(1, keepdim=True)) / tot
    else:
        ds = dw
    dscore = torch.zeros_like(score).scatter_(1, ids, ds)
    # of the balance loss, whose counts are constants, through the normalised scores
    f = st["fwd"]["counts_routed"].double() / (Sg * k)
    a = (ca * E / (G * Sg)) * f.repeat_interleave(Sg, dim=0)
    tot = score.sum(1, keepdim=True)
    q = score / tot
    dscore += (a - (a * q).sum(1, keepdim=True)) / tot
    if case["score"] == "sigmoid":
        dl = dscore * score * (1.0 - score)
    else:
        dl = score * (dscore - (dscore * score).sum(1, keepdim=True))
    l = st["logits"].double()
    lse = torch.logsumexp(l, 1, keepdim=True)
    dl += cz * 2.0 * lse / S * torch.exp(l - lse)
    return dl.float()


def _act_plain(name, v):
    if name == "relu":
        return v.clamp(min=0.0)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _act_grad_plain(name, v):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "gelu":
        return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) \
            + v * torch.exp(-0.5 * v * v) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        th = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * (1.0 + th) + 0.5 * v * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * v * v)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-v))
        return s * (1.0 + v * (1.0 - s))
    return torch.ones_like(v)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        return _route_plain(case, st["logits"], st["bias"])
    if op == "route_bwd":
        return _route_bwd_plain(case, st)
    dt = DT[case["dtype"]]
    if op == "norm":
        h = st["x"].float()
        if st["res"] is not None:
            h = h + st["res"].float()
        mean = h.mean(1)
        d = h - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(1) + EPS)
        y = d * rstd[:, None] * st["gamma"]
        if st["beta"] is not None:
            y = y + st["beta"]
        out = dict(y=y.to(dt), mean=mean, rstd=rstd)
        if st["res"] is not None:
            out["h"] = h.to(dt)
        return out
    if op == "norm_bwd":
        xh = (st["h"].float() - st["mean"][:, None]) * st["rstd"][:, None]
        dy = st["dy"].float()
        g = dy * st["gamma"]
        dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * st["rstd"][:, None]
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        out = dict(dx=dx.to(dt), dgamma=(dy * xh).sum(0))
        if st["beta"] is not None:
            out["dbeta"] = dy.sum(0)
        return out
    x, W = st["x"].float(), st["W"].float()
    if op == "linear":
        v = x @ W.t()
        if st["b"] is not None:
            v = v + st["b"]
        y = _act_plain(case["act"], v)
        if st["res"] is not None:
            y = y + st["res"].float()
        out = dict(y=y.to(dt))
        if case["pre"]:
            out["pre"] = v.to(dt)
        return out
    d = st["dy"].float()
    if st["pre"] is not None:
        d = d * _act_grad_plain(case["act"], st["pre"].float())
    out = dict(dx=(d @ W).to(dt), dW=(d.t() @ x).to(dt))
    if st["b"] is not None:
        out["db"] = d.sum(0)
    return out


# ------------------------------------------------------------------ the framework's calls
ROUTE_OUT = ("expert_id", "gate", "pos", "drop_reason", "row", "counts", "counts_routed",
             "expert_offsets", "token_of", "w_perm", "aux_loss", "z_loss")


def run(state):
    if not own:
        return _plain(state)
    from top_gating_expert_gb300 import block, moe
    st, case = state, state["case"]
    op = case["op"]
    if op == "route":
        moe.route_scored(st["cfg"], st["score"], st["logits"], st["bias"], st["out"], st["ws"])
        return {n: getattr(st["out"], n) for n in ROUTE_OUT}
    if op == "route_bwd":
        ca, cz = st["coef"]
        moe.route_scored_backward(st["cfg"], st["score"], st["logits"], st["out"], st["dgate"],
                                  st["dlogits"], aux_coef=ca, z_coef=cz)
        return st["dlogits"]
    if op == "norm":
        y, h, mean, rstd = block.layer_norm(st["x"], st["gamma"], st["beta"], eps=EPS, residual=st["res"],
                                            out=st["y"], h=st["h"], mean=st["mean"], rstd=st["rstd"])
        out = dict(y=y, mean=mean, rstd=rstd)
        if st["res"] is not None:
            out["h"] = h
        return out
    if op == "norm_bwd":
        dx, dgamma, dbeta = block.layer_norm_backward(
            st["dy"], st["h"], st["gamma"], st["mean"], st["rstd"], dh=st["dh"],
            need_beta=st["beta"] is not None, dx=st["dx"], ws=st["ws"])
        out = dict(dx=dx, dgamma=dgamma)
        if st["beta"] is not None:
            out["dbeta"] = dbeta
        return out
    if op == "linear":
        y, pre = block.linear(st["x"], st["W"], st["b"], act=case["act"], residual=st["res"],
                              save_pre=bool(case["pre"]), out=st["y"], pre=st["pre"], ws=st["ws"])
        out = dict(y=y)
        if case["pre"]:
            out["pre"] = pre
        return out
    dx, dW, db = block.linear_backward(st["dy"], st["x"], st["W"], act=case["act"], pre=st["pre"],
                                       need_bias=st["b"] is not None, dx=st["dx"], dW=st["dW"],
                                       dbias=st["db"], ws=st["ws"])
    out = dict(dx=dx, dW=dW)
    if st["b"] is not None:
        out["db"] = db
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("route", "route_bwd"):
        S, G, E, k = case["S"], case["G"], case["E"], case["k"]
        if op == "route":
            by = 4 * S * E + 4 * E * case["bias"] + S * k * (4 + 4 + 4 + 1 + 4) + 8 * G * E + 4 * (E + 1) \
                + 8 * _rows_max(case) + 8
            return dict(bytes=by, flops=6 * S * E)
        return dict(bytes=8 * S * E + S * k * (4 + 4 + 4) + 4 * G * E, flops=10 * S * E)
    eb = 2 if case["dtype"] == "bf16" else 4
    if op == "norm":
        T, M = case["T"], case["M"]
        n = 2 + 2 * case["res"]
        return dict(bytes=n * T * M * eb + 4 * M * (1 + case["beta"]) + 8 * T, flops=8 * T * M)
    if op == "norm_bwd":
        T, M = case["T"], case["M"]
        n = 3 + case["res"]
        return dict(bytes=n * T * M * eb + 4 * M * (2 + case["beta"]) + 8 * T, flops=14 * T * M)
    T, N, K = case["T"], case["N"], case["K"]
    if op == "linear":
        return dict(bytes=eb * (T * K + N * K + T * N * (1 + case["res"] + case["pre"])) + 4 * N * case["bias"],
                    flops=2 * T * N * K)
    n_pre = 0 if case["act"] == "none" else 1
    return dict(bytes=eb * (2 * T * K + 2 * N * K + T * N * (1 + n_pre)) + 4 * N * case["bias"],
                flops=4 * T * N * K)


# ------------------------------------------------------------------ 64-bit definitions
def _route_exact(case, logits, bias):
    """numpy, one token queue at a time; the scores and weights by logarithms."""
    S, G, E, k = case["S"], case["G"], case["E"], case["k"]
    Sg = S // G
    l = logits.double().cpu().numpy()
    mx = l.max(1, keepdims=True)
    lse = mx + np.log(np.exp(l - mx).sum(1, keepdims=True))
    if case["score"] == "sigmoid":
        score = 1.0 / (1.0 + np.exp(-l))
    else:
        score = np.exp(l - mx) / np.exp(l - mx).sum(1, keepdims=True)
    sel = score if bias is None else score + bias.double().cpu().numpy()[None, :]
    if case["ng"] > 1:
        ng, gsz = case["ng"], E // case["ng"]
        by_group = np.sort(sel.reshape(S, ng, gsz), axis=2)[:, :, ::-1]
        gs = by_group[:, :, 0].copy()
        if case["gtop"] == 2 and gsz > 1:
            gs += by_group[:, :, 1]
        rank = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1, kind="stable")
        sel = np.where(np.repeat(rank < case["tg"], gsz, axis=1), sel, -np.inf)
    ids = np.argsort(-sel, axis=1, kind="stable")[:, :k]
    s = np.take_along_axis(score, ids, 1)
    w = case["scale"] * (s / s.sum(1, keepdims=True) if case["renorm"] else s)
    C = _capacity(case)
    pos = np.full((S, k), -1, np.int64)
    fill = np.zeros((G, E), np.int64)
    routed = np.zeros((G, E), np.int64)
    for g in range(G):
        for j in range(k):
            col = ids[g * Sg:(g + 1) * Sg, j]
            for e in np.unique(col):
                at = np.nonzero(col == e)[0]
                slot = fill[g, e] + np.arange(at.size)
                fill[g, e] += at.size
                if C >= 0:
                    slot = np.where(slot < C, slot, -1)
                pos[g * Sg + at, j] = slot
    routed[:] = fill
    counts = np.minimum(fill, C) if C >= 0 else fill
    offsets = np.concatenate([[0], np.cumsum(counts.sum(0))])
    base = offsets[:-1][None, :] + np.cumsum(counts, axis=0) - counts
    keep = pos >= 0
    row = np.where(keep, base[np.arange(S)[:, None] // Sg, ids] + pos, -1)
    R = _rows_max(case)
    token_of, w_perm = np.zeros(R, np.int32), np.zeros(R)
    token_of[row[keep]] = np.broadcast_to(np.arange(S)[:, None], (S, k))[keep]
    w_perm[row[keep]] = w[keep]
    P = (score / score.sum(1, keepdims=True)).reshape(G, Sg, E).mean(1)
    aux = (E * (routed / (Sg * k) * P).sum(1)).mean()
    return dict(expert_id=ids.astype(np.int32), gate=np.where(keep, w, 0.0), pos=pos.astype(np.int32),
                drop_reason=(~keep).astype(np.uint8), row=row.astype(np.int32),
                counts=counts.astype(np.int32), counts_routed=routed.astype(np.int32),
                expert_offsets=offsets.astype(np.int32), token_of=token_of, w_perm=w_perm,
                aux_loss=np.array([aux]), z_loss=np.array([(lse ** 2).mean()]))


def _route_bwd_exact(case, st):
    """By differentiating the loss itself in 64 bits."""
    S, G, E, k = case["S"], case["G"], case["E"], case["k"]
    ca, cz = st["coef"]
    l = st["logits"].double().requires_grad_(True)
    ids = st["fwd"]["expert_id"].long()
    score = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    s = score.gather(1, ids)
    w = case["scale"] * (s / s.sum(1, keepdim=True) if case["renorm"] else s)
    kept = (st["fwd"]["row"] >= 0).double()
    P = (score / score.sum(1, keepdim=True)).reshape(G, S // G, E).mean(1)
    f = st["fwd"]["counts_routed"].double() / (S // G * k)
    loss = (w * kept * st["dgate"].double()).sum() + ca * (E * (f * P).sum(1)).mean() \
        + cz * torch.logsumexp(l, 1).square().mean()
    return torch.autograd.grad(loss, l)[0]


_ACT64 = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
          "silu": torch.nn.functional.silu}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _route_exact(case, st["logits"], st["bias"])
    if op == "route_bwd":
        return _route_bwd_exact(case, st)
    if op == "norm":
        h = st["x"].double() if st["res"] is None else st["x"].double() + st["res"].double()
        var, mean = torch.var_mean(h, dim=1, correction=0)
        rstd = (var + EPS) ** -0.5
        y = (h - mean[:, None]) * rstd[:, None] * st["gamma"].double()
        if st["beta"] is not None:
            y += st["beta"].double()
        out = dict(y=y, mean=mean, rstd=rstd)
        if st["res"] is not None:
            out["h"] = h
        return out
    if op == "norm_bwd":
        h, dy, gamma = st["h"].double(), st["dy"].double(), st["gamma"].double()
        mean, rstd = st["mean"].double()[:, None], st["rstd"].double()[:, None]
        M = h.shape[1]
        xh = (h - mean) * rstd
        s1 = (dy @ gamma)[:, None]
        s2 = ((dy * xh) @ gamma)[:, None]
        dx = rstd / M * (M * dy * gamma - s1 - xh * s2)
        if st["dh"] is not None:
            dx += st["dh"].double()
        out = dict(dx=dx, dgamma=torch.einsum("tm,tm->m", dy, xh))
        if st["beta"] is not None:
            out["dbeta"] = dy.sum(0)
        return out
    x, W = st["x"].double(), st["W"].double()
    if op == "linear":
        b = None if st["b"] is None else st["b"].double()
        v = torch.nn.functional.linear(x, W, b)
        y = _ACT64[case["act"]](v)
        if st["res"] is not None:
            y = y + st["res"].double()
        out = dict(y=y)
        if case["pre"]:
            out["pre"] = v
        return out
    d = st["dy"].double()
    if st["pre"] is not None:
        p = st["pre"].double().requires_grad_(True)
        d = torch.autograd.grad(_ACT64[case["act"]](p), p, d)[0]
    out = dict(dx=torch.mm(d, W), dW=torch.mm(d.t(), x))
    if st["b"] is not None:
        out["db"] = d.sum(0)
    return out
