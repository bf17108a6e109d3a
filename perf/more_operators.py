"""The operators that close a training step, as cases to time and compare.

A training step of a model made of this package's blocks runs, besides the blocks,

  xent       the model's head: logits x W^T over a large vocabulary, their logsumexp and each
             token's cross entropy (plus a z-loss), without keeping the logits
  xent_step  the same and its gradients: those of x and W for the mean loss
  norm       the global norm of all gradients, for clipping
  adamw      one AdamW step over all parameters at once, the two moments held in 32 or in 8 bits
  clip_step  norm, then adamw with the gradients clipped to a largest norm

``own = False`` computes them from elementary torch operations, ``own = True`` through this
package's entry points.
"""

from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100
BLOCK = 256  # elements that share a scale when the moments are held in 8 bits
M_LEVELS, V_LEVELS = 127.0 * 127.0, 255.0 * 255.0
TINY = 2.0 ** -100


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # scoring the last token of one sequence while serving: the head's weights are read once
        dict(name="xent_token", op="xent", T=1, V=32768, K=1024, dtype="bf16", z=0.0, pad=0, drop=0.0),
        # evaluating a batch: the losses alone
        dict(name="xent_eval", op="xent", T=8192, V=32768, K=1024, dtype="bf16", z=0.0, pad=0, drop=0.1),
        # the head of a training step, with z-loss; its gradients take several pieces of vocabulary
        dict(name="xent_train", op="xent_step", T=8192, V=65536, K=2048, dtype="bf16", z=1e-4, pad=0, drop=0.05),
        # sizes that no tile or 16-byte row divides, half of the tokens without a target
        dict(name="xent_odd", op="xent_step", T=1003, V=20011, K=1411, dtype="bf16", z=0.0, pad=3, drop=0.5),
        # a small fp32 model's head
        dict(name="xent_f32", op="xent_step", T=512, V=4099, K=256, dtype="f32", z=1e-4, pad=0, drop=0.1),
        # a small layer's gradients: latency
        dict(name="norm_small", op="norm", n=12, total=131072, dtype="f32", odd=0),
        # all gradients of a model of a quarter of a billion parameters, in many tensors
        dict(name="norm_large", op="norm", n=300, total=1 << 28, dtype="f32", odd=0),
        # the parameters of a small layer: latency
        dict(name="adamw_small", op="adamw", n=12, total=131072, dtype="f32", grad="f32", bits=32, copy=0, clip=0,
             seed=-1, odd=0),
        # the fp32 master weights of a bf16 model, the bf16 weights written beside them
        dict(name="adamw_master", op="adamw", n=40, total=1 << 28, dtype="f32", grad="f32", bits=32, copy=1, clip=0,
             seed=-1, odd=0),
        # the same weights with both moments in 8 bits, rounded at random, bf16 gradients
        dict(name="adamw_8bit", op="adamw", n=40, total=1 << 28, dtype="f32", grad="bf16", bits=8, copy=1, clip=1,
             seed=17, odd=0),
        # many small tensors on no 16-byte boundary, 8-bit moments rounded to the nearest
        dict(name="adamw_odd", op="adamw", n=200, total=1200007, dtype="f32", grad="f32", bits=8, copy=0, clip=0,
             seed=-1, odd=1),
        # clipping and the step of a mid-sized model, bf16 parameters without a master copy
        dict(name="clip_step", op="clip_step", n=120, total=1 << 24, dtype="bf16", grad="bf16", bits=32, copy=0, clip=1,
             seed=-1, odd=0),
    ]


def _logint(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["xent", "xent_step", "xent_step", "norm", "adamw", "adamw", "clip_step"])
    if op in ("xent", "xent_step"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        top = 1 << (39 if dtype == "bf16" else 32)
        V, K = _logint(rng, 2, 131072), _logint(rng, 1, 8192)
        if rng.random() < 0.6:
            V, K = (V + 63) // 64 * 64, (K + 63) // 64 * 64
        T = _logint(rng, 1, max(1, min(16384, top // (V * K))))
        return dict(op=op, T=T, V=V, K=K, dtype=dtype, z=rng.choice([0.0, 1e-4]), pad=rng.choice([0, 0, 8, 3]),
                    drop=rng.choice([0.0, 0.1, 0.5]))
    total = _logint(rng, 1, 1 << 27)
    n = min(total, _logint(rng, 1, 600))
    odd = rng.choice([0, 0, 1])
    if op == "norm":
        return dict(op=op, n=n, total=total, dtype=rng.choice(["f32", "bf16"]), odd=odd)
    dtype = rng.choice(["f32", "f32", "bf16"])
    bits = 32 if op == "clip_step" else rng.choice([32, 8])
    return dict(op=op, n=n, total=total, dtype=dtype, grad=rng.choice(["f32", "bf16"]), bits=bits,
                copy=rng.choice([0, 1]) if dtype == "f32" else 0, clip=1 if op == "clip_step" else rng.choice([0, 1]),
                seed=rng.choice([-1, 5]) if bits == 8 else -1, odd=odd)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, dtype=torch.float32, pad=0, scale=1.0):
    """Normal values; pad > 0 gives rows that lie `pad` elements further apart."""
    if not pad:
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)
    full = torch.empty((shape[0], shape[1] + pad), device=DEV, dtype=dtype)
    view = full[:, :shape[1]]
    view.copy_(torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(scale))
    return view


def _sizes(case):
    """Sizes of the case's n tensors: a few large ones (weight matrices) and many small ones."""
    n, total = case["n"], case["total"]
    w = [2.0 ** (-12.0 * ((7 * i) % n) / n) for i in range(n)]
    s = [max(1, int((total - n) * x / sum(w))) for x in w]
    s[0] += max(0, total - sum(s))
    return s


def _places(sizes):
    """Offsets of the tensors in a flat buffer, each on a block of 256 elements; its length last."""
    at = [0]
    for s in sizes:
        at.append(at[-1] + (s + BLOCK - 1) // BLOCK * BLOCK)
    return at


def _flat(gen, case, sizes, dtype, scale, lead):
    """A flat buffer of the tensors, each padded with zeros to whole blocks, and views of them.
    The buffer starts `lead` elements into its allocation."""
    at = _places(sizes)
    full = torch.zeros(at[-1] + 8, device=DEV, dtype=dtype)
    flat = full[lead:lead + at[-1]]
    flat.copy_(torch.randn(at[-1], generator=gen, device=DEV).mul_(scale))
    views = [flat[a:a + s] for a, s in zip(at, sizes)]
    for a, b, s in zip(at, at[1:], sizes):
        flat[a + s:b] = 0
    return flat, views


def _many(case, gen, st):
    sizes = _sizes(case)
    st["sizes"], odd = sizes, case["odd"]
    gdt = DT[case["grad"] if "grad" in case else case["dtype"]]
    st["g"], st["gs"] = _flat(gen, case, sizes, gdt, 1e-2, odd * 3)
    if case["op"] == "norm":
        return
    st["p"], st["ps"] = _flat(gen, case, sizes, DT[case["dtype"]], 0.05, odd)
    at = _places(sizes)
    st["wd"] = [0.1 if i % 2 == 0 else 0.0 for i in range(len(sizes))]  # matrices decay, norms and biases do not
    decay = torch.tensor(st["wd"], device=DEV, dtype=torch.float64)
    st["decay"] = (1.0 - LR * decay).float().repeat_interleave(
        torch.tensor([b - a for a, b in zip(at, at[1:])], device=DEV))
    # moments as after T0 steps with gradients of this size; each tensor has a scale of its own
    unit = torch.exp(_randn(gen, len(sizes))).repeat_interleave(
        torch.tensor([b - a for a, b in zip(at, at[1:])], device=DEV))
    real = torch.zeros(at[-1], device=DEV)
    for a, s in zip(at, sizes):
        real[a:a + s] = 1.0
    m = _randn(gen, at[-1]).mul_(2e-3).mul_(unit).mul_(real)
    v = _randn(gen, at[-1]).square_().mul_(1e-4).mul_(unit).mul_(unit).mul_(real)
    del unit, real
    st["clock"] = torch.tensor([float(T0), B1 ** T0, B2 ** T0], device=DEV, dtype=torch.float64)
    if case["bits"] == 8:
        st["m"], st["ms"] = _m_codes(m, 0.5)
        st["v"], st["vs"] = _v_codes(v.sqrt(), 0.5)
    else:
        st["m"], st["v"] = m, v
    if case["copy"]:
        st["copy"] = st["p"].bfloat16()
        st["copies"] = [st["copy"][a:a + s] for a, s in zip(at, sizes)]
    # the norm of the whole model's gradients: this process may hold a part of them
    st["norm"] = st["g"].double().square().sum().sqrt().mul(1.25).float().reshape(1)


LR, B1, B2, EPS, T0 = 3e-4, 0.9, 0.95, 1e-8, 200


def _max_norm(case):
    """A largest norm below the gradients' own (1e-2 an element), so that clipping takes place."""
    return 0.5 * 1e-2 * math.sqrt(case["total"])


def prepare(case, seed):
    gen = _gen(seed)
    st = dict(case=case, clock_host=T0)
    if case["op"] in ("xent", "xent_step"):
        T, V, K, pad, dt = case["T"], case["V"], case["K"], case["pad"], DT[case["dtype"]]
        st["x"] = _randn(gen, T, K, dtype=dt, pad=pad)
        st["W"] = _randn(gen, V, K, dtype=dt, pad=pad, scale=2.0 / math.sqrt(K))
        # frequent words have low numbers
        u = torch.rand(T, generator=gen, device=DEV, dtype=torch.float64)
        y = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp(0, V - 1)
        st["y"] = torch.where(torch.rand(T, generator=gen, device=DEV) < case["drop"], IGNORE, y)
        if own:
            from top_gating_expert_gb300 import train
            st["ws"] = train.linear_cross_entropy_workspace(T, V, K, dt, DEV, backward=case["op"] == "xent_step")
        return st
    _many(case, gen, st)
    if own:
        from top_gating_expert_gb300 import train
        st["ws"] = train.grad_norm_workspace(DEV)
        if case["op"] != "norm":
            st["opt"] = train.AdamW(st["ps"], lr=LR, betas=(B1, B2), eps=EPS, weight_decay=st["wd"], bits=case["bits"],
                                    seed=None if case["seed"] < 0 else case["seed"],
                                    copies=st["copies"] if case["copy"] else None,
                                    max_norm=_max_norm(case) if case["clip"] else None)
            st["opt"].m.copy_(st["m"])
            st["opt"].v.copy_(st["v"])
            st["opt"].clock.copy_(st["clock"])
            if case["bits"] == 8:
                st["opt"].m_scale.copy_(st["ms"])
                st["opt"].v_scale.copy_(st["vs"])
    return st


# ------------------------------------------------------------------ plain forms
def _xent_plain(st):
    case = st["case"]
    x, W, y = st["x"].float(), st["W"].float(), st["y"]
    z = case["z"]
    l = x @ W.t()
    top = l.amax(1, keepdim=True)
    lse = (l - top).exp().sum(1).log() + top[:, 0]
    keep = y != IGNORE
    at = torch.where(keep, y, 0)[:, None]
    loss = torch.where(keep, lse - l.gather(1, at)[:, 0] + z * lse * lse, 0.0)
    count = keep.sum()
    stats = torch.stack([loss.double().sum() / count.clamp(min=1), count.double()]).float()
    out = dict(loss=loss, lse=lse, stats=stats)
    if case["op"] == "xent":
        return out
    w = keep.float() / count.clamp(min=1).float()
    d = (l - lse[:, None]).exp() * (w * (1.0 + 2.0 * z * lse))[:, None]
    d.scatter_add_(1, at, -w[:, None])
    dt = DT[case["dtype"]]
    return dict(out, dx=(d @ W).to(dt), dW=(d.t() @ x).to(dt))


def _mix(h):
    """A 32-bit mix of whole numbers below 2^32."""
    h = h ^ (h >> 16)
    h = (h * 0x9E3779B1) & 0xFFFFFFFF
    h = h ^ (h >> 15)
    h = (h * 0x85157AF5) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _dither(case, n, step):
    """The two thresholds of every element, of (0, 1): 1/2, or from a hash of seed, step and place."""
    if case["seed"] < 0:
        return 0.5, 0.5
    key = _mix(torch.tensor((case["seed"] + 0x632BE5AB * step) & 0xFFFFFFFF, device=DEV))
    h = _mix(torch.arange(n, device=DEV) ^ key)  # fewer than 2^32 elements here
    return ((h & 0xFFFF).float() + 0.5) * 2.0 ** -16, ((h >> 16).float() + 0.5) * 2.0 ** -16


def _scaled(a, levels):
    """a >= 0 in units of its block's largest value, times levels; and that value."""
    top = a.reshape(-1, BLOCK).amax(1)
    top = torch.where(torch.isfinite(top), torch.where(top >= TINY, top, 0.0), math.nan)
    inv = torch.where(top == 0.0, 0.0, torch.full_like(top, levels) / top)
    return (a.reshape(-1, BLOCK) * inv[:, None]).reshape(-1), top


def _level(y, r, most):
    """The k with k^2 <= y < (k + 1)^2, or the next one where y lies beyond the fraction r of the way."""
    k = y.sqrt().floor()
    return (k + (y - k * k > r * (2.0 * k + 1.0)).float()).clamp(max=most)


def _m_codes(m, r):
    """m as signed 8-bit codes c of blocks of 256: m ~ sign(c) c^2 / 127^2 times the block's largest |m|."""
    y, top = _scaled(m.abs(), M_LEVELS)
    return (_level(y, r, 127.0) * m.sign()).nan_to_num(0.0).to(torch.int8), top


def _v_codes(u, r):
    """u = sqrt(v) as codes c of 0 .. 255: u ~ c^2 / 255^2 times the block's largest; only 0 goes to 0."""
    y, top = _scaled(u, V_LEVELS)
    c = torch.where(y > 0.0, _level(y, r, 255.0).clamp(min=1.0), 0.0)
    return c.nan_to_num(0.0).to(torch.uint8), top


def _moments(st):
    """m and v as 32-bit values."""
    if st["case"]["bits"] == 32:
        return st["m"], st["v"]
    cm, cv = st["m"].float().reshape(-1, BLOCK), st["v"].float().reshape(-1, BLOCK)
    u = cv * cv * (st["vs"] * (1.0 / V_LEVELS))[:, None]
    return (cm * cm.abs() * (st["ms"] * (1.0 / M_LEVELS))[:, None]).reshape(-1), (u * u).reshape(-1)


def _norm_plain(g):
    return g.double().square().sum().sqrt().float().reshape(1)


def _adamw_plain(st, norm):
    """Updates the state's tensors in place."""
    case = st["case"]
    step = st["clock_host"] = st["clock_host"] + 1
    g, p = st["g"].float(), st["p"].float()
    if case["clip"]:
        g = g * (torch.full_like(norm, _max_norm(case)) / (norm + 1e-6)).clamp(max=1.0)
    m, v = _moments(st)
    m = m * B1 + g * (1.0 - B1)
    v = v * B2 + g * g * (1.0 - B2)
    u = v.sqrt()
    p = p * st["decay"] - m / (u * (1.0 / math.sqrt(1.0 - B2 ** step)) + EPS) * (LR / (1.0 - B1 ** step))
    st["p"].copy_(p)
    if case["copy"]:
        st["copy"].copy_(p)
    if case["bits"] == 8:
        rm, rv = _dither(case, m.numel(), step)
        for name, x in zip(("m", "ms", "v", "vs"), _m_codes(m, rm) + _v_codes(u, rv)):
            st[name].copy_(x)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)


def _adamw_out(st, m, v):
    out = dict(p=st["p"], m=m, v=v)
    if st["case"]["copy"]:
        out["copy"] = st["copy"]
    return out


def _plain(st):
    op = st["case"]["op"]
    if op in ("xent", "xent_step"):
        return _xent_plain(st)
    if op == "norm":
        return _norm_plain(st["g"])
    norm = _norm_plain(st["g"]) if op == "clip_step" else st["norm"]
    _adamw_plain(st, norm)
    out = _adamw_out(st, *_moments(st))
    return dict(out, norm=norm) if op == "clip_step" else out


# ------------------------------------------------------------------ the framework's calls
def run(state):
    if not own:
        return _plain(state)
    from top_gating_expert_gb300 import train
    st, case = state, state["case"]
    op = case["op"]
    if op in ("xent", "xent_step"):
        loss, lse, stats = train.linear_cross_entropy(st["x"], st["W"], st["y"], ignore_index=IGNORE, z_coef=case["z"],
                                                      ws=st["ws"])
        out = dict(loss=loss, lse=lse, stats=stats)
        if op == "xent_step":
            out["dx"], out["dW"] = train.linear_cross_entropy_backward(
                st["x"], st["W"], st["y"], lse, stats=stats, ignore_index=IGNORE, z_coef=case["z"], ws=st["ws"])
        return out
    if op == "norm":
        return train.grad_norm(st["gs"], ws=st["ws"])
    norm = train.grad_norm(st["gs"], ws=st["ws"]) if op == "clip_step" else st["norm"]
    st["opt"].step(st["gs"], norm=norm if case["clip"] else None)
    out = _adamw_out(st, *st["opt"].moments())
    return dict(out, norm=norm) if op == "clip_step" else out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("xent", "xent_step"):
        T, V, K = case["T"], case["V"], case["K"]
        eb = 2 if case["dtype"] == "bf16" else 4
        by, fl = eb * (T + V) * K + 8 * T + 8 * T + 8, 2 * T * V * K
        if op == "xent_step":  # the logits are not kept: the gradients make them again
            by, fl = by + 2 * eb * (T + V) * K + 12 * T, fl + 6 * T * V * K
        return dict(bytes=by, flops=fl)
    n = sum(_sizes(case))
    gb = 2 if case.get("grad", case["dtype"]) == "bf16" else 4
    if op == "norm":
        return dict(bytes=n * gb + 4, flops=2 * n)
    pb = 2 if case["dtype"] == "bf16" else 4
    # 8-bit moments: read and written as codes, and given out as the values they stand for
    state = 16 if case["bits"] == 32 else 4 + 8
    return dict(bytes=n * (2 * pb + gb + state + 2 * case["copy"]) + (n * gb if op == "clip_step" else 0), flops=14 * n)


# ------------------------------------------------------------------ 64-bit definitions
def _xent_exact(st):
    case = st["case"]
    T, V, K, z = case["T"], case["V"], case["K"], case["z"]
    if T * V * K > 1.5e12:  # three products of this size in 64 bits take over 20 seconds
        return None
    x, W, y = st["x"].double(), st["W"].double(), st["y"]
    n = max(1, int((y != IGNORE).sum()))
    step = max(1, (1 << 28) // V)
    loss, lse = torch.zeros(T, device=DEV, dtype=torch.float64), torch.zeros(T, device=DEV, dtype=torch.float64)
    back = case["op"] == "xent_step"
    dx, dW = (torch.zeros_like(x), torch.zeros_like(W)) if back else (None, None)
    for a in range(0, T, step):
        r = slice(a, min(T, a + step))
        l = torch.nn.functional.linear(x[r], W)
        lse[r] = torch.logsumexp(l, 1)
        keep = y[r] != IGNORE
        i = torch.nonzero(keep)[:, 0]
        loss[r][i] = lse[r][i] - l[i, y[r][i]] + z * lse[r][i] ** 2
        if back:
            p = torch.softmax(l, 1)
            p *= (1 + 2 * z * lse[r])[:, None]
            p[i, y[r][i]] -= 1.0
            p[~keep] = 0.0
            p /= n
            dx[r] = torch.mm(p, W)
            dW += torch.mm(p.t(), x[r])
    out = dict(loss=loss, lse=lse, stats=torch.tensor([float(loss.sum()) / n, float((y != IGNORE).sum())],
                                                      dtype=torch.float64, device=DEV))
    return dict(out, dx=dx, dW=dW) if back else out


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("xent", "xent_step"):
        return _xent_exact(st)
    g = st["g"].double()
    own_norm = torch.linalg.vector_norm(g).reshape(1)
    if op == "norm":
        return own_norm
    norm = own_norm if op == "clip_step" else st["norm"].double()
    if case["clip"]:
        g = g * min(1.0, _max_norm(case) / (float(norm) + 1e-6))
    if case["bits"] == 8:
        c = st["m"].double().reshape(-1, BLOCK)
        m0 = (c.sign() * (c / 127) ** 2 * st["ms"].double()[:, None]).reshape(-1)
        v0 = ((st["v"].double().reshape(-1, BLOCK) / 255) ** 4 * st["vs"].double()[:, None] ** 2).reshape(-1)
    else:
        m0, v0 = st["m"].double(), st["v"].double()
    m, v = torch.lerp(g, m0, B1), torch.lerp(g * g, v0, B2)
    mh, vh = m / (1 - B1 ** (T0 + 1)), v / (1 - B2 ** (T0 + 1))
    at = _places(st["sizes"])
    p = st["p"].double()
    for a, b, wd in zip(at, at[1:], st["wd"]):
        p[a:b] *= 1 - LR * wd
    p -= LR * mh / (vh.sqrt() + EPS)
    out = dict(p=p, m=m, v=v)
    if case["bits"] == 8:  # a value next to the border of two codes has no one 64-bit answer
        out["m"] = out["v"] = None
    if case["copy"]:
        out["copy"] = p
    return dict(out, norm=norm) if op == "clip_step" else out
