"""AdamW over many tensors and the gradients' norm on the GPU: against the formula in 64 bits, the 8-bit
codes bit for bit against the formula in torch's own operations, over sizes, types, alignments, missing
gradients, many launches, clipping, streams and graphs.

Tolerances: each operation is off by u = 2^-24 relative, and so is a constant rounded to fp32. The clip
factor takes a sum and a quotient and its product with g one rounding more, g' is off by 3 u; then
(1 - b1) as a constant, its product and the sum: 6 u of m's terms. The square of g' is off by 7 u, with
(1 - b2), product and sum 10 u of v. The
step size * m / (sqrt(v) rs + eps): the error of m over the denominator, and 24 u of the step for v's
root, the scalars and the division; p: two more roundings of its terms, and half a step of its type."""

import math

import pytest
import torch

from block_util import U, assert_within, generator, half_step
from perf import more_operators as plain
from top_gating_expert_gb300 import train

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def tensors(sizes, dtype, lead, scale, seed):
    """Tensors that start `lead` elements into their allocations, with 9 guards behind each."""
    gen = generator(seed)
    out, guards = [], []
    for n in sizes:
        full = torch.full((n + lead + 9,), 3.0, device="cuda", dtype=dtype)
        full[lead:lead + n] = torch.randn(n, generator=gen, device="cuda") * scale
        out.append(full[lead:lead + n])
        guards.append((full[:lead], full[lead + n:]))
    return out, guards


def reference(p, g, m, v, t, lr, b1, b2, eps, wd, coef):
    """(p, m, v) in 64 bits and their tolerances, before p is rounded to its type."""
    g = g.double() * coef
    rm, rv = b1 * m.double() + (1 - b1) * g, b2 * v.double() + (1 - b2) * g * g
    em = 6 * U * ((b1 * m.double()).abs() + ((1 - b1) * g).abs()) + 1e-44
    ev = 10 * U * rv + 1e-44
    den = (rv / (1 - b2 ** t)).sqrt() + eps
    step = lr * rm / (1 - b1 ** t) / den
    rp = p.double() * (1 - lr * wd) - step
    ep = lr / (1 - b1 ** t) * em / den + 24 * U * step.abs() + 4 * U * (p.double().abs() + step.abs())
    ep = ep + step.abs() * (ev.sqrt() if eps == 0 else torch.zeros_like(ev))
    return (rp, rm, rv), (ep, em, ev)


def flat(opt, buf, i):
    return buf[opt.first[i]:opt.first[i] + opt.params[i].numel()]


SIZES = [[1], [5, 256, 257], [4096, 3, 2048, 2049, 1, 100000], [7] * 40, [1031] * 130, [64 * 1024 + 5] * 5 + [2] * 600]


@pytest.mark.parametrize("pt,gt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("lead", [0, 1])
def test_steps(native_lib, pt, gt, sizes, lead):
    """Three steps in 32 bits, copies for fp32, clipping on, weight decay for every second tensor."""
    ps, guards = tensors(sizes, DT[pt], lead, 0.5, 1)
    wd = [0.1 if i % 2 == 0 else 0.0 for i in range(len(sizes))]
    copies = cguards = None
    if pt == "f32":
        copies, cguards = tensors(sizes, torch.bfloat16, lead, 1.0, 2)
    lr, betas, eps = 1e-2, (0.9, 0.99), 1e-8
    opt = train.AdamW(ps, lr=lr, betas=betas, eps=eps, weight_decay=wd, copies=copies, max_norm=0.5)
    for t in range(1, 4):
        gs, _ = tensors(sizes, DT[gt], lead, 10.0 ** -t, 10 + t)
        old = [p.clone() for p in ps]
        om, ov = opt.m.clone(), opt.v.clone()
        norm = train.grad_norm(gs)
        total = math.sqrt(sum(g.double().square().sum().item() for g in gs))
        assert abs(norm.item() - total) <= 40 * U * total
        opt.step(gs, norm=norm)
        coef = min(1.0, 0.5 / (norm.item() + 1e-6))
        for i in range(len(sizes)) if len(sizes) < 50 else list(range(4)) + list(range(len(sizes) - 4, len(sizes))):
            m0, v0 = flat(opt, om, i), flat(opt, ov, i)
            ref, tol = reference(old[i], gs[i], m0, v0, t, lr, *betas, eps, wd[i], coef)
            assert_within(flat(opt, opt.m, i), ref[1], tol[1], f"m {i}")
            assert_within(flat(opt, opt.v, i), ref[2], tol[2], f"v {i}")
            tp = tol[0] + half_step(DT[pt]) * (ref[0].abs() + tol[0])
            assert_within(ps[i], ref[0], tp, f"p {i}")
            if copies:
                assert torch.equal(copies[i], ps[i].bfloat16())
    for a, b in guards + (cguards or []):
        assert (a == 3).all() and (b == 3).all()
    assert opt.clock[0].item() == 3 and abs(opt.clock[2].item() - betas[1] ** 3) < 1e-14
    used = torch.zeros(opt.m.numel(), dtype=torch.bool, device="cuda")
    for i, n in enumerate(sizes):
        used[opt.first[i]:opt.first[i] + n] = True
    assert (opt.m[~used] == 0).all() and (opt.v[~used] == 0).all()


def codes_case(seed, gt, clip):
    return dict(op="adamw", n=9, total=70001, dtype="f32", grad=gt, bits=8, copy=1, clip=clip, seed=seed, odd=seed % 2)


@pytest.mark.parametrize("seed", [-1, 5, 12])
@pytest.mark.parametrize("gt,clip", [("f32", 0), ("bf16", 1)])
def test_codes_bit_for_bit(native_lib, seed, gt, clip):
    """Four steps in 8 bits: codes, scales and the moments they stand for are those of the formula in
    separately rounded operations; p within its tolerance."""
    case = codes_case(seed, gt, clip)
    old = plain.own
    try:
        plain.own = True
        own = plain.prepare(case, 3)
        plain.own = False
        ref = plain.prepare(case, 3)
        for _ in range(4):
            plain.own = True
            a = plain.run(own)
            plain.own = False
            b = plain.run(ref)
            opt = own["opt"]
            assert torch.equal(opt.m, ref["m"]) and torch.equal(opt.v, ref["v"])
            assert torch.equal(opt.m_scale, ref["ms"]) and torch.equal(opt.v_scale, ref["vs"])
            assert torch.equal(a["m"], b["m"]) and torch.equal(a["v"], b["v"])
            assert (a["p"] - b["p"]).abs().max().item() <= 32 * U * (b["p"].abs().max().item() + 1)
    finally:
        plain.own = old


@pytest.mark.parametrize("sizes", [[1], [255, 256, 257, 3], [5000, 40000]])
@pytest.mark.parametrize("lead", [0, 3])
def test_codes_are_near(native_lib, sizes, lead):
    """Nearest codes stand for values at most half a gap off, random ones at most a gap; zero moments stay 0,
    no sqrt(v) above 0 becomes 0."""
    for seed, share in ((None, 0.5), (3, 1.0)):
        ps, _ = tensors(sizes, torch.float32, lead, 0.5, 1)
        gs, _ = tensors(sizes, torch.float32, lead, 1e-3, 2)
        for g in gs:
            g[::7] = 0.0
            g[1::5] *= 1e-4
        opt = train.AdamW(ps, bits=8, seed=seed)
        opt.step(gs)
        m, v = opt.moments()
        for i, g in enumerate(gs):
            for got, want, levels in ((flat(opt, m, i), 0.1 * g.double(), 127.0), (flat(opt, v, i).sqrt(),
                                                                                   (1e-3 * g.double() ** 2).sqrt(), 255.0)):
                pad = torch.zeros((want.numel() + 255) // 256 * 256, dtype=torch.float64, device="cuda")
                pad[:want.numel()] = want.abs()
                top = pad.reshape(-1, 256).amax(1).repeat_interleave(256)[:want.numel()]
                k = (want.abs() / top.clamp_min(1e-300) * levels ** 2).sqrt().floor()
                gap = (2 * k + 1) / levels ** 2 * top
                low = top / levels ** 2 if levels == 255.0 else 0.0  # code 1 in place of 0
                tol = torch.maximum(share * gap, torch.as_tensor(low, device="cuda").double()) * (1 + 1e-3) + 8 * U * top
                assert_within(got.double(), want, tol, f"{i} {levels}")
                assert torch.equal(got == 0, want == 0) if levels == 255.0 else (got[want == 0] == 0).all()


def test_random_codes_keep_the_mean(native_lib):
    """Over many seeds the value that a random code stands for is the moment itself: within 5 standard
    errors of the mean (a gap times a half is the largest deviation), nearest codes are not."""
    n, seeds = 256, 400
    g = torch.linspace(0.02, 1.0, n, device="cuda")
    m = torch.zeros(n, dtype=torch.float64, device="cuda")
    u = torch.zeros(n, dtype=torch.float64, device="cuda")
    for s in range(seeds):
        opt = train.AdamW([torch.zeros(n, device="cuda")], bits=8, seed=s)
        opt.step([g])
        a, b = opt.moments()
        m += a.double() / seeds
        u += b.double().sqrt() / seeds
    for got, want, levels in ((m, 0.1 * g.double(), 127.0), (u, 1e-3 ** 0.5 * g.double(), 255.0)):
        gap = (2 * (want / want[-1]).sqrt() * levels + 3) / levels ** 2 * want[-1]
        assert ((got - want).abs() <= 5 * 0.5 * gap / seeds ** 0.5 + 16 * U * want[-1]).all()


def test_codes_at_the_top(native_lib):
    """Blocks whose largest element has the highest threshold (65535.5 / 65536): its y may come out a rounding below
    the highest square, and its code is then the one below 255 or 127."""
    n, seed = 1 << 24, 17
    rm, rv = plain._dither(dict(seed=seed), n, 1)
    gen = generator(3)
    for r in (rm, rv):
        g = torch.randn(n, generator=gen, device="cuda") * 1e-2
        at = (r > 0.99999).nonzero()[:, 0]
        assert at.numel() > 100
        g[at] = 0.2 + 0.1 * torch.rand(at.numel(), generator=gen, device="cuda")
        opt = train.AdamW([torch.zeros(n, device="cuda")], bits=8, seed=seed, betas=(0.9, 0.95))
        opt.step([g])
        want = plain._m_codes(g * (1.0 - 0.9), rm) + plain._v_codes((g * g * (1.0 - 0.95)).sqrt(), rv)
        for got, w in zip((opt.m, opt.m_scale, opt.v, opt.v_scale), want):
            assert torch.equal(got, w)
        # met for v, where one rounding below 255^2 is 2^-8 of a gap of 509, more than 2^-17 of it; one below 127^2 is
        # 2^-10 of 253, less
        assert r is rm or (opt.v[at] == 254).any()


def test_hash_is_spread(native_lib):
    """The two thresholds of neighbouring elements and successive steps: mean 1/2 and no correlation
    (within 5 standard errors of 2^18 draws)."""
    n = 1 << 18
    case = dict(seed=5)
    a, b = plain._dither(case, n, 1)
    c, d = plain._dither(case, n, 2)
    se = 5 / math.sqrt(n)
    z = lambda r: (r.double() - 0.5) * math.sqrt(12.0)
    for r in (a, b, c, d):
        assert abs(z(r).mean()) < se and r.min() > 0 and r.max() < 1
        assert abs((z(r)[1:] * z(r)[:-1]).mean()) < se and abs((z(r)[2:] * z(r)[:-2]).mean()) < se
    for r, s in ((a, b), (a, c), (b, d), (a, d)):
        assert abs((z(r) * z(s)).mean()) < se


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients(native_lib, bits):
    """NaN and infinite gradients reach their own element (32 bits) or block (8 bits) alone."""
    n = 1024
    p, g = torch.ones(n, device="cuda"), torch.full((n,), 0.1, device="cuda")
    g[300], g[700] = float("nan"), float("inf")
    opt = train.AdamW([p], bits=bits, weight_decay=0.0)
    opt.step([g])
    bad = torch.zeros(n, dtype=torch.bool, device="cuda")
    bad[[300, 700]] = True
    assert torch.equal(~torch.isfinite(p), bad)
    m, v = opt.moments()
    if bits == 8:
        bad[256:512] = bad[512:768] = True
    assert torch.equal(~torch.isfinite(m), bad) and torch.equal(~torch.isfinite(v), bad)


@pytest.mark.parametrize("bits", [32, 8])
def test_tiny_and_zero_gradients(native_lib, bits):
    """Gradients of 0 move p by the decay alone and stay 0; denormal ones give no NaN."""
    p, g = torch.ones(700, device="cuda"), torch.zeros(700, device="cuda")
    opt = train.AdamW([p], lr=0.1, weight_decay=0.5, bits=bits)
    opt.step([g])
    assert torch.allclose(p, torch.full_like(p, 0.95), rtol=4 * U, atol=0)
    assert all((x == 0).all() for x in opt.moments())
    for tiny in (1e-42, 1e-36, 1e-30, 1e-22):
        g.fill_(tiny)
        opt.step([g])
        assert torch.isfinite(p).all() and all(torch.isfinite(x).all() for x in opt.moments())
    opt = train.AdamW([p], bits=bits, eps=0.0)
    opt.step([torch.full((700,), 1e-3, device="cuda")])
    assert torch.isfinite(p).all()


@pytest.mark.parametrize("seed", [None, 7])
@pytest.mark.parametrize("scale", [1e-21, 1e-18, 1e-15, 1e-8, 1.0, 1e8, 1e14, 1e16, 1e18])
def test_codes_at_every_magnitude(native_lib, scale, seed):
    """Codes and scales bit for bit, and steps of the right size without eps, for gradients whose squares are
    denormal, ordinary and near fp32's end; some 10^-6 of the others."""
    n = 2048
    g = torch.randn(n, generator=generator(1), device="cuda") * scale
    g[::9] *= 1e-6
    g[::50] = 0.0
    p = torch.zeros(n, device="cuda")
    opt = train.AdamW([p], lr=1.0, bits=8, seed=seed, eps=0.0, weight_decay=0.0, betas=(0.9, 0.95))
    opt.step([g])
    m, v = g * (1.0 - 0.9), g * g * (1.0 - 0.95)
    rm, rv = plain._dither(dict(seed=-1 if seed is None else seed), n, 1)
    for got, want in zip((opt.m, opt.m_scale, opt.v, opt.v_scale), plain._m_codes(m, rm) + plain._v_codes(v.sqrt(), rv)):
        assert torch.equal(got, want)
    some = (g != 0) & (v > 1e-37)
    assert torch.isnan(p[g == 0]).all()  # 0 / 0 without eps
    ref = -(m.double() / 0.1) / (v.double() / 0.05).sqrt()
    assert ((p.double() - ref).abs() <= 64 * U)[some].all()
    assert torch.isfinite(p[(g != 0) & (v > 0)]).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_missing_gradients_and_lr(native_lib, bits):
    """A parameter without a gradient, its moments and its copy are left alone; lr by number, by call and
    from the device give the same step."""
    sizes = [300, 4000, 5]
    runs = []
    for lr in ("own", "call", "device"):
        ps, _ = tensors(sizes, torch.float32, 0, 1.0, 4)
        gs, _ = tensors(sizes, torch.float32, 0, 1.0, 5)
        copies = [torch.zeros(k, dtype=torch.bfloat16, device="cuda") for k in sizes]
        opt = train.AdamW(ps, lr=2.0 ** -6 if lr == "own" else 5.0, bits=bits, weight_decay=0.0, copies=copies)
        how = dict(own=None, call=2.0 ** -6, device=torch.full((1,), 2.0 ** -6, device="cuda"))[lr]
        before = ps[1].clone()
        opt.step([gs[0], None, gs[2]], lr=how)
        assert torch.equal(ps[1], before) and (copies[1] == 0).all()
        assert (flat(opt, opt.m, 1) == 0).all() and (flat(opt, opt.v, 1) == 0).all()
        opt.step(gs, lr=how)
        runs.append([*ps, opt.m, opt.v, opt.clock])
        assert opt.clock[0].item() == 2
        opt.step([None] * 3, lr=how)
        assert opt.clock[0].item() == 3
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_parameters_that_move(native_lib):
    """A parameter's memory replaced between steps: the new memory is updated."""
    p = torch.ones(600, device="cuda")
    opt = train.AdamW([p], lr=0.1)
    g = torch.ones(600, device="cuda")
    opt.step([g])
    first = p.clone()
    other = torch.full((600,), 2.0, device="cuda")
    p.set_(other)
    opt.step([g])
    assert (other < 2.0).all() and (first < 1.0).all()
    p.set_(torch.ones(500, device="cuda"))
    with pytest.raises(ValueError):
        opt.step([g])


@pytest.mark.parametrize("bits,seed", [(32, None), (8, None), (8, 9)])
def test_graph_and_streams(native_lib, bits, seed):
    """Replays of a captured clip and step count on: the same bits as eager steps, and as steps on another
    stream."""
    sizes = [5000, 77, 1]
    def run(mode):
        ps, _ = tensors(sizes, torch.float32, 0, 1.0, 4)
        gs, _ = tensors(sizes, torch.float32, 0, 0.0, 5)
        opt = train.AdamW(ps, lr=1e-2, bits=bits, seed=seed, max_norm=1.0)
        ws = train.grad_norm_workspace()
        lr = torch.zeros(1, device="cuda")
        stream = torch.cuda.Stream() if mode != "eager" else None
        one = lambda: opt.step(gs, lr=lr, norm=train.grad_norm(gs, ws=ws))
        graph = None
        if mode == "graph":
            torch.cuda.synchronize()
            keep = [t.clone() for t in (*ps, opt.m, opt.v, opt.clock)] + \
                ([] if bits == 32 else [opt.m_scale.clone(), opt.v_scale.clone()])
            with torch.cuda.stream(stream):
                one()
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                one()
            for t, k in zip((*ps, opt.m, opt.v, opt.clock) + (() if bits == 32 else (opt.m_scale, opt.v_scale)), keep):
                t.copy_(k)
        for t in range(5):
            for i, g in enumerate(gs):
                g.copy_(torch.randn(g.shape, generator=generator(100 * t + i), device="cuda"))
            lr.fill_(1e-2 / (t + 1))
            if graph:
                graph.replay()
            elif stream:
                stream.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(stream):
                    one()
                torch.cuda.current_stream().wait_stream(stream)
            else:
                one()
        torch.cuda.synchronize()
        return [*ps, opt.m, opt.v, opt.clock]

    want = run("eager")
    assert want[-1][0].item() == 5
    for mode in ("graph", "stream"):
        assert all(torch.equal(a, b) for a, b in zip(run(mode), want)), mode


def test_norm(native_lib):
    """Sizes, alignments, empty tensors and None; repeats give the same bits; a small tensor beside a large one
    is not lost; the workspace is used again."""
    ws = train.grad_norm_workspace()
    for dtype in (torch.float32, torch.bfloat16):
        for sizes in ([1], [0, 5], [3, 0, 4097], [100] * 700, [1 << 22, 9], [2048] * 3):
            for lead in (0, 1):
                gs, _ = tensors(sizes, dtype, lead, 1.0, 7)
                want = math.sqrt(sum(g.double().square().sum().item() for g in gs))
                got = train.grad_norm([None, *gs, None], ws=ws)
                assert abs(got.item() - want) <= 64 * U * want
                assert torch.equal(train.grad_norm(gs), got)
    assert train.grad_norm([torch.zeros(0, device="cuda")], ws=ws).item() == 0.0
    assert math.isnan(train.grad_norm([torch.tensor([1.0, float("nan")], device="cuda")]).item())
    assert train.grad_norm([torch.tensor([1.0, float("-inf")], device="cuda")]).item() == math.inf
    assert train.grad_norm([torch.ones(5000, 3000, device="cuda")]).item() == pytest.approx(math.sqrt(15e6), rel=64 * U)


def test_large_tensor(native_lib):
    """Offsets beyond 2^32 elements: a tensor of 2^32 + 12345 bf16 parameters, its last elements."""
    n = (1 << 32) + 12345
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-300:], g[-300:] = 1.0, 0.5
    p[1 << 32], g[1 << 32] = 1.0, -0.5
    opt = train.AdamW([p], lr=0.25, weight_decay=0.0, bits=8)
    opt.step([g])
    assert train.grad_norm([g]).item() == pytest.approx(0.5 * math.sqrt(301.0), rel=64 * U)
    assert (p[-300:] == 0.75).all() and p[1 << 32].item() == 1.25 and (p[:1 << 20] == 0).all()
    assert (opt.m[n - 300:n] == 127).all() and opt.m[1 << 32].item() == -127 and (opt.v[n - 300:n] == 255).all()
    assert (opt.m[n:] == 0).all() and (p[(1 << 32) + 1:n - 300] == 0).all()
