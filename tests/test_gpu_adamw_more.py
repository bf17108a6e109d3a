"""AdamW on the GPU where a run of steps or a choice of arguments counts: clipping by its own norm, lr on the device with
weight decay, many steps with random codes."""

import pytest
import torch

from block_util import U, assert_within, generator, half_step
from test_gpu_adamw import flat, reference, tensors
from top_gating_expert_gb300 import train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_clips_by_its_own_norm(native_lib, bits):
    """A step without a norm gives the bits of one that is given its gradients' norm, eager and replayed; gradients
    below the largest norm are left alone."""
    sizes = [4000, 3, 257]
    runs = []
    for how in ("given", "own", "graph"):
        ps, _ = tensors(sizes, torch.float32, 0, 1.0, 4)
        gs, _ = tensors(sizes, torch.float32, 0, 1.0, 5)
        opt = train.AdamW(ps, lr=1e-2, bits=bits, max_norm=0.25)
        if how == "graph":
            start = [t.clone() for t in (*ps, opt.m, opt.v, opt.clock)]
            graph = torch.cuda.CUDAGraph()
            opt.step(gs)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                opt.step(gs)
            for t, k in zip((*ps, opt.m, opt.v, opt.clock), start):
                t.copy_(k)
            if bits == 8:
                opt.m_scale.zero_()
                opt.v_scale.zero_()
        for t in range(3):
            if how == "graph":
                graph.replay()
            else:
                opt.step(gs, norm=train.grad_norm(gs) if how == "given" else None)
        runs.append([*ps, opt.m, opt.v, opt.clock])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
    free, _ = tensors(sizes, torch.float32, 0, 1.0, 4)
    loose, _ = tensors(sizes, torch.float32, 0, 1.0, 4)
    for ps, top in ((free, None), (loose, 1e9)):
        train.AdamW(ps, lr=1e-2, bits=bits, max_norm=top).step(gs)
    assert all(torch.equal(a, b) for a, b in zip(free, loose))
    assert not torch.equal(runs[0][-3], torch.zeros_like(runs[0][-3]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pt", ["f32", "bf16"])
def test_decay_with_lr_on_the_device(native_lib, bits, pt):
    """Weight decay of each tensor's own with an lr that the device reads and that changes between steps, against the
    formula in 64 bits. The factor 1 - lr wd takes a constant and a fused product, 2 u of p, beside the product with p
    and the sum with the step: within the 4 u of `reference`."""
    dt = dict(f32=torch.float32, bf16=torch.bfloat16)[pt]
    sizes, wd = [300, 4000, 5, 257], [0.5, 0.0, 0.03, 0.1]
    ps, _ = tensors(sizes, dt, 1, 1.0, 4)
    opt = train.AdamW(ps, lr=7.0, betas=(0.9, 0.99), bits=bits, seed=3 if bits == 8 else None, weight_decay=wd)
    lr = torch.zeros(1, device="cuda")
    for t, value in enumerate((0.3, 2.0 ** -4, 0.0123, 0.0), 1):
        lr.fill_(value)
        gs, _ = tensors(sizes, torch.float32, 1, 0.1, 10 + t)
        old = [p.clone() for p in ps]
        m, v = (x.clone() for x in opt.moments())
        opt.step(gs, lr=lr)
        for i in range(len(sizes)):
            ref, tol = reference(old[i], gs[i], flat(opt, m, i), flat(opt, v, i), t, lr.item(), 0.9, 0.99, 1e-8, wd[i],
                                 1.0)
            assert_within(ps[i], ref[0], tol[0] + half_step(dt) * (ref[0].abs() + tol[0]), f"step {t}, p {i}")


LEVEL = 255.0 ** 2


def test_random_codes_of_small_moments(native_lib):
    """One step, roots of v from far below the lowest code's value to some codes above: u = sqrt(v) keeps its expectation
    where a code's value is at most u, the others take code 1, and v has u's squared expectation and variance. Within 5
    standard errors over 2^18 elements, of the two-valued distribution itself; thresholds have 16 bits, 2^-17 of a
    gap."""
    blocks = 1 << 18
    for y in (0.01, 0.3, 0.9, 1.5, 2.5, 5.0, 10.5, 60.0):
        u = torch.zeros(blocks, 256, device="cuda")
        u[:, 0], u[:, 7] = 1.0, y / LEVEL
        opt = train.AdamW([torch.zeros(blocks * 256, device="cuda")], bits=8, seed=11, betas=(0.9, 0.0))
        opt.step([u.view(-1)])
        got = opt.moments()[1].view(blocks, 256)[:, 7].double().sqrt() * LEVEL
        k = int(y ** 0.5)
        gap, f = 2 * k + 1, (y - k * k) / (2 * k + 1)
        if k == 0:
            assert ((got - 1).abs() <= 16 * U).all()
            continue
        assert (((got - k * k).abs() <= 16 * U * y) | ((got - k * k - gap).abs() <= 16 * U * (k + 1) ** 2)).all()
        slack = 2.0 ** -16 * gap
        assert abs(got.mean().item() - y) <= 5 * gap * (f * (1 - f) / blocks) ** 0.5 + slack
        v = y * y + f * (1 - f) * gap * gap
        se = ((k + 1) ** 4 - k ** 4) * (f * (1 - f) / blocks) ** 0.5
        assert abs(got.square().mean().item() - v) <= 5 * se + slack * 2 * (k + 1) ** 2


def test_random_codes_over_many_steps(native_lib):
    """Normal gradients, beta2 = 0.95, 600 steps from the gradients' own variance on: v behaves as the recursion with
    unbiased roots does (emulated in 64 bits with other random numbers), and is high by about 1 / c of itself at code c;
    m follows its own recursion without a bias. Within 5 standard errors of the elements' averages."""
    blocks, b1, b2, steps, skip = 64, 0.9, 0.95, 600, 100
    codes = [1, 2, 4, 8, 14, 25, 50, 81]
    gen = generator(5)
    c = torch.tensor(codes, device="cuda", dtype=torch.float64).repeat(32)[:255]
    size = torch.cat([torch.ones(1, device="cuda", dtype=torch.float64), (c / 255) ** 2]).repeat(blocks, 1)
    n = size.numel()
    opt = train.AdamW([torch.zeros(n, device="cuda")], bits=8, seed=2, betas=(b1, b2))
    opt.v.copy_(torch.cat([torch.full((1,), 255.0, device="cuda"), c.float()]).repeat(blocks).to(torch.uint8))
    opt.v_scale.fill_(1.0)
    opt.clock.copy_(torch.tensor([1000.0, b1 ** 1000, b2 ** 1000], dtype=torch.float64))
    v = size.square()
    m = torch.zeros_like(v)
    mean, want, off = torch.zeros_like(v), torch.zeros_like(v), torch.zeros_like(v)
    for t in range(steps):
        g = torch.randn(blocks, 256, generator=gen, device="cuda") * size.float()
        g[:, 0] = 1.0
        opt.step([g.view(-1)])
        gm, gv = (x.view(blocks, 256).double() for x in opt.moments())
        gd = g.double()
        m = b1 * m + (1 - b1) * gd
        y = (b2 * v + (1 - b2) * gd * gd).sqrt() * LEVEL
        k = y.sqrt().floor()
        k = torch.where((y - k * k) / (2 * k + 1) > torch.rand(y.shape, generator=gen, device="cuda"), k + 1, k)
        v = (k.clamp(min=1.0) / 255) ** 4
        v[:, 0] = 1.0
        if t >= skip:
            mean += gv / size.square() / (steps - skip)
            want += v / size.square() / (steps - skip)
            off += (gm - m) / size / (steps - skip)
    se = lambda x: x.std().item() / x.numel() ** 0.5
    for i, code in enumerate(codes):
        a, b, d = (x[:, 1 + i::len(codes)] for x in (mean, want, off))
        assert abs(a.mean().item() - b.mean().item()) <= 5 * (se(a) ** 2 + se(b) ** 2) ** 0.5, code
        assert abs(d.mean().item()) <= 5 * se(d), code
        if code <= 14:
            assert 0.4 / code - 5 * se(a) <= a.mean().item() - 1 <= 2.2 / code + 5 * se(a), (code, a.mean().item())
