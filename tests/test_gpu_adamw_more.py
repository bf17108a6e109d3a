"""AdamW on the GPU where a run of steps or a choice of arguments counts."""

import pytest
import torch

from block_util import assert_within, half_step
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

