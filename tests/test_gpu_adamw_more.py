"""AdamW on the GPU where a run of steps or a choice of arguments counts."""

import pytest
import torch

from test_gpu_adamw import tensors
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

