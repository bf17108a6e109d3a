"""What TrainStep makes of the weights, draws and inputs that it is given."""

import pytest
import torch

from block_util import assert_within, generator
from test_gpu_train import MOE, SCORE, dense64, dense_weights, moe_weights
from top_gating_expert_gb300 import block, train

pytestmark = pytest.mark.gpu


def test_masters_are_the_values_given(native_lib):
    """Blocks in bf16 made from float32 weights, as a resumed run has them: the masters are those, experts' and
    dense ones alike, and the weights that the forward reads their rounding."""
    w, x = moe_weights(MOE, 5)
    w = {n: t if t is None or not torch.is_tensor(t) or t.dtype is not torch.bfloat16 else
         t.float() * (1 + 2.0 ** -12) for n, t in w.items()}
    d = dense_weights(MOE["M"], 256, 6, torch.float32)
    head = torch.randn(1003, MOE["M"], generator=generator(7), device="cuda").bfloat16()
    blocks = [block.MoeBlock(MOE, w, score=SCORE), block.DenseBlock(MOE["S"], d)]
    before = blocks[0].forward(x).clone()
    step = train.TrainStep(blocks, [w, d], head, lr=1e-3)
    values = {f"{i}.{n}": t for i, v in enumerate((w, d)) for n, t in v.items() if torch.is_tensor(t)}
    values["head"] = head
    assert len(step.masters) == 17
    for (n, p), c in zip(step.masters, step.opt.copies):
        assert p.dtype is torch.float32 and torch.equal(p, values[n].to("cuda", torch.float32)), n
        assert c is None or torch.equal(c, p.bfloat16()), n
        assert (c is None) == (values[n].dim() == 1), n
    step.blocks[0].layer.set_weights(step._unpacked[0])
    assert torch.equal(blocks[0].forward(x), before)


@pytest.mark.parametrize("M,lead", [(64, 0), (64, 1), (68, 0), (67, 3)])
def test_workspace_of_the_head(native_lib, M, lead):
    """Room for copies of x and the head only where rows are on no 16-byte boundary; a step runs in what there is."""
    T, V = 200, 3001
    d = dense_weights(M, 96, 6, torch.bfloat16)
    head = torch.zeros(V * M + 8, device="cuda", dtype=torch.bfloat16)[lead:lead + V * M].view(V, M)
    head.copy_(torch.randn(V, M, generator=generator(7), device="cuda") * M ** -0.5)
    first = head.clone()
    step = train.TrainStep([block.DenseBlock(T, d)], [d], head, lr=1e-2)
    least, most = (train.linear_cross_entropy_workspace(T, V, M, aligned=a).numel() for a in (True, False))
    copies = lead or M % 8
    assert step.ws.numel() == (most if copies else least) and (most - least > 2 * V * M or M % 8)
    x = torch.randn(T, M, generator=generator(8), device="cuda").bfloat16()
    stats = step.step(x, torch.randint(0, V, (T,), generator=generator(9), device="cuda"))
    assert torch.isfinite(stats).all() and not torch.equal(head, first)


@pytest.mark.parametrize("blocks", [0, 2])
def test_gradient_of_the_input(native_lib, blocks):
    """Against the same model in 64 bits; tolerance as in the float32 steps' test: 1e-4 of a gradient and of their
    root mean square."""
    T, M, V = 130, 64, 700
    ws = [dense_weights(M, 96, s, torch.float32) for s in range(blocks)]
    head = torch.randn(V, M, generator=generator(7), device="cuda") * M ** -0.5
    step = train.TrainStep([block.DenseBlock(T, w, dtype=torch.float32) for w in ws], ws, head, lr=1e-2)
    x = torch.randn(T, M, generator=generator(8), device="cuda")
    y = torch.randint(0, V, (T,), generator=generator(9), device="cuda")
    x64 = x.double().requires_grad_(True)
    h = x64
    for w in ws:
        h = dense64(h, {n: t.double() for n, t in w.items()})
    want, = torch.autograd.grad(torch.nn.functional.cross_entropy(h @ head.double().t(), y), x64)
    step.step(x, y)
    assert step.dx.shape == x.shape
    assert_within(step.dx, want, 1e-4 * (want.abs() + want.square().mean().sqrt()), "dx")


def test_draws_of_each_block(native_lib):
    """Blocks with random routing take draws of their own from a list; one tensor serves all of them."""
    cfg = dict(MOE, act="relu", n_shared=0, H_shared=0, random_routing=1, capacity_factor=1.0, bias=False)
    w, x = moe_weights(cfg, 5)
    w.pop("select_bias")
    d = dense_weights(cfg["M"], 96, 6, torch.bfloat16)
    head = (torch.randn(1003, cfg["M"], generator=generator(7), device="cuda") * 0.1).bfloat16()
    make = lambda: [block.MoeBlock(cfg, w), block.DenseBlock(cfg["S"], d), block.MoeBlock(cfg, w)]
    step, own = train.TrainStep(make(), [w, d, w], head, lr=1e-3), make()
    y = torch.randint(0, 1003, (cfg["S"],), generator=generator(8), device="cuda")
    u = torch.rand(2, cfg["S"], generator=generator(9), device="cuda")
    for draws, each in ((u[0], (u[0], u[0])), ([u[0], None, u[1]], (u[0], u[1])), ((u[1], u[0], u[0]), (u[1], u[0]))):
        step.gradients(x, y, draws)
        want = own[2].forward(own[1].forward(own[0].forward(x, each[0])), each[1])
        assert torch.equal(step.blocks[2].y, want)
        for a, b in ((0, 0), (2, 2)):
            assert torch.equal(step.blocks[a].layer.route_out.row, own[b].layer.route_out.row)
    assert not torch.equal(step.blocks[0].layer.route_out.drop_reason, step.blocks[2].layer.route_out.drop_reason)
    with pytest.raises(ValueError):
        step.gradients(x, y, [u[0], u[1]])


def test_weights_that_a_step_would_refuse(native_lib):
    """Experts in another shape, as a layer packs them by address: refused before the first step changes anything.
    A layer made from other values takes the dict's at once."""
    cfg = dict(MOE, bias=False)
    w, x = moe_weights(cfg, 5)
    w.pop("select_bias")
    head = torch.zeros(100, cfg["M"], device="cuda", dtype=torch.bfloat16)
    flat_ = dict(w, W_in=w["W_in"].reshape(-1, cfg["M"]))
    with pytest.raises(ValueError):
        train.TrainStep([block.MoeBlock(cfg, flat_)], [flat_], head)
    other = dict(w, W_in=2 * w["W_in"])
    b = block.MoeBlock(cfg, other)
    before = b.forward(x).clone()
    train.TrainStep([b], [w], head)
    after = b.forward(x).clone()
    assert torch.equal(after, block.MoeBlock(cfg, w).forward(x)) and not torch.equal(after, before)
