"""The cross entropy, the norm and the optimiser together with the blocks: training steps against the same
steps in 64 bits (float32 blocks), against the formulas on the step's own gradients (bf16 with experts),
repeated and captured.

Tolerance of the float32 steps: AdamW divides by sqrt(v), so where a gradient is as small as its own error the
step may be off by as much as the step itself, lr; elsewhere the gradients' relative error (1e-4 as float32
layers' products of a few hundred terms have at most, forward and backward, with their cancellations) counts."""

import numpy as np
import pytest
import torch

from block_util import U, assert_within, generator, half_step
from top_gating_expert_gb300 import block, moe, train
from top_gating_expert_gb300.inputs import make_inputs

pytestmark = pytest.mark.gpu


def dense_weights(M, H, seed, dtype):
    g = generator(seed)
    r = lambda *s, k=1.0: torch.randn(s, generator=g, device="cuda") * k
    return dict(W1=r(H, M, k=M ** -0.5).to(dtype), W2=r(M, H, k=H ** -0.5).to(dtype), b1=r(H, k=0.1), b2=r(M, k=0.1),
                norm_gamma=1 + r(M, k=0.1), norm_beta=r(M, k=0.1))


def moe_weights(cfg, seed):
    inp = make_inputs(cfg, seed=seed)
    g = torch.Generator().manual_seed(seed)
    return dict(inp.host, select_bias=0.1 * torch.randn(cfg["E"], generator=g),
                norm_gamma=1 + 0.1 * torch.randn(cfg["M"], generator=g),
                norm_beta=0.1 * torch.randn(cfg["M"], generator=g)), inp.host["x"].cuda()


def dense64(x, w):
    F = torch.nn.functional
    n = F.layer_norm(x, (x.shape[1],), w["norm_gamma"], w["norm_beta"], 1e-5)
    return x + F.linear(F.gelu(F.linear(n, w["W1"], w["b1"])), w["W2"], w["b2"])


def test_dense_steps_against_64_bits(native_lib):
    T, M, H, V, lr = 300, 64, 96, 700, 1e-2
    ws = [dense_weights(M, H, s, torch.float32) for s in (1, 2)]
    g = generator(3)
    head = torch.randn(V, M, generator=g, device="cuda") * M ** -0.5
    names = ["W1", "W2", "b1", "b2", "norm_gamma", "norm_beta"]
    p64 = [w[n].double() for w in ws for n in names] + [head.double()]
    decay = [0.1 if t.dim() == 2 else 0.0 for t in p64]
    blocks = [block.DenseBlock(T, {k: v.clone() for k, v in w.items()}, dtype=torch.float32) for w in ws]
    step = train.TrainStep(blocks, ws, head.clone(), z_coef=1e-3, lr=lr, betas=(0.9, 0.99), weight_decay=0.1,
                           max_norm=0.3)
    m64 = [torch.zeros_like(t) for t in p64]
    v64 = [torch.zeros_like(t) for t in p64]
    assert [n for n, _ in step.masters][:3] == ["0.W1", "0.W2", "0.b1"] and step.masters[-1][0] == "head"
    slack = [torch.zeros_like(t) for t in p64]
    for t in range(1, 4):
        x = torch.randn(T, M, generator=g, device="cuda")
        y = torch.randint(0, V, (T,), generator=g, device="cuda")
        y[::7] = -100
        # the reference steps from the state that the step itself starts from
        p64 = [p.detach().double().requires_grad_(True) for _, p in step.masters]
        o = step.opt
        m64 = [o.m[a:a + p.numel()].double().view(p.shape) for a, p in zip(o.first, p64)]
        v64 = [o.v[a:a + p.numel()].double().view(p.shape) for a, p in zip(o.first, p64)]
        h = x.double()
        for i in range(2):
            h = dense64(h, dict(zip(names, p64[6 * i:6 * i + 6])))
        l = h @ p64[-1].t()
        lse = torch.logsumexp(l, 1)
        keep = y != -100
        each = lse - l.gather(1, torch.where(keep, y, 0)[:, None])[:, 0] + 1e-3 * lse ** 2
        loss = (each * keep).sum() / keep.sum()
        grads = torch.autograd.grad(loss, p64)
        norm = torch.sqrt(sum(k.square().sum() for k in grads))
        coef = min(1.0, 0.3 / (norm.item() + 1e-6))
        stats = step.step(x, y)
        assert abs(stats[0].item() - loss.item()) <= 1e-5 * abs(loss.item()) and stats[1] == keep.sum()
        for (name, p), p0, k, m, v, wd in zip(step.masters, p64, grads, m64, v64, decay):
            k = k * coef
            m, v = 0.9 * m + 0.1 * k, 0.99 * v + 0.01 * k * k
            den = (v / (1 - 0.99 ** t)).sqrt() + 1e-8
            ref = p0.detach() * (1 - lr * wd) - lr * m / (1 - 0.9 ** t) / den
            e = 1e-4 * (k.abs() + k.square().mean().sqrt())  # of a gradient
            tol = 4 * U * ref.abs() + 40 * U * lr + lr * torch.minimum(torch.full_like(e, 2.0), 2 * e / den)
            assert_within(p.detach(), ref, tol, f"step {t}: {name}")


MOE = dict(S=512, G=1, E=8, M=128, H=128, k=2, capacity_factor=0.0, random_routing=0, n_shared=2, H_shared=64,
           act="swiglu", dtype="bf16", bias=True)
SCORE = dict(score="sigmoid", group_top=1, renorm=1, scale=1.5)


def moe_step(bits, seed=None, cfg=MOE, score=SCORE):
    M, T, V = cfg["M"], cfg["S"], 1003
    dt = torch.bfloat16 if cfg["dtype"] == "bf16" else torch.float32
    w, x = moe_weights(cfg, 5)
    if score is None:
        w.pop("select_bias")
    d = dense_weights(M, 256, 6, dt)
    head = (torch.randn(V, M, generator=generator(7), device="cuda") * M ** -0.5).to(dt)
    blocks = [block.MoeBlock(cfg, w, score=score), block.DenseBlock(T, d, dtype=dt)]
    step = train.TrainStep(blocks, [w, d], head, aux_coef=0.01, router_z=1e-3, z_coef=1e-4, lr=1e-3, max_norm=1.0,
                           bits=bits, seed=seed)
    y = torch.randint(0, V, (T,), generator=generator(8), device="cuda")
    return step, x, y


@pytest.mark.parametrize("bits,seed", [(32, None), (8, 3)])
def test_moe_step(native_lib, bits, seed):
    """A step moves every weight by AdamW's formula on the step's own gradients; the bf16 weights are the rounded
    masters; the packed experts are those of a layer made from them: the next forward's bits say so."""
    step, x, y = moe_step(bits, seed)
    names = [n for n, _ in step.masters]
    assert names == [f"0.{n}" for n in ("W_g", "W_in", "W_up", "W_out", "Ws_in", "Ws_up", "Ws_out", "bias",
                                        "norm_gamma", "norm_beta")] + \
        [f"1.{n}" for n in ("W1", "W2", "b1", "b2", "norm_gamma", "norm_beta")] + ["head"]
    for t in range(1, 3):
        stats, grads = step.gradients(x, y)
        grads = [g.clone() for g in grads]
        assert all(g.numel() == p.numel() for g, (_, p) in zip(grads, step.masters))
        old = [p.detach().clone() for _, p in step.masters]
        m0, v0 = (z.clone() for z in step.opt.moments())
        again = step.step(x, y)
        assert torch.equal(stats, again)
        norm = train.grad_norm(grads)
        coef = min(1.0, 1.0 / (norm.item() + 1e-6))
        for (n, p), o, g, at in zip(step.masters, old, grads, step.opt.first):
            g = g.float().view(o.shape).double() * coef
            m = 0.9 * m0[at:at + o.numel()].view(o.shape).double() + 0.1 * g
            v = 0.999 * v0[at:at + o.numel()].view(o.shape).double() + 0.001 * g * g
            den = (v / (1 - 0.999 ** t)).sqrt() + 1e-8
            ref = o.double() * (1 - 1e-3 * (0.01 if o.dim() > 1 else 0)) - 1e-3 * m / (1 - 0.9 ** t) / den
            # m is off by 6 u of its terms, the rest of the step by 40 u
            e = 1e-3 / (1 - 0.9 ** t) * 6 * U * ((0.9 * m0[at:at + o.numel()].view(o.shape).double()).abs()
                                                 + 0.1 * g.abs()) / den
            assert_within(p.detach(), ref, 4 * U * ref.abs() + 40 * U * 1e-3 * (m / den).abs() * 10 + e + 1e-12,
                          f"step {t}: {n}")
    low = dict(zip(names, (c for c in step.opt.copies)))
    for n, p in step.masters:
        if low[n] is not None:
            assert torch.equal(low[n], p.bfloat16()), n
    b = step.blocks[0]
    fresh = dict(step._unpacked[0], norm_gamma=b.gamma, norm_beta=b.beta)
    other = block.MoeBlock(MOE, {k: v.clone() for k, v in fresh.items()}, score=SCORE)
    assert torch.equal(other.forward(x), b.forward(x))
    other.enable_backward({k: v.clone() for k, v in fresh.items()})
    dy = torch.randn(x.shape, generator=generator(9), device="cuda").bfloat16()
    for s, t in zip(other.backward(x, dy)[:3], b.backward(x, dy)[:3]):
        assert torch.equal(s, t)


@pytest.mark.parametrize("cfg,score", [(dict(MOE, dtype="f32", bias=False), None),
                                       (dict(MOE, act="relu", n_shared=0, H_shared=0, random_routing=1,
                                             capacity_factor=1.0), None)])
def test_other_layers_and_capture(native_lib, cfg, score):
    """float32 layers, default and random routing: steps run, and a captured step's replays give the bits of eager
    steps on the same inputs."""
    u = torch.rand(cfg["S"], generator=generator(2), device="cuda") if cfg["random_routing"] else None
    runs = []
    for mode in ("eager", "graph"):
        step, x, y = moe_step(32, cfg=cfg, score=score)
        if mode == "graph":
            keep = [t.clone() for t in (step.opt.m, step.opt.v, step.opt.clock)]
            first = [p.detach().clone() for _, p in step.masters]
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step.step(x, y, u)
            torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                stats = step.step(x, y, u)
            # back to the start: masters, what the forward reads, moments and clock
            for (_, p), f, c in zip(step.masters, first, step.opt.copies):
                p.detach().copy_(f)
                if c is not None:
                    c.copy_(f)
            for t, k in zip((step.opt.m, step.opt.v, step.opt.clock), keep):
                t.copy_(k)
            step.blocks[0].layer.set_weights(step._unpacked[0])
            got = []
            for _ in range(3):
                graph.replay()
                got.append(stats.clone())
        else:
            got = [step.step(x, y, u).clone() for _ in range(3)]
        assert step.opt.clock[0].item() == 3
        assert all(torch.isfinite(s).all() for s in got)
        runs.append(got + [p.detach().clone() for _, p in step.masters])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_set_weights_refuses(native_lib):
    step, x, y = moe_step(32)
    layer, w = step.blocks[0].layer, step._unpacked[0]
    for bad in (dict(w, W_in=w["W_in"].float()), dict(w, W_out=w["W_out"][:, :-1]), dict(w, W_up=None),
                dict(w, bias=w["bias"][:-1]), dict(w, W_g=w["W_g"].cpu()), dict(w, Ws_in=w["Ws_in"].transpose(1, 2)),
                dict(w, select_bias=None)):
        with pytest.raises(ValueError):
            layer.set_weights(bad)
    before = layer.W_in_packed.clone()
    layer.set_weights(w)
    assert torch.equal(before, layer.W_in_packed)
