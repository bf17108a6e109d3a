"""The scored MoE layer and the two pre-norm blocks on the GPU, forward and backward, against a
64-bit evaluation differentiated by autograd with the routing decisions held fixed. Tolerance: the
bf16 layer form |g - r| <= 2e-2 (|r| + rms(row)) (bf16 operands and stored intermediates, fp32
accumulation), fp32 layers 1e-5 as the other layer tests; routing bit for bit."""

import numpy as np
import pytest
import torch

from gpu_util import RTOL, assert_close, oracle_cfg, route_np, to_np
from oracle import scored as SC
from top_gating_expert_gb300 import block, moe
from top_gating_expert_gb300.inputs import make_inputs

pytestmark = pytest.mark.gpu


def _cfg(**kw):
    base = dict(S=1024, G=1, E=16, M=256, H=256, k=4, capacity_factor=0.0, random_routing=0, n_shared=0,
                H_shared=0, act="swiglu", dtype="bf16", bias=False)
    base.update(kw)
    return base


CASES = {
    "groups_shared_dropless": (_cfg(E=32, n_expert_groups=8, topk_groups=3, n_shared=1, H_shared=128),
                               dict(score="sigmoid", group_top=2, renorm=1, scale=2.5)),
    "capacity_relu": (_cfg(G=4, E=8, k=2, capacity_factor=0.75, act="relu"),
                      dict(score="sigmoid", group_top=1, renorm=0, scale=1.0)),
    "softmax_ragged": (_cfg(S=777, E=12, k=3, act="relu"), dict(score="softmax", group_top=1, renorm=0, scale=1.5)),
    "one_token": (_cfg(S=1, E=64, k=6), dict(score="sigmoid", group_top=1, renorm=1, scale=2.5)),
    "fp32": (_cfg(S=200, E=8, M=64, H=128, k=2, dtype="f32", act="relu"),
             dict(score="sigmoid", group_top=1, renorm=1, scale=1.0)),
}
AUX, Z = 0.5, 0.1


def weights_of(cfg, seed):
    inp = make_inputs(cfg, seed=seed)
    w = dict(inp.host)
    g = torch.Generator().manual_seed(seed)
    w["select_bias"] = 0.1 * torch.randn(cfg["E"], generator=g)
    w["norm_gamma"] = 1 + 0.2 * torch.randn(cfg["M"], generator=g)
    w["norm_beta"] = 0.1 * torch.randn(cfg["M"], generator=g)
    return w


def moe64(n, w, cfg, score, r, logits_gpu):
    """The MoE output of normalised tokens n (float64, on autograd) with r's decisions; the router's
    logits take the GPU's values and this expression's gradient."""
    logits = n @ w["W_g"].t()
    logits = logits + (logits_gpu - logits).detach()
    ids = torch.from_numpy(r["expert_id"])
    kept = torch.from_numpy((r["pos"] >= 0).astype(np.float64))
    s = torch.sigmoid(logits) if score["score"] == "sigmoid" else torch.softmax(logits, 1)
    g = s.gather(1, ids)
    if score["renorm"]:
        g = g / g.sum(1, keepdim=True)
    g = g * score["scale"] * kept

    def ffn(x, W_in, W_up, W_out):
        a = x @ W_in.t()
        h = torch.relu(a) if cfg["act"] == "relu" else torch.nn.functional.silu(a) * (x @ W_up.t())
        return h @ W_out.t()

    y = torch.zeros_like(n)
    for e in range(cfg["E"]):
        t, j = torch.nonzero((ids == e) & (kept > 0), as_tuple=True)
        if len(t):
            y = y.index_add(0, t, g[t, j][:, None] * ffn(n[t], w["W_in"][e], w["W_up"][e] if "W_up" in w else None,
                                                         w["W_out"][e]))
    for i in range(cfg["n_shared"]):
        y = y + ffn(n, w["Ws_in"][i], w["Ws_up"][i] if "Ws_up" in w else None, w["Ws_out"][i])
    q = s / s.sum(1, keepdim=True)
    G, Sg = cfg["G"], cfg["S"] // cfg["G"]
    f = torch.from_numpy(r["counts_routed"] / float(Sg * cfg["k"]))
    aux = (cfg["E"] * (f * q.reshape(G, Sg, -1).mean(1)).sum(1)).mean()
    z = torch.logsumexp(logits, 1).square().mean()
    return y, aux, z


@pytest.mark.parametrize("name", sorted(CASES))
def test_moe_block(native_lib, name):
    cfg, score = CASES[name]
    w = weights_of(cfg, 5)
    blk = block.MoeBlock(cfg, w, score=score)
    blk.enable_backward(w)
    dt = moe.torch_dtype(cfg)
    x = (w["x"].float() * 0.8 + 0.3).to(dt).cuda()
    out = blk.forward(x)
    assert moe.device_status(blk.layer.ws) == 0
    logits = blk.layer.logits.cpu().numpy()
    r = SC.route(logits, w["select_bias"].numpy(), oracle_cfg(cfg), score)
    got = route_np(blk.layer.route_out)
    for key in ("expert_id", "pos", "row", "counts", "counts_routed", "expert_offsets"):
        np.testing.assert_array_equal(got[key], r[key], err_msg=key)
    # 64-bit reference, from the GPU's own normalised tokens onward so that roundings of n do not count
    names = [k for k in ("W_g", "W_in", "W_up", "W_out", "Ws_in", "Ws_up", "Ws_out") if w.get(k) is not None]
    w64 = {k: w[k].double().requires_grad_(True) for k in names}
    x64 = x.double().cpu().requires_grad_(True)
    gamma, beta = (w[k].double().requires_grad_(True) for k in ("norm_gamma", "norm_beta"))
    mean = x64.mean(1, keepdim=True)
    n64 = (x64 - mean) / torch.sqrt((x64 - mean).square().mean(1, keepdim=True) + 1e-5) * gamma + beta
    assert_close(to_np(blk.n), n64.detach().numpy(), RTOL[cfg["dtype"]], "n")
    n_used = n64 + (blk.n.double().cpu() - n64).detach()
    y, aux, z = moe64(n_used, w64, cfg, score, r, torch.from_numpy(logits).double())
    ref = x64 + y
    rtol = RTOL[cfg["dtype"]]
    assert_close(to_np(out), ref.detach().numpy(), rtol, "out")
    dy = torch.randn((cfg["S"], cfg["M"]), generator=torch.Generator().manual_seed(9)).to(dt)
    (ref * dy.double()).sum().add(AUX * aux + Z * z).backward()
    dx, dgamma, dbeta, g = blk.backward(x, dy.cuda(), aux_coef=AUX, z_coef=Z)
    assert moe.device_status(blk.layer.ws_bwd) == 0
    assert_close(to_np(dx), x64.grad.numpy(), rtol, "dx")
    assert_close(to_np(dgamma), gamma.grad.numpy(), rtol, "dgamma")
    assert_close(to_np(dbeta), beta.grad.numpy(), rtol, "dbeta")
    for key in names:
        mine, theirs = getattr(g, "d" + key), w64[key].grad
        for e in range(theirs.shape[0] if theirs.dim() == 3 and key[:2] != "Ws" else 1):
            a = mine[e] if theirs.dim() == 3 and key[:2] != "Ws" else mine
            b = theirs[e] if theirs.dim() == 3 and key[:2] != "Ws" else theirs
            if key in ("Ws_in", "Ws_up"):
                b = theirs.reshape(-1, cfg["M"])
            if key == "Ws_out":
                b = theirs.permute(1, 0, 2).reshape(cfg["M"], -1)
            assert_close(to_np(a), b.numpy(), rtol, f"d{key}[{e}]")


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (5, 3)])
@pytest.mark.parametrize("name", ["softmax_ragged", "fp32", "one_token"])
def test_moe_block_on_strided_rows(native_lib, name, pad, offset):
    """x and dy whose rows lie apart or start off a 16-byte boundary: what the layer gives for
    contiguous ones, bit for bit, on the current stream and on another."""
    cfg, score = CASES[name]
    w = weights_of(cfg, 7)
    dt, (S, M) = moe.torch_dtype(cfg), (cfg["S"], cfg["M"])
    g = torch.Generator().manual_seed(11)
    x, dy = (torch.randn((S, M), generator=g).to(dt).cuda() for _ in range(2))

    def apart(t):
        full = torch.full((S * (M + pad) + offset,), 1e3, dtype=dt, device="cuda")
        return full[offset:].as_strided((S, M), (M + pad, 1)).copy_(t)

    xs, dys = apart(x), apart(dy)
    for stream in (None, torch.cuda.Stream()):
        blk, layer = block.MoeBlock(cfg, w, score=score), moe.MoeLayer(cfg, w, score=score)
        blk.enable_backward(w)
        layer.enable_backward(w)
        torch.cuda.synchronize()
        y = blk.forward(xs, stream=stream)
        dx, dgamma, dbeta, got = blk.backward(xs, dys, aux_coef=AUX, z_coef=Z, stream=stream)
        torch.cuda.synchronize()
        assert moe.device_status(blk.layer.ws) == 0 and moe.device_status(blk.layer.ws_bwd) == 0
        assert torch.equal(y, layer.forward(blk.n, residual=x))
        want = layer.backward(blk.n, dy, aux_coef=AUX, z_coef=Z)
        for k in ("dx", "dW_g", "dW_in", "dW_out"):
            assert torch.equal(getattr(got, k), getattr(want, k)), k
        norm = block.layer_norm_backward(want.dx, xs, blk.gamma, blk.mean, blk.rstd, dh=dy)
        for a, b in zip((dx, dgamma, dbeta), norm):
            assert torch.equal(a, b)


def test_moe_block_backward_refuses_other_shapes(native_lib):
    cfg, score = CASES["softmax_ragged"]
    w = weights_of(cfg, 7)
    blk = block.MoeBlock(cfg, w, score=score)
    blk.enable_backward(w)
    x = w["x"].to(torch.bfloat16).cuda()
    blk.forward(x)
    for bad in (x[:-1], x[:, :-8], x.float(), x.cpu()):
        with pytest.raises(ValueError):
            blk.backward(x, bad)
        with pytest.raises(ValueError):
            blk.backward(bad, x)


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_of_shifted_logits(native_lib, dtype, renorm):
    """Softmax scores do not know a common offset: with every logit 78 lower (exactly: x and W_g on
    coarse grids) the layer of 8 experts routes the same, and its gradients are the same but for
    roundings."""
    cfg = _cfg(S=300, E=8, k=2, act="relu", dtype=dtype, M=256 if dtype == "bf16" else 64)
    score = dict(score="softmax", group_top=1, renorm=renorm, scale=1.5)
    w = weights_of(cfg, 8)
    w["W_g"] = (w["W_g"].float() * 64).round().div(64).to(w["W_g"].dtype)
    x = (w["x"].float() * 4).round().div(4).to(w["x"].dtype).cuda()
    dy = torch.randn((cfg["S"], cfg["M"]), generator=torch.Generator().manual_seed(3)).to(x.dtype).cuda()
    results = []
    for shift in (0.0, -78.0):
        layer = moe.MoeLayer(cfg, dict(w, bias=torch.full((8,), shift)), score=score)
        layer.enable_backward(w)
        y = layer.forward(x)
        g = layer.backward(x, dy, aux_coef=AUX)
        results.append([layer.route_out.expert_id, layer.logits - shift, layer.route_out.gate, y, g.dx, g.dW_g,
                        g.dbias, g.dW_in, g.dW_out])
    a, b = results
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # dbias sums over all tokens to (nearly) nothing: its row rms is that of its own terms
    for name, u, v in zip(("gate", "y", "dx", "dW_g", "dbias", "dW_in", "dW_out"), a[2:], b[2:]):
        assert_close(to_np(v), to_np(u), RTOL[dtype], name)


def test_layer_refuses_a_selection_bias_of_another_length(native_lib):
    cfg, score = CASES["capacity_relu"]
    w = weights_of(cfg, 6)
    for n in (cfg["E"] - 1, cfg["E"] + 1):
        with pytest.raises(ValueError, match="select_bias"):
            moe.MoeLayer(cfg, dict(w, select_bias=torch.zeros(n)), score=score)


def test_scored_layer_equals_step_calls(native_lib):
    """moe_layer_forward_scored against the separate calls, bit for bit."""
    cfg, score = CASES["groups_shared_dropless"]
    w = weights_of(cfg, 6)
    layer = moe.MoeLayer(cfg, w, score=score)
    x = w["x"].cuda()
    y = layer.forward(x, residual=x).clone()
    c = layer.cfg
    out = moe.RouteOutputs.allocate(c)
    logits = torch.empty_like(layer.logits)
    R = moe.rows_max(c)
    new = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    x_perm, h, y_perm = new(R, c.M), new(R, c.H), new(R, c.M)
    hs, so = new(c.S, c.n_shared * c.H_shared), new(c.S, c.M)
    moe.router(c, x, layer.W_g, None, logits, layer.ws)
    moe.route_scored(c, score, logits, layer.select_bias, out, layer.ws)
    moe.dispatch(c, x, out, x_perm)
    moe.expert_ffn(c, x_perm, out.expert_offsets, out.w_perm, layer.W_in_packed, layer.W_out_packed, h, y_perm,
                   layer.ws)
    moe.shared_ffn(c, x, layer.Ws_in_packed, layer.Ws_out_packed, hs, so, layer.ws)
    y2 = torch.empty_like(y)
    moe.combine(c, y_perm, out, so, x, y2)
    assert torch.equal(logits, layer.logits)
    for f, v in route_np(out).items():
        np.testing.assert_array_equal(v, route_np(layer.route_out)[f], err_msg=f)
    assert torch.equal(y, y2)
    with pytest.raises(ValueError):
        layer.forward(x, u=torch.rand(c.S, device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("T,M,H", [(1, 256, 512), (300, 200, 333), (1500, 512, 1024)])
def test_dense_block(native_lib, dtype, act, T, M, H):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(T + M)
    rn = lambda *s: torch.randn(s, generator=g)
    w = dict(W1=(rn(H, M) / M ** 0.5).to(dt), W2=(rn(M, H) / H ** 0.5).to(dt), b1=0.1 * rn(H), b2=0.1 * rn(M),
             norm_gamma=1 + 0.2 * rn(M), norm_beta=0.1 * rn(M))
    x, dy = (rn(T, M) + 0.5).to(dt), rn(T, M).to(dt)
    blk = block.DenseBlock(T, w, act=act, dtype=dt)
    out = blk.forward(x.cuda())
    got = blk.backward(x.cuda(), dy.cuda())
    w64 = {k: v.double().requires_grad_(True) for k, v in w.items()}
    x64 = x.double().requires_grad_(True)
    # each stored intermediate (n, pre, a) takes the GPU's value and the expression's gradient: the
    # backward is defined on what the forward stored, and with one token a slope near zero would
    # otherwise turn pre's rounding into any relative error of d
    stored = lambda v, t: v + (t.double().cpu() - v).detach()
    n = torch.nn.functional.layer_norm(x64, (M,), w64["norm_gamma"], w64["norm_beta"], 1e-5)
    pre = stored(n, blk.n) @ w64["W1"].t() + w64["b1"]
    used = stored(pre, blk.pre)
    a = {"relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[act](used)
    rtol = RTOL[dtype] if dtype == "bf16" else 2e-5  # five fp32 products and norms in a row
    for name, mine, theirs in (("n", blk.n, n), ("pre", blk.pre, pre), ("a", blk.a, a)):
        assert_close(to_np(mine), theirs.detach().numpy(), rtol, name)
    a = stored(a, blk.a)
    ref = x64 + a @ w64["W2"].t() + w64["b2"]
    (ref * dy.double()).sum().backward()
    assert_close(to_np(out), ref.detach().numpy(), rtol, "out")
    assert_close(to_np(got["dx"]), x64.grad.numpy(), rtol, "dx")
    for k in w:
        assert_close(to_np(got[k]), w64[k].grad.numpy(), rtol, f"d{k}")


def test_backward_captured_beside_an_eager_graph(native_lib):
    """Capturing a block's step while an autograd graph over the same weights is alive: the entry
    points touch no autograd state, and the replay repeats the eager results."""
    g = torch.Generator().manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g)
    w = dict(W1=(rn(256, 128) / 12).bfloat16(), W2=(rn(128, 256) / 16).bfloat16(), b1=rn(256), b2=rn(128),
             norm_gamma=rn(128), norm_beta=rn(128))
    blk = block.DenseBlock(200, w)
    x, dy = rn(200, 128).bfloat16().cuda(), rn(200, 128).bfloat16().cuda()
    leaf = blk.W1.requires_grad_(True)
    eager = (x @ leaf.t()).sum()  # alive during the capture
    out = blk.forward(x).clone()
    ref = {k: v.clone() for k, v in blk.backward(x, dy).items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = blk.forward(x)
        got = blk.backward(x, dy)
    graph.replay()
    assert torch.equal(y, out)
    for k in ref:
        assert torch.equal(got[k], ref[k]), k
    eager.backward()
    assert leaf.grad is not None
