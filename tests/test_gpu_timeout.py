"""The bounded waits' timeout path, on a real launch: with a one-microsecond wait limit set in
its workspace header, the router's single-CTA tcgen05 GEMM (moe_router, bf16) gives up
(every CTA's epilogue waits tens of microseconds for its first accumulator), drains what it
issued, frees its tensor memory and returns early; moe_get_device_status reports
MOE_ERR_TIMEOUT. With the default limit restored, the next call on the same workspace and
context succeeds and its logits match the oracle's fp64 projection."""

import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from gpu_util import LOGIT_RTOL, assert_close, to_np
from top_gating_expert_gb300 import _native as N
from top_gating_expert_gb300 import moe
from top_gating_expert_gb300.inputs import make_inputs

pytestmark = pytest.mark.gpu

MOE_ERR_TIMEOUT = -5
# 128 tiles of 128 rows, each a K loop of 128 k-blocks (M = 8192): the first accumulator of
# a CTA takes far longer than the limit below
CFG = dict(S=16384, G=1, E=64, M=8192, H=128, k=2, capacity_factor=0.0, random_routing=0,
           n_shared=0, H_shared=0, act="relu", dtype="bf16", bias=False)


def test_wait_limit_times_out_then_recovers(native_lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    inp = make_inputs(CFG, seed=4242, names=("x", "W_g"))
    x = inp.host["x"].cuda()
    W_g = inp.host["W_g"].cuda()
    ws = moe.workspace(CFG, N.MOE_WS_STEP)
    logits = torch.empty((CFG["S"], CFG["E"]), dtype=torch.float32, device="cuda")

    moe.set_wait_limit(ws, 1000)  # 1 microsecond
    moe.router(CFG, x, W_g, None, logits, ws)
    assert moe.device_status(ws) == MOE_ERR_TIMEOUT

    moe.set_wait_limit(ws, 0)  # back to the default
    for _ in range(2):
        logits.fill_(float("nan"))
        moe.router(CFG, x, W_g, None, logits, ws)
        assert moe.device_status(ws) == 0
    got = to_np(logits)
    rng = np.random.default_rng(5)
    rows = np.unique(np.concatenate([rng.choice(CFG["S"], 96, replace=False), [0, CFG["S"] - 1]]))
    ref = O.router_logits(inp.np["x"][rows], inp.np["W_g"])
    assert_close(got[rows], ref, LOGIT_RTOL["bf16"], "logits after the timeout")
    assert np.isfinite(got).all()


@pytest.mark.parametrize("act", ["relu", "swiglu"])
@pytest.mark.parametrize("limit_ns", [1, 1000, 5000])
def test_pairs_that_give_up_leave_nothing_behind(native_lib, act, limit_ns):
    """The expert GEMMs' CTA pairs and the backward's GEMMs with limits that stop the two CTAs of a
    pair at k-blocks of their own: a status, and with the default limit the very next calls, on the
    same SMs and shared memory, give what they gave before, bit for bit."""
    cfg = dict(S=3000, G=1, E=6, M=4096, H=4096, k=2, capacity_factor=0.0, random_routing=0, n_shared=1,
               H_shared=512, act=act, dtype="bf16", bias=False)
    inp = make_inputs(cfg, seed=9)
    layer = moe.MoeLayer(cfg, inp.host)
    layer.enable_backward(inp.host)
    c, out = layer.cfg, layer.route_out
    x = inp.host["x"].cuda()
    dy = torch.randn((c.S, c.M), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    names = ["dx", "dW_g", "dW_in", "dW_out", "dWs_in", "dWs_out"] + (["dW_up", "dWs_up"] if act == "swiglu" else [])

    def step():
        y = layer.forward(x, residual=x).clone()
        g = layer.backward(x, dy, residual=True, aux_coef=0.1)
        got = [y] + [getattr(g, n).clone() for n in names]
        assert moe.device_status(layer.ws) == 0 and moe.device_status(layer.ws_bwd) == 0
        return got

    want = step()
    R = moe.rows_max(c)
    x_perm, h, y_perm = (torch.zeros((R, n), dtype=torch.bfloat16, device="cuda") for n in (c.M, c.H, c.M))
    hs, so = (torch.zeros((c.S, n), dtype=torch.bfloat16, device="cuda") for n in (c.n_shared * c.H_shared, c.M))
    moe.dispatch(c, x, out, x_perm)
    for _ in range(4):
        moe.set_wait_limit(layer.ws, limit_ns)
        moe.expert_ffn(c, x_perm, out.expert_offsets, out.w_perm, layer.W_in_packed, layer.W_out_packed, h, y_perm,
                       layer.ws)
        moe.shared_ffn(c, x, layer.Ws_in_packed, layer.Ws_out_packed, hs, so, layer.ws)
        moe.set_wait_limit(layer.ws, 0)
        gave_up = moe.device_status(layer.ws)
        assert gave_up in ((MOE_ERR_TIMEOUT,) if limit_ns == 1 else (0, MOE_ERR_TIMEOUT))
        for a, b in zip(step(), want):
            assert torch.equal(a, b)
        moe.set_wait_limit(layer.ws_bwd, limit_ns)
        layer.backward(x, dy, residual=True, aux_coef=0.1)
        moe.set_wait_limit(layer.ws_bwd, 0)
        assert moe.device_status(layer.ws_bwd) in (0, MOE_ERR_TIMEOUT)
        for a, b in zip(step(), want):
            assert torch.equal(a, b)
