"""Scored routing on the GPU against the 64-bit oracle: integer outputs bit for bit, over score
kinds, groups, biases, capacities, sizes of one token and one expert up; logits rounded to a
coarse grid (ties), saturated scores, non-finite entries; the gradient; other streams, graphs.

Weights: a choice's score carries the error of expf (2 ulp), of the argument (|l| u), a sum and two
divisions, and of the renormalising sum: 64 u relative covers them (k <= 8), plus the argument's
(spread + 16) u. Un-normalised softmax weights add the sum over E: (E + 16 + spread) u."""

import numpy as np
import pytest
import torch

from gpu_util import LOSS_RTOL, compare_route, route_np
from oracle import scored as SC
from top_gating_expert_gb300 import _native as N
from top_gating_expert_gb300 import moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _cfg(S, G=1, E=64, k=2, cf=0.0, ng=0, tg=0):
    return dict(S=S, G=G, E=E, M=64, H=64, k=k, capacity_factor=cf, random_routing=0, n_shared=0,
                H_shared=0, act="relu", dtype="bf16", n_expert_groups=ng, topk_groups=tg)


def gpu(cfg, score, logits, bias, stream=None):
    lg = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).cuda()
    b = None if bias is None else torch.from_numpy(np.ascontiguousarray(bias, np.float32)).cuda()
    out = moe.RouteOutputs.allocate(cfg)
    ws = moe.workspace(cfg, N.MOE_WS_STEP)
    moe.route_scored(cfg, score, lg, b, out, ws)
    return out, moe.device_status(ws), lg


def check(cfg, score, logits, bias, what=""):
    logits = np.asarray(logits, np.float32)
    out, status, lg = gpu(cfg, score, logits, bias)
    assert status == 0
    o = SC.route(logits, bias, dict(cfg, capacity_factor=float(np.float32(cfg["capacity_factor"]))), score)
    spread = float(logits.max() - logits.min())
    compare_route(route_np(out), o, what, grtol=(cfg["E"] + 64 + spread) * U)
    return out, o, lg


KINDS = [dict(score=s, group_top=g, renorm=r, scale=c)
         for s in ("sigmoid", "softmax") for g, r, c in ((1, 1, 1.0), (2, 0, 2.5), (2, 1, 2.5))]
CASES = [_cfg(1, E=256, k=8, ng=8, tg=4), _cfg(1, E=1, k=1), _cfg(2, E=2, k=2), _cfg(5, E=5, k=3),
         _cfg(127, E=64, k=1), _cfg(128, E=33, k=8), _cfg(129, E=256, k=8, ng=16, tg=3),
         _cfg(300, G=3, E=40, k=4, cf=1.0, ng=5, tg=2), _cfg(1000, G=2, E=64, k=2, cf=1.25),
         _cfg(2048, E=256, k=8, ng=8, tg=4), _cfg(4096, G=16, E=128, k=6, cf=0.5),
         _cfg(777, E=16, k=2, ng=16, tg=2), _cfg(513, E=100, k=7, ng=4, tg=1), _cfg(20000, E=64, k=2, cf=1.25),
         _cfg(64, E=8, k=8, ng=8, tg=8), _cfg(3000, E=160, k=6, ng=8, tg=3)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_routing(native_lib, case, kind):
    cfg, score = CASES[case], KINDS[kind]
    rng = np.random.default_rng(100 * case + kind)
    logits = rng.standard_normal((cfg["S"], cfg["E"])) * (3.0 if kind % 2 else 1.0)
    bias = None if (case + kind) % 3 == 0 else (0.1 * rng.standard_normal(cfg["E"])).astype(np.float32)
    check(cfg, score, logits, bias)


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_ties(native_lib, kind):
    """Logits on a grid of halves and equal biases: exact ties in most tokens."""
    rng = np.random.default_rng(kind)
    for cfg in (_cfg(700, E=64, k=4), _cfg(700, E=128, k=6, ng=8, tg=3), _cfg(200, E=96, k=8, ng=6, tg=2)):
        logits = np.round(rng.standard_normal((cfg["S"], cfg["E"])) * 2) / 2
        check(cfg, KINDS[kind], logits, None)
        check(cfg, KINDS[kind], logits, np.full(cfg["E"], 0.25, np.float32))
        check(cfg, KINDS[kind], np.zeros_like(logits), None)


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_close_scores(native_lib, kind):
    """Scores a few fp32 steps apart, saturated on either side, and biases that bring different
    logits next to each other: the order is that of the 64-bit scores."""
    rng = np.random.default_rng(7 + kind)
    cfg = _cfg(600, E=64, k=5, ng=4, tg=2)
    base = rng.standard_normal((600, 1))
    near = base + rng.integers(-3, 4, (600, 64)) * 2.0 ** -23
    check(cfg, KINDS[kind], near, None, "near")
    bias = (0.5 + rng.integers(-3, 4, 64) * 2.0 ** -24).astype(np.float32)
    check(cfg, KINDS[kind], near, bias, "near with bias")
    if KINDS[kind]["score"] == "sigmoid":
        check(cfg, KINDS[kind], 12 + 4 * rng.random((600, 64)), None, "high")
        check(cfg, KINDS[kind], -30 - 60 * rng.random((600, 64)), None, "low")
        check(cfg, KINDS[kind], -100 - 60 * rng.random((600, 64)), None, "very low")


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_non_finite(native_lib, kind):
    """Non-finite logits and biases: the status says so, their experts come last with weight 0,
    every other token is as without them."""
    rng = np.random.default_rng(kind)
    cfg, score = _cfg(260, E=32, k=4, ng=4, tg=2), KINDS[kind]
    logits = rng.standard_normal((260, 32)).astype(np.float32)
    logits[3, 5] = np.nan
    logits[4, :] = -np.inf
    logits[7, 8:] = np.inf
    logits[9, ::2] = np.nan
    for bias in (None, np.where(np.arange(32) == 6, np.nan, 0.1).astype(np.float32)):
        out, status, _ = gpu(cfg, score, logits, bias)
        assert status == -6
        o = SC.route(logits, bias, cfg, score)
        r = route_np(out)
        for key in ("expert_id", "pos", "row", "counts", "expert_offsets"):
            np.testing.assert_array_equal(r[key], o[key])
        np.testing.assert_allclose(r["gate"], o["gate"], rtol=200 * U, atol=1e-30)
        np.testing.assert_allclose([r["aux_loss"][0], r["z_loss"][0]], [o["aux_loss"], o["z_loss"]], rtol=LOSS_RTOL)


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("shift", [-1e5, -1e3, -70.0, 70.0, 1e3, 1e5])
def test_offset_of_the_logits(native_lib, kind, shift):
    """A common offset costs the weights nothing (the spread in their tolerance is the token's own)."""
    for cfg in (_cfg(200, E=64, k=4), _cfg(150, E=256, k=8, ng=8, tg=4), _cfg(1, E=5, k=2)):
        rng = np.random.default_rng(kind)
        logits = (rng.standard_normal((cfg["S"], cfg["E"])) + shift).astype(np.float32)
        check(cfg, KINDS[kind], logits, None)


@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("value", [-1e20, -1e9, 1e9, 1e20])
def test_equal_logits_of_any_size(native_lib, value, renorm):
    """Equal logits: equal softmax weights, 1 / E (or 1 / k), whatever the logits are."""
    for E, k in ((7, 3), (64, 2), (200, 8)):
        cfg, score = _cfg(33, E=E, k=k), dict(score="softmax", group_top=1, renorm=renorm, scale=1.0)
        out, status, _ = gpu(cfg, score, np.full((33, E), value), None)
        assert status == 0
        np.testing.assert_array_equal(route_np(out)["expert_id"], np.tile(np.arange(k), (33, 1)))
        np.testing.assert_allclose(route_np(out)["gate"], 1.0 / (k if renorm else E), rtol=(E + 64) * U)


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_logits_of_the_lowest_values(native_lib, kind):
    """Tokens of which every logit is hugely negative but finite (masked with the type's lowest
    value, say), between ordinary ones: no status, choices and weights of the 64-bit scores."""
    rng = np.random.default_rng(kind)
    lowest = float(np.finfo(np.float32).min)
    for cfg in (_cfg(40, E=4, k=2), _cfg(40, E=64, k=4, ng=8, tg=3), _cfg(40, E=200, k=8)):
        E = cfg["E"]
        logits = rng.standard_normal((40, E)).astype(np.float32)
        logits[0] = lowest
        logits[1] = np.resize(np.float32([-2e30, -1.5e30, -3e30, -1.5e30]), E)
        logits[2] = -1e30
        logits[3] = -1e30 * (1 + rng.random(E))
        logits[4] = lowest
        logits[4, E // 2] = -1e30
        logits[5, 1:] = lowest
        logits[6] = -2e30
        logits[6, :3] = 0.5
        for bias in (None, (0.1 * rng.standard_normal(E)).astype(np.float32)):
            out, status, _ = gpu(cfg, KINDS[kind], logits, bias)
            assert status == 0
            o, r = SC.route(logits, bias, cfg, KINDS[kind]), route_np(out)
            for key in ("expert_id", "pos", "row", "counts", "expert_offsets"):
                np.testing.assert_array_equal(r[key], o[key], err_msg=key)
            np.testing.assert_allclose(r["gate"], o["gate"], rtol=(E + 80) * U, atol=2.0 ** -126)


@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 6, 31])
def test_non_finite_bias_alone(native_lib, kind, bad, at):
    """A bias that is not finite beside finite logits is reported and takes its expert out; biases
    of any finite size are not reported."""
    rng = np.random.default_rng(kind)
    for cfg in (_cfg(1, E=32, k=4, ng=4, tg=2), _cfg(260, E=32, k=4), _cfg(200, E=160, k=8, ng=8, tg=3)):
        logits = rng.standard_normal((cfg["S"], cfg["E"])).astype(np.float32)
        bias = (0.1 * rng.standard_normal(cfg["E"])).astype(np.float32)
        bias[at] = bad
        out, status, _ = gpu(cfg, KINDS[kind], logits, bias)
        assert status == -6
        o, r = SC.route(logits, bias, cfg, KINDS[kind]), route_np(out)
        for key in ("expert_id", "pos", "row", "counts", "expert_offsets"):
            np.testing.assert_array_equal(r[key], o[key])
        np.testing.assert_allclose(r["gate"], o["gate"], rtol=(cfg["E"] + 80) * U, atol=1e-30)
        bias[at] = 3e38 if bad > 0 else -3e38
        assert gpu(cfg, KINDS[kind], logits, bias)[1] == 0


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_backward(native_lib, case, kind):
    """Element by element: each of the three terms of dlogits within 64 u of its parts (k + E terms
    in the inner sums: (E + 64 + spread) u)."""
    cfg, score = CASES[case], KINDS[kind]
    rng = np.random.default_rng(1000 + 100 * case + kind)
    S, E, k = cfg["S"], cfg["E"], cfg["k"]
    logits = (rng.standard_normal((S, E)) * 2).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    out, o, lg = check(cfg, score, logits, bias)
    dgate = rng.standard_normal((S, k)).astype(np.float32)
    dl = torch.full((S, E), float("nan"), device="cuda")
    moe.route_scored_backward(cfg, score, lg, out, torch.from_numpy(dgate).cuda(), dl, 0.7, 0.3)
    ref = SC.logit_grad(logits, cfg, score, o, dgate, 0.7, 0.3)
    q = SC.normalised(logits, score["score"])
    lse = SC.losses(logits, o["counts_routed"], cfg, score)[2]
    f = np.repeat(o["counts_routed"] / (S // cfg["G"] * k), S // cfg["G"], axis=0)
    p = np.exp(logits - lse[:, None])
    w = np.abs(o["gate_raw"])
    mag = 0.7 * E / S * q * (f + (f * q).sum(1, keepdims=True)) + 0.6 / S * np.abs(lse)[:, None] * p
    dabs = np.abs(dgate) + (np.abs(dgate) * w).sum(1, keepdims=True)
    at = np.zeros((S, E))
    np.add.at(at, (np.repeat(np.arange(S), k), o["expert_id"].ravel()), (w * dabs).ravel())
    if score["score"] == "softmax" and not score["renorm"]:
        at += p * (np.abs(dgate) * w).sum(1, keepdims=True)
    spread = float(logits.max() - logits.min())
    tol = (E + 64 + spread) * U * (mag + at) + 1e-30
    err = np.abs(dl.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), (err / tol).max()
    # without the losses, experts that were not chosen get exactly nothing (renormalised weights)
    if score["renorm"]:
        moe.route_scored_backward(cfg, score, lg, out, torch.from_numpy(dgate).cuda(), dl)
        chosen = np.zeros((S, E), bool)
        np.put_along_axis(chosen, o["expert_id"], True, axis=1)
        assert not dl.cpu().numpy()[~chosen].any()


@pytest.mark.parametrize("E", [5, 8, 40, 100, 160])
@pytest.mark.parametrize("kind", range(len(KINDS)))
@pytest.mark.parametrize("shift", [-60.0, -70.0, -74.0, -78.0, -81.0, -500.0, 70.0, 90.0])
def test_backward_of_shifted_logits(native_lib, E, kind, shift):
    """Tokens whose logits all lie far from 0, experts that fill no warp: only the experts count in
    the sums. Tolerance as above, and a step of the logsumexp more (half of one, |lse| u, is in the
    z term's own magnitude)."""
    cfg, score = _cfg(90, E=E, k=min(4, E)), KINDS[kind]
    rng = np.random.default_rng(E + kind)
    S, k = cfg["S"], cfg["k"]
    logits = (rng.standard_normal((S, E)) + shift).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    out, status, lg = gpu(cfg, score, logits, bias)
    assert status == 0
    o = SC.route(logits, bias, cfg, score)
    np.testing.assert_array_equal(route_np(out)["expert_id"], o["expert_id"])
    dgate = rng.standard_normal((S, k)).astype(np.float32)
    dl = torch.full((S, E), float("nan"), device="cuda")
    moe.route_scored_backward(cfg, score, lg, out, torch.from_numpy(dgate).cuda(), dl, 0.7, 0.3)
    ref = SC.logit_grad(logits, cfg, score, o, dgate, 0.7, 0.3)
    q = SC.normalised(logits, score["score"])
    lse = SC.losses(logits, o["counts_routed"], cfg, score)[2]
    f = np.repeat(o["counts_routed"] / (S * k), S, axis=0)
    p = np.exp(logits - lse[:, None])
    w = np.abs(o["gate_raw"])
    mag = 0.7 * E / S * q * (f + (f * q).sum(1, keepdims=True)) + 0.6 / S * np.abs(lse)[:, None] * p
    dabs = np.abs(dgate) + (np.abs(dgate) * w).sum(1, keepdims=True)
    at = np.zeros((S, E))
    np.add.at(at, (np.repeat(np.arange(S), k), o["expert_id"].ravel()), (w * dabs).ravel())
    if score["score"] == "softmax" and not score["renorm"]:
        at += p * (np.abs(dgate) * w).sum(1, keepdims=True)
    spread = float((logits.max(1) - logits.min(1)).max())
    tol = (E + 66 + spread) * U * (mag + at) + 1e-30
    err = np.abs(dl.cpu().numpy().astype(np.float64) - ref)
    assert (err <= tol).all(), (err / tol).max()


def test_repeatable_in_a_graph_and_on_another_stream(native_lib):
    cfg, score = _cfg(1500, E=256, k=8, ng=8, tg=4, cf=1.0), KINDS[2]
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((1500, 256)).astype(np.float32)
    first, _, lg = gpu(cfg, score, logits, None)
    a = route_np(first)
    ws = moe.workspace(cfg, N.MOE_WS_STEP)
    out = moe.RouteOutputs.allocate(cfg)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.route_scored(cfg, score, lg, None, out, ws, stream=side)
    side.synchronize()
    b = route_np(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.route_scored(cfg, score, lg, None, out, ws)
    for _ in range(3):
        graph.replay()
    c = route_np(out)
    R = int(a["expert_offsets"][-1])
    for f in N.ROUTE_FIELDS:
        n = R if f in ("token_of", "w_perm") else None
        np.testing.assert_array_equal(a[f][:n], b[f][:n])
        np.testing.assert_array_equal(a[f][:n], c[f][:n])


@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_chosen_by_bias_alone(native_lib, kind):
    """Biases that put experts of vanishing score in front: their renormalised weights are still
    the ratios of those scores."""
    rng = np.random.default_rng(kind)
    cfg = _cfg(70, E=64, k=4)
    logits = rng.standard_normal((70, 64)).astype(np.float32)
    logits[:, 10:20] = -95.0 - rng.random((70, 10))
    bias = np.where((np.arange(64) >= 10) & (np.arange(64) < 20), 3.0 + np.arange(64) / 64, 0.0).astype(np.float32)
    score = KINDS[kind]
    out, status, _ = gpu(cfg, score, logits, bias)
    o = SC.route(logits, bias, cfg, score)
    r = route_np(out)
    np.testing.assert_array_equal(r["expert_id"], o["expert_id"])
    # un-normalised, these scores lie below the smallest normal fp32 (2^-126)
    np.testing.assert_allclose(r["gate"], o["gate"], rtol=400 * U, atol=2.0 ** -126)


@pytest.mark.parametrize("E,k,ng,tg", [(256, 8, 8, 4), (64, 2, 0, 0), (200, 8, 8, 3), (32, 4, 0, 0)])
def test_wide_range_of_biases(native_lib, E, k, ng, tg):
    """Large, small and negative biases; scores far apart and close together in one batch."""
    rng = np.random.default_rng(E)
    cfg = _cfg(500, E=E, k=k, ng=ng, tg=tg)
    for scale in (1e-6, 1.0, 300.0):
        for shift in (-5.0, 0.0, 5.0):
            logits = rng.standard_normal((500, E)) * 2 + shift
            bias = (scale * rng.standard_normal(E)).astype(np.float32)
            check(cfg, KINDS[2], logits, bias, f"{scale} {shift}")
