"""Refusals of the norm, linear and scored-routing entry points, before anything is launched:
the C ABI's checks on made-up pointers and the Python binding's on CPU tensors."""

import copy
import ctypes
import pickle

import pytest
import torch

from top_gating_expert_gb300 import _native as N
from top_gating_expert_gb300 import block, moe
from top_gating_expert_gb300.inputs import preset

P = ctypes.c_void_p(1 << 20)
REF = ctypes.byref


def norm(**kw):
    d = dict(rows=4, cols=64, dtype=1, eps=1e-5, ldx=64, ldr=64, ldh=64, ldy=64)
    d.update(kw)
    return N.MoeNorm(**d)


def lin(**kw):
    d = dict(T=4, N=64, K=32, act=0, dtype=1)
    d.update(kw)
    return N.MoeLinear(**d)


@pytest.mark.parametrize("bad", [dict(rows=-1), dict(cols=0), dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(eps=float("inf")), dict(ldx=63), dict(ldr=1), dict(ldh=0), dict(ldy=-64)])
def test_norm_refuses(native_lib, bad):
    n = norm(**bad)
    b = N.c_size_t()
    assert native_lib.moe_norm_forward(REF(n), P, None, P, None, None, P, None, None, None) == -1
    assert native_lib.moe_norm_backward(REF(n), P, P, P, P, P, None, P, P, P, P, 1 << 30, None) == -1
    assert native_lib.moe_norm_workspace_bytes(REF(n), REF(b)) == -1


def test_norm_pointers_and_workspace(native_lib):
    n, b = norm(), N.c_size_t()
    L = native_lib
    assert L.moe_norm_forward(None, P, None, P, None, None, P, None, None, None) == -1
    assert L.moe_norm_forward(REF(n), None, None, P, None, None, P, None, None, None) == -1
    assert L.moe_norm_forward(REF(n), P, None, None, None, None, P, None, None, None) == -1
    assert L.moe_norm_forward(REF(n), P, None, P, None, None, None, None, None, None) == -1
    assert L.moe_norm_forward(REF(n), P, None, P, None, P, P, None, None, None) == -1  # h is y
    assert L.moe_norm_workspace_bytes(REF(n), REF(b)) == 0 and b.value > 256
    assert L.moe_norm_workspace_bytes(REF(n), None) == -1
    args = [P, P, P, P, P, None, P, P, P]
    for i in (0, 1, 2, 3, 4, 6):
        a = list(args)
        a[i] = None
        assert L.moe_norm_backward(REF(n), *a, P, b.value, None) == -1
    assert L.moe_norm_backward(REF(n), *args, P, b.value - 1, None) == -3
    assert L.moe_norm_backward(REF(n), *args, None, b.value, None) == -3
    assert L.moe_norm_backward(REF(n), *args, ctypes.c_void_p((1 << 20) + 16), b.value, None) == -3
    zero = norm(rows=0)
    assert L.moe_norm_forward(REF(zero), None, None, None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("bad", [dict(T=-1), dict(N=0), dict(K=0), dict(act=5), dict(act=-1), dict(dtype=7),
                                 dict(ldx=31), dict(ldw=8), dict(ldy=63), dict(ldr=1), dict(ldp=63), dict(lddx=31),
                                 dict(lddw=31)])
def test_linear_refuses(native_lib, bad):
    p, b = lin(**bad), N.c_size_t()
    assert native_lib.moe_linear_workspace_bytes(REF(p), 1, 1, REF(b)) == -1
    assert native_lib.moe_linear_forward(REF(p), P, P, None, None, P, None, P, 1 << 40, None) == -1
    assert native_lib.moe_linear_backward(REF(p), P, P, P, P, P, P, P, P, 1 << 40, None) == -1


@pytest.mark.parametrize("dtype", [0, 1])
def test_linear_pointers_and_workspace(native_lib, dtype):
    L, p = native_lib, lin(dtype=dtype, act=2)
    sizes = {}
    for back in (0, 1):
        for un in (0, 1):
            b = N.c_size_t()
            assert L.moe_linear_workspace_bytes(REF(p), back, un, REF(b)) == 0
            sizes[back, un] = b.value
    assert sizes[0, 0] <= sizes[0, 1] <= sizes[1, 1] and sizes[0, 0] <= sizes[1, 0] <= sizes[1, 1]
    assert L.moe_linear_workspace_bytes(REF(p), 1, 1, None) == -1
    fwd = sizes[0, 0]
    assert L.moe_linear_forward(REF(p), None, P, None, None, P, None, P, fwd, None) == -1
    assert L.moe_linear_forward(REF(p), P, None, None, None, P, None, P, fwd, None) == -1
    assert L.moe_linear_forward(REF(p), P, P, None, None, None, None, P, fwd, None) == -1
    assert L.moe_linear_forward(REF(p), P, P, None, None, P, P, P, fwd, None) == -1  # pre is y
    assert L.moe_linear_forward(REF(p), P, P, None, None, P, None, P, fwd - 1, None) == -3
    assert L.moe_linear_forward(REF(p), P, P, None, None, P, None, None, fwd, None) == -3
    if dtype == 1:  # an operand off its 16-byte boundary needs room for its copy
        off = ctypes.c_void_p((1 << 20) + 2)
        assert L.moe_linear_forward(REF(p), off, P, None, None, P, None, P, fwd, None) == -3
    bwd = sizes[1, 0]
    assert L.moe_linear_backward(REF(p), P, P, P, None, P, P, P, P, bwd, None) == -1   # no pre
    assert L.moe_linear_backward(REF(p), None, P, P, P, P, P, P, P, bwd, None) == -1
    assert L.moe_linear_backward(REF(p), P, None, P, P, P, P, P, P, bwd, None) == -1   # dW needs x
    assert L.moe_linear_backward(REF(p), P, P, None, P, P, P, P, P, bwd, None) == -1   # dx needs W
    assert L.moe_linear_backward(REF(p), P, P, P, P, P, P, P, P, bwd - 1, None) == -3
    zero = lin(T=0, dtype=dtype)
    assert L.moe_linear_forward(REF(zero), None, None, None, None, None, None, None, 0, None) == 0


def test_scored_routing_refuses(native_lib):
    L = native_lib
    c = moe.make_config(preset(2, random_routing=0))
    need = moe.workspace_bytes(c, N.MOE_WS_STEP)
    out = N.MoeRouteOut(**{f: (1 << 20) for f in N.ROUTE_FIELDS})
    good = dict(score=0, group_top=1, renorm=1, scale=1.0)
    call = lambda cfg, s, lg=P, o=out, ws=P, n=need: L.moe_route_scored(REF(cfg), REF(s) if s else None, lg, None,
                                                                       REF(o), ws, n, None)
    back = lambda cfg, s, lg=P, dg=P, dl=P, o=out: L.moe_route_scored_backward(REF(cfg), REF(s), lg, REF(o), dg, 0.0,
                                                                              0.0, dl, None)
    for bad in (dict(score=2), dict(score=-1), dict(group_top=0), dict(group_top=3), dict(renorm=2),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        s = N.MoeScore(**dict(good, **bad))
        assert call(c, s) == -1 and back(c, s) == -1
    s = N.MoeScore(**good)
    assert call(c, None) == -1 and call(c, s, lg=None) == -1
    assert call(c, s, n=need - 1) == -3 and call(c, s, ws=None) == -3
    holes = N.MoeRouteOut(**{f: (1 << 20) for f in N.ROUTE_FIELDS if f != "row"})
    assert call(c, s, o=holes) == -1 and back(c, s, o=holes) == -1
    assert back(c, s, lg=None) == -1 and back(c, s, dg=None) == -1 and back(c, s, dl=None) == -1
    for over in (dict(random_routing=1), dict(uniform_assignment=1, random_routing=0),
                 dict(gate_norm="none", random_routing=0)):
        assert call(moe.make_config(preset(2, **over)), s) == -2
    assert call(moe.make_config(preset(2, random_routing=0, k=9)), s) == -1
    lay = moe.workspace_bytes(c, N.MOE_WS_LAYER)
    assert L.moe_layer_forward_scored(REF(c), None, P, P, None, None, P, P, None, None, None, P, None, REF(out), P,
                                      lay, None) == -1
    assert L.moe_layer_forward_scored(REF(c), REF(s), P, P, None, None, P, P, None, None, None, P, None, REF(out), P,
                                      16, None) == -3


def test_binding_refuses_before_the_library(native_lib):
    cpu = torch.zeros(4, 8)
    for call in (lambda: block.layer_norm(cpu, torch.ones(8)),
                 lambda: block.layer_norm_backward(cpu, cpu, torch.ones(8), torch.ones(4), torch.ones(4)),
                 lambda: block.linear(cpu, cpu), lambda: block.linear_backward(cpu, cpu, cpu),
                 lambda: block.linear(cpu, cpu, act="tanh"), lambda: block.linear_backward(cpu, cpu, cpu, act="x"),
                 lambda: block.layer_norm(cpu[0], torch.ones(8))):
        with pytest.raises(ValueError):
            call()
    cfg = preset(2, random_routing=0)
    with pytest.raises(ValueError):
        moe.route_scored(cfg, dict(score="sigmoid"), torch.zeros(4, 4), None, None, None)
    with pytest.raises(KeyError):
        moe.make_score(dict(score="tanh"))


def test_scored_layer_refuses_other_selection_biases(native_lib):
    """The kernel reads E floats at the bias's address: other shapes, types and devices stop here."""
    c = preset(2, random_routing=0)
    call = lambda b: moe.layer_forward_scored(c, dict(score="sigmoid"), *[None] * 3, b, *[None] * 7, None, None)
    for bad in (torch.zeros(c["E"]), torch.zeros(c["E"] - 1), torch.zeros(1, c["E"]), torch.zeros(c["E"]).double(), [0.0]):
        with pytest.raises(ValueError, match="select_bias"):
            call(bad)


class OnDevice1(torch.Tensor):
    """A CPU tensor that says that it is on CUDA device 1 (nothing is launched on it)."""
    is_cuda = True

    def get_device(self):
        return 1


@pytest.mark.parametrize("current", [0, 1])
def test_launches_on_the_tensors_device(native_lib, monkeypatch, current):
    """Every call makes the tensors' device the current one around the library's call, and takes
    that device's stream."""
    at, seen = [current], []
    make = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype).as_subclass(OnDevice1)

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            at.append(self.dev)

        def __exit__(self, *exc):
            at.pop()

    monkeypatch.setattr(moe, "_one_device", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(moe, "_entry", lambda name: lambda *a: seen.append((name, at[-1], a[-1])) or 0)
    x, v, t = make(4, 8), make(8), make(4)
    W, b, ws = make(6, 8), make(6), make(1 << 16, dtype=torch.uint8)
    block.layer_norm(x, v, v, out=make(4, 8), mean=t, rstd=t)
    block.layer_norm_backward(x, x, v, t, t, dx=make(4, 8), dgamma=v, dbeta=v, ws=ws)
    block.linear(x, W, b, out=make(4, 6), ws=ws)
    block.linear_backward(make(4, 6), x, W, dx=make(4, 8), dW=make(6, 8), dbias=b, ws=ws)
    c = preset(1, random_routing=0, S=4, E=8)
    out = moe.RouteOutputs(*[make(1) for _ in N.ROUTE_FIELDS])
    moe.route_scored(c, dict(score="sigmoid"), x, v, out, ws)
    moe.route_scored_backward(c, dict(score="sigmoid"), x, out, make(4, 2), make(4, 8))
    moe.route(c, x, None, out, ws)
    moe.layer_forward_scored(c, dict(score="sigmoid"), x, x, None, v, x, x, None, None, x, x, None, out, ws)
    moe.layer_backward(c, x, x, x, x, x, x, None, None, None, x, out, ws, 0, 0.0, 0.0, moe.Grads(c, "cpu"), ws)
    moe.set_wait_limit(ws, 0)
    assert moe.device_status(ws) == 0
    assert len(seen) == 11 and {s[1:] for s in seen} == {(1, 101)}, seen
    assert at == [current]


def test_route_outputs_follow_their_tensors():
    """The struct of pointers after a field was set, resized or swapped in place; copies and pickles
    of outputs that were in use."""
    out = moe.RouteOutputs(*[torch.zeros(4) for _ in N.ROUTE_FIELDS])
    now = lambda o: [getattr(o, f).data_ptr() for f in N.ROUTE_FIELDS]
    held = lambda o: [getattr(o.struct(), f) for f in N.ROUTE_FIELDS]
    assert held(out) == now(out)
    assert out.struct() is out.struct()
    keep = out.gate
    out.gate = torch.ones(4)
    assert held(out) == now(out) and keep.data_ptr() not in held(out)
    out.row.set_(torch.ones(9))
    assert held(out) == now(out)
    out.pos.resize_(1 << 16)
    assert held(out) == now(out)
    for other in (copy.deepcopy(out), pickle.loads(pickle.dumps(out))):
        assert held(other) == now(other) and not set(now(other)) & set(now(out))
        assert torch.equal(other.gate, out.gate)
    assert held(copy.copy(out)) == now(out)
    assert held(out) == now(out)


def test_scores_are_not_shared(native_lib):
    """A score made from a dict is the caller's: changing it changes no other one and no later call."""
    d = dict(score="softmax", group_top=2, renorm=0, scale=2.5)
    a, b = moe.make_score(d), moe.make_score(d)
    a.scale = 7.0
    held = moe._score(d)._obj
    assert b.scale == 2.5 and moe.make_score(d).scale == 2.5 and held.scale == 2.5 and held.score == 1
    assert moe.make_score(a) is a and moe._score(a)._obj is a


def test_workspace_sizes(native_lib):
    """The header alone where nothing is copied or split; the norm's partials at most one an SM."""
    def linear_bytes(back, un, **kw):
        b = N.c_size_t()
        assert native_lib.moe_linear_workspace_bytes(REF(lin(**kw)), back, un, REF(b)) == 0
        return b.value

    for un in (0, 1):
        assert linear_bytes(0, un, T=1, N=14336, K=4097) == 256
        assert linear_bytes(0, un, T=8, N=14336, K=4097, dtype=0) == 256
    assert linear_bytes(0, 0, T=8192, N=14336, K=4096) == 256
    assert linear_bytes(0, 1, T=8192, N=14336, K=4096) >= 256 + 2 * 4096 * (8192 + 14336)
    b = N.c_size_t()
    for cols in (1, 64, 8192, 20000):
        n = norm(rows=1 << 20, cols=cols, ldx=cols, ldr=cols, ldh=cols, ldy=cols)
        assert native_lib.moe_norm_workspace_bytes(REF(n), REF(b)) == 0
        assert b.value <= 256 + 160 * 2 * cols * 4 + 255
