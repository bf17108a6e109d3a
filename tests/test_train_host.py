"""Refusals of the cross entropy, norm and optimiser entry points before anything is launched, and their
host-only queries: the C ABI's checks on made-up pointers, the binding's on CPU tensors and on tensors that
say that they lie on a GPU."""

import ctypes
from ctypes import c_void_p

import pytest
import torch

from test_block_host import OnDevice1
from top_gating_expert_gb300 import _native as N
from top_gating_expert_gb300 import moe, train

P = ctypes.c_void_p(1 << 20)
REF = ctypes.byref


def xent(**kw):
    d = dict(T=4, V=64, K=32, dtype=1, ignore_index=-100)
    d.update(kw)
    return N.MoeXent(**d)


def xent_bytes(L, back, un, **kw):
    b = N.c_size_t()
    assert L.moe_xent_workspace_bytes(REF(xent(**kw)), back, un, REF(b)) == 0
    return b.value


@pytest.mark.parametrize("bad", [dict(T=-1), dict(V=0), dict(K=0), dict(dtype=2), dict(ldx=31), dict(ldw=31),
                                 dict(lddx=8), dict(lddw=-1), dict(z_coef=-1.0), dict(z_coef=float("nan")),
                                 dict(z_coef=float("inf")), dict(piece=-1)])
def test_xent_refuses(native_lib, bad):
    p, b = xent(**bad), N.c_size_t()
    assert native_lib.moe_xent_workspace_bytes(REF(p), 1, 1, REF(b)) == -1
    assert native_lib.moe_xent_forward(REF(p), P, P, P, P, P, P, P, 1 << 40, None) == -1
    assert native_lib.moe_xent_backward(REF(p), P, P, P, P, P, None, 1.0, P, P, P, 1 << 40, None) == -1


@pytest.mark.parametrize("dtype", [0, 1])
def test_xent_pointers_and_workspace(native_lib, dtype):
    L, p = native_lib, xent(dtype=dtype)
    fwd, bwd = xent_bytes(L, 0, 0, dtype=dtype), xent_bytes(L, 1, 0, dtype=dtype)
    assert 256 < fwd <= bwd <= xent_bytes(L, 1, 1, dtype=dtype)
    assert L.moe_xent_workspace_bytes(REF(p), 1, 1, None) == -1 and L.moe_xent_workspace_bytes(None, 1, 1, None) == -1
    args = [P] * 6
    for i in range(6):
        a = list(args)
        a[i] = None
        assert L.moe_xent_forward(REF(p), *a, P, fwd, None) == -1
    assert L.moe_xent_forward(REF(p), *args, P, fwd - 1, None) == -3
    assert L.moe_xent_forward(REF(p), *args, None, fwd, None) == -3
    assert L.moe_xent_forward(REF(p), *args, ctypes.c_void_p((1 << 20) + 16), fwd, None) == -3
    back = lambda x=P, W=P, y=P, lse=P, dl=P, st=None, dx=P, dW=P, ws=P, n=bwd: L.moe_xent_backward(
        REF(p), x, W, y, lse, dl, st, 1.0, dx, dW, ws, n, None)
    for none in ("x", "W", "y", "lse", "dl"):
        assert back(**{none: None}) == -1
    assert back(n=300) == -3 and back(ws=None) == -3
    assert back(dx=None, dW=None, ws=None) == 0  # nothing asked for
    if dtype == 1:
        off = ctypes.c_void_p((1 << 20) + 2)
        assert L.moe_xent_forward(REF(p), off, P, P, P, P, P, P, fwd, None) == -3
        assert back(W=off) == -3
    assert L.moe_xent_forward(REF(xent(T=0)), None, None, None, None, None, None, None, 0, None) == -1  # stats
    assert L.moe_xent_backward(REF(xent(T=0)), None, None, None, None, None, None, 1.0, None, None, None, 0, None) == 0
    for big in (dict(V=(1 << 22) + 1), dict(K=(1 << 22) + 1), dict(T=(1 << 30) + 1)):
        assert L.moe_xent_forward(REF(xent(**big)), *args, P, 1 << 60, None) == -2


def test_xent_workspace_sizes(native_lib):
    """No room for the logits: a piece of d of about 512 MB, the forward far less."""
    L = native_lib
    big = dict(T=8192, V=131072, K=4096)
    assert xent_bytes(L, 0, 0, **big) <= 300 << 20
    assert xent_bytes(L, 1, 0, **big) <= (520 << 20) + 8192 * 4096 * 4 + 8192 * 16
    assert xent_bytes(L, 1, 0, T=8192, V=131072, K=4096, piece=4096) <= (70 << 20) + 8192 * 4096 * 4
    assert xent_bytes(L, 0, 0, T=1, V=32768, K=1024) <= 8192
    for T in (1 << 20, 1 << 30):  # the least piece
        assert xent_bytes(L, 1, 0, T=T, V=131072, K=64) <= T * (512 * 2 + 64 * 4 + 16) + (600 << 20)


def param(n=8, **kw):
    d = dict(p=1 << 20, g=1 << 21, copy=None, n=n, first=0, weight_decay=0.0, p_dtype=0, g_dtype=0)
    d.update(kw)
    return N.MoeParam(**d)


def adam(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.0, bits=32, seed=-1)
    d.update(kw)
    return N.MoeAdamW(**d)


def test_adamw_refuses(native_lib):
    L = native_lib
    def call(a=None, ps=(param(),), n=None, m=P, v=P, ms=None, vs=None, clock=P, norm=None, ws=P, nb=256):
        arr = (N.MoeParam * max(1, len(ps)))(*ps)
        return L.moe_adamw_step(REF(a or adam()), arr, len(ps) if n is None else n, m, v, ms, vs, clock, None, norm, ws,
                                nb, None)
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1.0),
                dict(eps=float("inf")), dict(lr=float("nan")), dict(lr=float("inf")), dict(bits=16), dict(bits=0)):
        assert call(adam(**bad)) == -1, bad
    for bad in (dict(n=-1), dict(p=None), dict(g=None), dict(p_dtype=2), dict(g_dtype=-1), dict(first=-256),
                dict(first=100), dict(weight_decay=-1.0), dict(weight_decay=float("nan"))):
        assert call(ps=(param(), param(**bad))) == -1, bad
    assert call(n=-1) == -1 and call(m=None) == -1 and call(v=None) == -1 and call(clock=None) == -1
    assert call(norm=P) == -1                       # no max_norm
    assert call(adam(bits=8)) == -1                 # no scales
    assert call(m=ctypes.c_void_p((1 << 20) + 4)) == -1
    assert call(ws=None) == -3 and call(nb=255) == -3 and call(ws=ctypes.c_void_p((1 << 20) + 8)) == -3
    assert L.moe_adamw_step(REF(adam()), None, 1, P, P, None, None, P, None, None, P, 256, None) == -1
    assert L.moe_adamw_step(None, None, 0, P, P, None, None, P, None, None, P, 256, None) == -1
    vals = lambda m=P, n=256, out=P: L.moe_adamw_values(m, P, P, P, n, out, P, None)
    assert vals(n=100) == -1 and vals(n=-256) == -1 and vals(m=None) == -1 and vals(out=None) == -1
    assert vals(n=0) == 0 and vals(out=ctypes.c_void_p((1 << 20) + 4)) == -1


def test_norm_refuses(native_lib):
    L, b = native_lib, N.c_size_t()
    assert L.moe_grad_norm_workspace_bytes(None) == -1
    assert L.moe_grad_norm_workspace_bytes(REF(b)) == 0 and b.value > 256
    arr = (N.MoeParam * 1)(param(p=None, first=3))  # p and first are not read
    assert L.moe_grad_norm(arr, 1, None, P, b.value, None) == -1
    assert L.moe_grad_norm(None, 1, P, P, b.value, None) == -1
    assert L.moe_grad_norm(arr, -1, P, P, b.value, None) == -1
    assert L.moe_grad_norm(arr, 1, P, P, b.value - 1, None) == -3
    assert L.moe_grad_norm(arr, 1, P, None, b.value, None) == -3
    for bad in (dict(g=None), dict(g_dtype=3), dict(n=-5)):
        assert L.moe_grad_norm((N.MoeParam * 1)(param(**bad)), 1, P, P, b.value, None) == -1


def there(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype).as_subclass(OnDevice1)


def test_binding_refuses(native_lib):
    x, W, y, v = there(4, 8), there(6, 8), there(4, dtype=torch.int64), there(4)
    xe, xb = train.linear_cross_entropy, train.linear_cross_entropy_backward
    cpu = torch.zeros(4, 8)
    ws = there(1 << 10, dtype=torch.uint8)
    for call in (lambda: xe(cpu, cpu, y), lambda: xe(x, there(6, 7), y), lambda: xe(x, W.bfloat16(), y),
                 lambda: xe(x, W, y.int()), lambda: xe(x, W, there(5, dtype=torch.int64)), lambda: xe(x, W, None),
                 lambda: xe(x, W, there(8, dtype=torch.int64)[::2]), lambda: xe(x, W, y, loss=there(5), lse=v, stats=there(2)),
                 lambda: xe(x, W, y, loss=v, lse=v, stats=there(3)), lambda: xe(x.half(), W.half(), y),
                 lambda: xe(x, W, y, loss=v, lse=v, stats=there(2), ws=there(9)),
                 lambda: xb(x, W, y, v), lambda: xb(x, W, y, there(3), dloss=v), lambda: xb(x, W, y, v, dloss=there(5)),
                 lambda: xb(x, W, y, v, dloss=v, dx=there(4, 7), dW=W, ws=ws),
                 lambda: xb(x, W, y, v, stats=there(1), dx=x, dW=W, ws=ws),
                 lambda: train.grad_norm([]), lambda: train.grad_norm([None]), lambda: train.grad_norm([cpu]),
                 lambda: train.grad_norm([x, cpu]), lambda: train.grad_norm([x.half()]),
                 lambda: train.grad_norm([there(4, 8)[:, ::2]]), lambda: train.grad_norm([x], out=there(2)),
                 lambda: train.grad_norm([x], out=there(1), ws=there(5)),
                 lambda: train.AdamW([]), lambda: train.AdamW([cpu]), lambda: train.AdamW([x], bits=16),
                 lambda: train.AdamW([x], seed=3), lambda: train.AdamW([x], bits=8, seed=-1),
                 lambda: train.AdamW([x], max_norm=0.0), lambda: train.AdamW([x], weight_decay=[0.0, 0.1]),
                 lambda: train.AdamW([x], copies=[None, None]), lambda: train.AdamW([x], copies=[there(4, 8)]),
                 lambda: train.AdamW([x], copies=[there(4, 7, dtype=torch.bfloat16)]),
                 lambda: train.AdamW([x, cpu]), lambda: train.AdamW([x, x]), lambda: train.AdamW([x, x[1:]]),
                 lambda: train.AdamW([x.half()]), lambda: train.AdamW([there(4, 8)[:, ::2]])):
        with pytest.raises(ValueError):
            call()


def test_calls_reach_the_library_on_the_tensors_device(native_lib, monkeypatch):
    """What the binding passes on: the device current around every call, the table's fields."""
    at, seen = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            at.append(self.dev)

        def __exit__(self, *exc):
            at.pop()

    def entry(name):
        def call(*a):
            table = None
            if name in ("moe_adamw_step", "moe_grad_norm"):
                addr, n = (a[1], a[2]) if name == "moe_adamw_step" else (a[0], a[1])
                addr = ctypes.cast(addr, c_void_p).value if isinstance(addr, bytes) else addr
                table = [N.MoeParam.from_address(addr + i * ctypes.sizeof(N.MoeParam)) for i in range(n)]
                table = [{f: getattr(t, f) for f, _ in N.MoeParam._fields_} for t in table]
            seen.append((name, at[-1], a[-1], table))
            return 0
        return call

    monkeypatch.setattr(moe, "_one_device", lambda: False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: at[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(train, "_device", lambda dev: torch.device("cpu"))
    monkeypatch.setattr(moe, "_entry", entry)
    x, W, y, v, ws = there(4, 8), there(6, 8), there(4, dtype=torch.int64), there(4), there(1 << 16, dtype=torch.uint8)
    train.linear_cross_entropy(x, W, y, loss=v, lse=there(4), stats=there(2), ws=ws)
    train.linear_cross_entropy_backward(x, W, y, v, dloss=there(4), dx=there(4, 8), dW=there(6, 8), ws=ws)
    train.grad_norm([x, None, W.bfloat16()], out=there(1), ws=ws)
    a, b, c = there(300), there(256, dtype=torch.bfloat16), there(0)
    cp = there(300, dtype=torch.bfloat16)
    monkeypatch.setattr(torch, "zeros", lambda *s, dtype=torch.float32, device=None, _z=torch.zeros:
                        _z(*s, dtype=dtype).as_subclass(OnDevice1))
    monkeypatch.setattr(torch, "tensor", lambda *s, device=None, _t=torch.tensor, **k: _t(*s, **k).as_subclass(OnDevice1))
    opt = train.AdamW([a, b, c], weight_decay=[0.1, 0.0, 0.2], copies=[cp, None, None], bits=8, seed=4)
    assert opt.m.numel() == 768 and opt.m_scale.numel() == 3 and opt.first == [0, 512, 768]
    g = [there(300, dtype=torch.bfloat16), None, there(0)]
    opt.step(g)
    assert [s[:3] for s in seen] == [(n, 1, 101) for n in ("moe_xent_forward", "moe_xent_backward", "moe_grad_norm",
                                                          "moe_adamw_step")]
    assert [(t["g"], t["n"], t["g_dtype"]) for t in seen[2][3]][0] == (x.data_ptr(), 32, 0)
    t = seen[3][3]
    assert (t[0]["p"], t[0]["g"], t[0]["copy"], t[0]["n"], t[0]["first"], t[0]["weight_decay"], t[0]["g_dtype"]) == \
        (a.data_ptr(), g[0].data_ptr(), cp.data_ptr(), 300, 0, 0.1, 1)
    assert t[1]["n"] == 0 and t[1]["g"] is None and t[1]["first"] == 512 and t[1]["p_dtype"] == 1 and t[2]["n"] == 0
    for bad in ([g[0]], [there(299), None, there(0)], [there(300)[::1], there(5), there(0)], [torch.zeros(300), 1, None]):
        with pytest.raises(ValueError):
            opt.step(bad)
    with pytest.raises(ValueError):
        opt.step(g, norm=there(1))  # no max_norm
    held, opt.params = opt.params, [a, 5, c]  # lists that were changed behind its back
    with pytest.raises(ValueError):
        opt.step(g)
    opt.params = held + [a]
    with pytest.raises(ValueError):
        opt.step(g + [None])
    opt.params = held
    with pytest.raises(ValueError):
        opt.step(g, lr=there(2))
