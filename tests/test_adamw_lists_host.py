"""What AdamW's step checks of its tensors before anything is launched, on CPU tensors that say that they lie on a
GPU, the library's calls replaced by a record of them."""

import pytest
import torch

from test_block_host import OnDevice1
from top_gating_expert_gb300 import moe, train


def there(*s, dtype=torch.float32):
    return torch.zeros(s, dtype=dtype).as_subclass(OnDevice1)


@pytest.fixture
def calls(native_lib, monkeypatch):
    """The names of the library's calls, in order."""
    made = []

    def entry(name):
        def call(*a):
            made.append(name)
            return 0
        return call

    monkeypatch.setattr(moe, "_one_device", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 100 + dev, raising=False)
    monkeypatch.setattr(train, "_device", lambda dev: torch.device("cpu"))
    monkeypatch.setattr(moe, "_entry", entry)
    monkeypatch.setattr(torch, "zeros", lambda *s, dtype=torch.float32, device=None, _z=torch.zeros:
                        _z(*s, dtype=dtype).as_subclass(OnDevice1))
    monkeypatch.setattr(torch, "tensor", lambda *s, device=None, _t=torch.tensor, **k: _t(*s, **k).as_subclass(OnDevice1))
    return made


def refused_twice(opt, grads, calls, **kw):
    for _ in range(2):
        with pytest.raises(ValueError):
            opt.step(grads, **kw)
    assert "moe_adamw_step" not in calls


@pytest.mark.parametrize("new", [lambda a, b: there(200), lambda a, b: there(300, dtype=torch.float16),
                                 lambda a, b: there(20, 30)[:, ::2], lambda a, b: b[10:]],
                         ids=["shorter", "type", "strided", "overlapping"])
def test_a_refused_step_is_refused_again(calls, new):
    """A parameter's memory replaced by one that cannot be updated: every step says so, none uses its address."""
    a, b = there(300), there(310)
    opt = train.AdamW([a, b])
    opt.step([there(300), there(310)])
    assert calls == ["moe_adamw_step"]
    calls.clear()
    a.data = new(a, b)
    refused_twice(opt, [there(300), there(310)], calls)
    a.data = there(300)
    opt.step([there(300), there(310)])
    assert calls == ["moe_adamw_step"] and opt._tab["p"][0] == a.data_ptr()


def test_a_parameter_changed_in_place(calls):
    """The same memory as another tensor (transposed, shorter, of another type), a copy likewise: seen at every step."""
    a, cp = there(20, 30), there(20, 30, dtype=torch.bfloat16)
    opt = train.AdamW([a], copies=[cp])
    held = a.data
    for t, other in ((a, held.t()), (a, held[:10]), (a, held.view(torch.int32)), (cp, cp.data.t()), (cp, cp.data[:3])):
        was = t.data
        t.data = other
        assert t.data_ptr() == was.data_ptr()
        refused_twice(opt, [there(600)], calls)
        t.data = was
    opt.step([there(20, 30)])
    a.data = held.view(30, 20)  # the same elements in the same order
    opt.copies[0] = None
    opt.step([there(30, 20)])
    assert calls == ["moe_adamw_step"] * 2 and opt._tab["copy"][0] == 0


def test_gradients_of_another_shape(calls):
    """As many elements in another order are refused; a flat gradient, or a flat parameter's, has one order only."""
    a, b = there(20, 30), there(3, 4, 5)
    opt = train.AdamW([a, b])
    for ga, gb in (((30, 20), (3, 4, 5)), ((20, 30), (12, 5)), ((20, 30), (3, 5, 4)), ((1, 30, 20), (60,))):
        refused_twice(opt, [there(*ga), there(*gb)], calls)
    refused_twice(opt, [None, there(5, 4, 3)], calls)
    for ga, gb in (((20, 30), (3, 4, 5)), ((600,), (60,)), ((1, 20, 1, 30), (3, 4, 5, 1))):
        opt.step([there(*ga), there(*gb)])
    train.AdamW([there(600)]).step([there(20, 30)])
    assert calls == ["moe_adamw_step"] * 4


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_that_is_replaced(calls, bits):
    """Moments, scales and clock of another device, type or length, as a checkpoint may hold them, are refused."""
    opt = train.AdamW([there(300), there(5)], bits=bits)
    g = [there(300), there(5)]
    dt, ut = (torch.float32, torch.float32) if bits == 32 else (torch.int8, torch.uint8)
    good = dict(m=there(768, dtype=dt), v=there(768, dtype=ut), clock=there(3, dtype=torch.float64))
    bad = [("m", torch.empty(768, dtype=dt)), ("m", there(767, dtype=dt)), ("v", there(1536, dtype=ut)[::2]),
           ("v", there(768, dtype=torch.float16)), ("clock", there(3)), ("clock", there(2, dtype=torch.float64)),
           ("m", None), ("clock", [0.0, 1.0, 1.0])]
    if bits == 8:
        good.update(m_scale=there(3), v_scale=there(3))
        bad += [("m_scale", there(2)), ("v_scale", None), ("v_scale", torch.empty(3)), ("v", there(768, dtype=dt))]
    for name, t in bad:
        was = getattr(opt, name)
        setattr(opt, name, t)
        refused_twice(opt, g, calls)
        if bits == 8 and name != "clock":
            with pytest.raises(ValueError):
                opt.moments()
        setattr(opt, name, was)
    for name, t in good.items():
        setattr(opt, name, t)
    opt.step(g)
    assert calls == ["moe_adamw_step"]


def test_clipping_takes_a_norm(calls, monkeypatch):
    """With max_norm a step that is given no norm takes its own gradients' first; none without gradients."""
    opt = train.AdamW([there(300), there(5)], max_norm=1.0)
    opt.step([there(300), there(5)], norm=there(1))
    assert calls == ["moe_adamw_step"]
    calls.clear()
    monkeypatch.setattr(train, "grad_norm", lambda grads, ws, stream: calls.append("moe_grad_norm") or there(1))
    opt.step(g for g in [there(300), None])
    opt.step([None, None])
    train.AdamW([there(300)]).step([there(300)])
    assert calls == ["moe_grad_norm"] + ["moe_adamw_step"] * 3
