"""What closes a training step around the blocks: the loss of a linear head, the gradients' norm and
the optimiser.

``linear_cross_entropy`` and its backward are the C ABI's moe_xent_* on torch tensors (logits over a
large vocabulary that are never stored), ``grad_norm`` is moe_grad_norm and ``AdamW`` holds the
moments of a list of parameters and updates all of them in one launch (moe_adamw_*). ``TrainStep`` runs
them around a stack of blocks: one training step of a model made of this package. Matrices, types,
strides and streams as in `block`.
"""

from __future__ import annotations

import ctypes
from functools import lru_cache

import numpy as np
import torch

from . import _native as N
from . import block
from .block import _DTYPES, _F32, _device, _first, _matrix, _new, _on, _p, _scratch, _unaligned, _vector, \
    _workspace_ok
from .moe import _check, _launch


# ------------------------------------------------------------------ cross entropy of a linear head
@lru_cache(maxsize=512)
def _xent_args(*fields):
    return ctypes.byref(N.MoeXent(*fields))


@lru_cache(maxsize=512)
def _xent_ws_bytes(backward, unaligned, *fields):
    b = N.c_size_t()
    _check(N.lib().moe_xent_workspace_bytes(_xent_args(*fields), backward, unaligned, ctypes.byref(b)),
           "moe_xent_workspace_bytes")
    return b.value


def linear_cross_entropy_workspace(T, V, K, dtype=torch.bfloat16, device="cuda", *, backward=True, aligned=False,
                                   piece=0):
    """A zero-filled workspace for linear_cross_entropy (and its backward, unless backward is False)
    with x [T, K] and W [V, K]. aligned: x and W start on a 16-byte boundary and have rows of a
    multiple of 16 bytes. piece: as the calls will be given it."""
    n = _xent_ws_bytes(int(bool(backward)), int(not aligned), T, V, K, _DTYPES[dtype], 0, 0, 0, 0, 0, 0.0, piece)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _xent_checked(x, W, target, where):
    (T, K), dt, dev, ldx = _first(x, "x", where)
    (V, kw), dtw, devw, ldw = _first(W, "W", where)
    if kw != K or dtw is not dt or devw != dev or V < 1:
        raise ValueError(f"{where}: W must be a {dt} tensor of shape (any >= 1, {K}) on CUDA device {dev}")
    if not isinstance(target, torch.Tensor) or target.dtype is not torch.int64 or target.shape != (T,) \
            or target.get_device() != dev or not target.is_contiguous():
        raise ValueError(f"{where}: target must be a contiguous int64 tensor of {T} elements on CUDA device {dev}")
    return T, V, K, dt, dev, ldx, ldw


def linear_cross_entropy(x, W, target, *, ignore_index=-100, z_coef=0.0, loss=None, lse=None, stats=None, piece=0,
                         ws=None, stream=None):
    """(loss, lse, stats) of the logits x W^T for x [T, K], W [V, K] and target int64 [T]: each
    token's loss lse - logit of its target + z_coef lse^2 (0 where the target is ignore_index) and
    the logsumexp lse of its logits, float32 [T], and stats, float32 [2]: the mean loss over the
    tokens with a target, and their number. The logits are not stored. A target outside of the
    vocabulary gives a NaN loss and, in ws, the status MOE_ERR_DEVICE_DATA. piece: vocabulary entries
    at a time (0: chosen from the sizes). Outputs that are not given may share an allocation (up to 1 MB): who keeps
    stats for long and little memory gives a tensor for it, or clones it."""
    w = "linear_cross_entropy"
    T, V, K, dt, dev, ldx, ldw = _xent_checked(x, W, target, w)
    if loss is None and lse is None and stats is None:
        with _on(stream):
            loss, lse, stats = _lists().outputs(dev, N.MOE_F32, 0, T, T, 2)
    else:
        loss, lse, stats = (_new((n,), _F32, dev, stream) if t is None else t
                            for t, n in ((loss, T), (lse, T), (stats, 2)))
        _vector(loss, "loss", w, T, dev)
        _vector(lse, "lse", w, T, dev)
        _vector(stats, "stats", w, 2, dev)
    fields = (T, V, K, _DTYPES[dt], ldx, ldw, K, K, ignore_index, z_coef, piece)
    if ws is None:
        ws = _scratch(_xent_ws_bytes(0, _unaligned(x, W), *fields), dev, stream)
    _workspace_ok(ws, w, dev)
    _launch("moe_xent_forward", x, stream, _xent_args(*fields), x.data_ptr(), W.data_ptr(), target.data_ptr(),
            loss.data_ptr(), lse.data_ptr(), stats.data_ptr(), ws.data_ptr(), ws.numel())
    return loss, lse, stats


def linear_cross_entropy_backward(x, W, target, lse, *, dloss=None, stats=None, scale=1.0, ignore_index=-100,
                                  z_coef=0.0, need_x=True, need_W=True, dx=None, dW=None, piece=0, ws=None,
                                  stream=None):
    """(dx, dW) of linear_cross_entropy, in the element type: the gradient of sum(dloss * loss) for
    dloss float32 [T], or without it of scale times the mean loss, from the forward's stats. lse,
    ignore_index and z_coef as in the forward; None for what is not needed. A token without a gradient has its row of x
    in dW's sums with weight 0: the row has to be finite."""
    w = "linear_cross_entropy_backward"
    T, V, K, dt, dev, ldx, ldw = _xent_checked(x, W, target, w)
    _vector(lse, "lse", w, T, dev)
    if dloss is not None:
        _vector(dloss, "dloss", w, T, dev)
    elif stats is None:
        raise ValueError(f"{w}: dloss or the forward's stats must be given")
    else:
        _vector(stats, "stats", w, 2, dev)
    if need_x and need_W and dx is None and dW is None:
        with _on(stream):
            dx, dW = _lists().outputs(dev, _DTYPES[dt], K, T, V)
    if need_x and dx is None:
        dx = _new((T, K), dt, dev, stream)
    if need_W and dW is None:
        dW = _new((V, K), dt, dev, stream)
    lddx = K if dx is None else _matrix(dx, "dx", w, (T, K), dt, dev)
    lddw = K if dW is None else _matrix(dW, "dW", w, (V, K), dt, dev)
    fields = (T, V, K, _DTYPES[dt], ldx, ldw, lddx, lddw, ignore_index, z_coef, piece)
    if ws is None:
        ws = _scratch(_xent_ws_bytes(1, _unaligned(x, W), *fields), dev, stream)
    _workspace_ok(ws, w, dev)
    _launch("moe_xent_backward", x, stream, _xent_args(*fields), x.data_ptr(), W.data_ptr(), target.data_ptr(),
            lse.data_ptr(), _p(dloss), _p(stats), scale, _p(dx), _p(dW), ws.data_ptr(), ws.numel())
    return dx, dW


# ------------------------------------------------------------------ many tensors
_PARAM = np.dtype([("p", np.uint64), ("g", np.uint64), ("copy", np.uint64), ("n", np.int64), ("first", np.int64),
                   ("weight_decay", np.float64), ("p_dtype", np.int32), ("g_dtype", np.int32)])
_BLOCK = 256  # elements that share a scale in 8 bits; every tensor's moments start at a multiple


@lru_cache(maxsize=1)
def _lists():
    """The extension that reads lists of tensors (built beside the library)."""
    N.lib()
    try:
        from . import _lists as m
    except ImportError as e:
        raise RuntimeError("the extension _lists is not built; run `python -m top_gating_expert_gb300.build`") from e
    if m.built_for != torch.__version__:
        raise RuntimeError(f"_lists was built for torch {m.built_for}, not {torch.__version__}; run `python -m "
                           "top_gating_expert_gb300.build` again")
    return m


def _elements(t, name, where, dev):
    """Checks a tensor of a list by its elements alone: its address."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous float32 or bfloat16 tensor on CUDA device {dev}")
    return t.data_ptr()


@lru_cache(maxsize=1)
def _grad_norm_ws_bytes():
    b = N.c_size_t()
    _check(N.lib().moe_grad_norm_workspace_bytes(ctypes.byref(b)), "moe_grad_norm_workspace_bytes")
    return b.value


def grad_norm_workspace(device="cuda"):
    """A zero-filled workspace for grad_norm."""
    return torch.zeros(_grad_norm_ws_bytes(), dtype=torch.uint8, device=device)


def grad_norm(grads, *, out=None, ws=None, stream=None):
    """float32 [1]: the 2-norm of all elements of the tensors (float32 or bfloat16, contiguous; None
    is left out). Nothing is read back: AdamW.step takes it as it is."""
    w = "grad_norm"
    grads = list(grads)
    t = next((g for g in grads if g is not None), None)
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise ValueError(f"{w}: there must be a gradient, and all of them on a CUDA device")
    tab, n = _lists().gradients(grads, dev)
    if out is None:
        with _on(stream):
            out, = _lists().outputs(dev, N.MOE_F32, 0, 1)
    else:
        _vector(out, "out", w, 1, dev)
    if ws is None:
        ws = _scratch(_grad_norm_ws_bytes(), dev, stream)
    _workspace_ok(ws, w, dev)
    _launch("moe_grad_norm", out, stream, tab, n, out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


class AdamW:
    """AdamW over a list of parameters (float32 or bfloat16, contiguous), updated in place.

    bits 32 holds both moments as float32 (`m`, `v`), bits 8 as codes (int8, uint8) of blocks of 256
    elements with a float32 scale each (`m_scale`, `v_scale`); seed: None rounds to the nearest code,
    a number >= 0 at random around the value, the same way for the same seed (m and sqrt(v) keep their means; v is
    high by its root's variance, about 1 / c of itself at code c). All parameters' moments
    lie in one buffer, parameter i's from element first[i] on. weight_decay: one number or one for each
    parameter. copies: bfloat16 tensors (or None) that receive the rounded parameters, for float32
    master weights. max_norm: a step scales the gradients to at most this norm, by the norm that it is given or else by
    that of its own gradients.

    `clock` (float64 [3]: the steps made, and both betas to that power) is on the device and advanced by
    the step itself, so a captured step counts at every replay. A checkpoint is m, v, the scales and
    clock: copied into them, or put in their place as tensors of the same type and length on the same
    device. A parameter that gets no gradient keeps its moments; the bias corrections are those of the
    common clock."""

    def __init__(self, params, *, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32, seed=None,
                 copies=None, max_norm=None):
        w = "AdamW"
        self.params = list(params)
        if not self.params:
            raise ValueError(f"{w}: no parameters")
        t0 = self.params[0]
        self.dev = t0.get_device() if isinstance(t0, torch.Tensor) else -1
        if self.dev < 0:
            raise ValueError(f"{w}: the parameters must be tensors on a CUDA device")
        if bits not in (32, 8):
            raise ValueError(f"{w}: bits must be 32 or 8, not {bits!r}")
        if seed is not None and (bits != 8 or not 0 <= int(seed) < 1 << 63):
            raise ValueError(f"{w}: seed must be >= 0 and belongs to bits 8")
        if max_norm is not None and not max_norm > 0:
            raise ValueError(f"{w}: max_norm must be positive")
        n = len(self.params)
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        self.copies = [None] * n if copies is None else list(copies)
        if len(decay) != n or len(self.copies) != n:
            raise ValueError(f"{w}: weight_decay and copies must have an entry for each of the {n} parameters")
        self.lr, self.betas, self.eps, self.max_norm = lr, betas, eps, max_norm
        self.bits, self.seed = bits, -1 if seed is None else int(seed)
        self._tab = np.zeros(n, _PARAM)
        self._tab["weight_decay"] = decay
        self._tab_at = self._tab.ctypes.data
        self._n = np.array([p.numel() if isinstance(p, torch.Tensor) else 0 for p in self.params], np.int64)
        self._n_at = self._n.ctypes.data
        at = np.concatenate([[0], np.cumsum((self._n + _BLOCK - 1) // _BLOCK * _BLOCK)])
        self._tab["first"] = at[:-1]
        self.first, total = at[:-1].tolist(), int(at[-1])
        self._total = total
        self._addresses()
        z = lambda k, dt: torch.zeros(k, dtype=dt, device=_device(self.dev))
        if bits == 8:
            self.m, self.v = z(total, torch.int8), z(total, torch.uint8)
            self.m_scale, self.v_scale = z(total // _BLOCK, _F32), z(total // _BLOCK, _F32)
        else:
            self.m, self.v = z(total, _F32), z(total, _F32)
            self.m_scale = self.v_scale = None
        self.clock = torch.tensor([0.0, 1.0, 1.0], dtype=torch.float64, device=_device(self.dev))
        self.ws = z(256, torch.uint8)
        self.norm_ws = None if max_norm is None else z(_grad_norm_ws_bytes(), torch.uint8)

    def _addresses(self):
        """Reads the parameters' and copies' addresses and checks that no two overlap. The table is written when all
        of them are found right: a step that is refused is refused again."""
        w, dev, tab = "AdamW", self.dev, self._tab
        p = [_elements(t, "every parameter", w, dev) for t in self.params]
        spans = []
        for i, (t, c) in enumerate(zip(self.params, self.copies)):
            k = int(self._n[i])
            if t.numel() != k:
                raise ValueError(f"{w}: parameter {i} has {t.numel()} elements now and had {k}")
            if c is not None:
                if not isinstance(c, torch.Tensor) or c.dtype is not torch.bfloat16 or c.numel() != k \
                        or c.get_device() != dev or not c.is_contiguous():
                    raise ValueError(f"{w}: copy {i} must be a contiguous bfloat16 tensor of {k} elements on CUDA "
                                     f"device {dev}")
                spans.append((c.data_ptr(), 2 * k))
            spans.append((p[i], t.element_size() * k))
        spans = sorted(s for s in spans if s[1])
        if any(a + k > b for (a, k), (b, _) in zip(spans, spans[1:])):
            raise ValueError(f"{w}: parameters or copies overlap in memory")
        tab["p"] = p
        tab["p_dtype"] = [_DTYPES[t.dtype] for t in self.params]
        tab["copy"] = [0 if c is None else c.data_ptr() for c in self.copies]

    def step(self, grads, *, lr=None, norm=None, stream=None):
        """One step with a gradient for each parameter, of its shape or flat (None: that parameter is left as it is). lr: a
        number for this step, or a float32 CUDA tensor [1] that the device reads. With max_norm the gradients are scaled
        by min(1, max_norm / (norm + 1e-6)); norm: float32 [1], as grad_norm gives it (None: that of these gradients,
        one launch more)."""
        w, dev = "AdamW.step", self.dev
        clip = self.max_norm is not None and norm is None
        if clip:
            grads = list(grads)  # read twice
        self._state_ok()
        if _lists().step(self._tab_at, self._n_at, len(self._n), grads, self.params, self.copies, dev):
            self._addresses()  # a parameter's memory is another one now
        if norm is not None:
            _vector(norm, "norm", w, 1, dev)
            if self.max_norm is None:
                raise ValueError(f"{w}: norm given, but no max_norm to scale to")
        elif clip and any(g is not None for g in grads):
            norm = grad_norm(grads, ws=self.norm_ws, stream=stream)
        lr_dev = None
        if isinstance(lr, torch.Tensor):
            _vector(lr, "lr", w, 1, dev)
            lr_dev, lr = lr, self.lr
        lr = self.lr if lr is None else lr
        a = N.MoeAdamW(lr, self.betas[0], self.betas[1], self.eps, self.max_norm or 0.0, self.bits, self.seed)
        _launch("moe_adamw_step", self.m, stream, ctypes.byref(a), self._tab_at, len(self._n), self.m.data_ptr(),
                self.v.data_ptr(), _p(self.m_scale), _p(self.v_scale), self.clock.data_ptr(), _p(lr_dev), _p(norm),
                self.ws.data_ptr(), self.ws.numel())

    def _state_ok(self):
        """Checks what a program may have put in the place of the moments and the clock."""
        _lists().state(self.dev, self._total, self.bits, self.m, self.v, self.m_scale, self.v_scale, self.clock)

    def moments(self, stream=None):
        """(m, v) as float32 buffers: themselves with bits 32, what the codes stand for with bits 8."""
        if self.bits == 32:
            return self.m, self.v
        self._state_ok()
        with _on(stream):
            m, v = torch.empty_like(self.m, dtype=_F32), torch.empty_like(self.v, dtype=_F32)
        _launch("moe_adamw_values", m, stream, self.m.data_ptr(), self.v.data_ptr(), self.m_scale.data_ptr(),
                self.v_scale.data_ptr(), m.numel(), m.data_ptr(), v.data_ptr())
        return m, v


# ------------------------------------------------------------------ a training step
_MOE_MATRICES = ("W_g", "W_in", "W_up", "W_out", "Ws_in", "Ws_up", "Ws_out")


class TrainStep:
    """One step of training a model x -> blocks -> logits over a vocabulary: forward, the mean cross entropy
    of the head, the blocks' backward passes, clipping and AdamW.

    blocks: MoeBlock and DenseBlock objects of one number of tokens and width, weights: the dicts that each
    was made from; head: W [V, M] in the element type. bf16 matrices have float32 master weights (made from
    the dicts and the head), and the optimiser writes the bf16 ones beside them; float32 weights are trained
    where they lie. Experts' weights are packed again after every step (MoeLayer.set_weights). Matrices decay,
    norm and bias vectors do not. aux_coef, router_z: the MoE layers' balance and z-loss; z_coef: the head's.
    The other arguments are AdamW's. `masters` holds (name, tensor) of every trained weight, in the order of
    the optimiser's parameters."""

    def __init__(self, blocks, weights, head, *, aux_coef=0.0, router_z=0.0, z_coef=0.0, ignore_index=-100,
                 weight_decay=0.01, **adamw):
        if len(blocks) != len(weights):
            raise ValueError("TrainStep: a dict of weights for each block")
        self.blocks, self.head = list(blocks), head
        self.aux_coef, self.router_z, self.z_coef, self.ignore = aux_coef, router_z, z_coef, ignore_index
        self.masters, copies, decay = [], [], []

        def train(name, value, held=None, vector=False, kind=None):
            """Adds a weight: `held` is what the forward reads (None: a tensor of its own, `kind` its device and type);
            returns that. The master is the value as it was given."""
            if vector or held is not None and held.dtype is _F32:
                self.masters.append((name, held)); copies.append(None)
            else:
                dev, dt = (held.device, held.dtype) if kind is None else kind
                master = value.to(dev, _F32, copy=True).contiguous()
                low = dt is torch.bfloat16
                if low and held is None:
                    held = master.bfloat16()
                self.masters.append((name, master)); copies.append(held if low else None)
                held = held if low else master
            decay.append(0.0 if vector else weight_decay)
            return held

        self._unpacked = []  # what set_weights takes, block by block (None: a dense one)
        for i, (b, w) in enumerate(zip(self.blocks, weights)):
            at = lambda n: f"{i}.{n}"
            if isinstance(b, block.DenseBlock):
                for n, t in (("W1", b.W1), ("W2", b.W2)):
                    train(at(n), w[n], t)
                for n, t in (("b1", b.b1), ("b2", b.b2)):
                    train(at(n), None, t, vector=True)
                self._unpacked.append(None)
            else:
                kind = b.layer.device, b.n.dtype
                if not hasattr(b, "norm_ws"):
                    b.enable_backward(w)
                u = {n: train(at(n), w[n], kind=kind) for n in _MOE_MATRICES if w.get(n) is not None}
                if b.layer.bias is not None:
                    u["bias"] = train(at("bias"), None, b.layer.bias, vector=True)
                if b.layer.select_bias is not None:
                    u["select_bias"] = b.layer.select_bias
                b.layer.set_weights(u)  # what a step would refuse is refused here, and the layer's are the dict's
                self._unpacked.append(u)
            for n, t in (("norm_gamma", b.gamma), ("norm_beta", b.beta)):
                train(at(n), None, t, vector=True)
        train("head", head, head)
        self.dx = None
        self.opt = AdamW([t for _, t in self.masters], weight_decay=decay, copies=copies, **adamw)
        T, M = self.blocks[0].n.shape if self.blocks else (0, head.shape[1])
        # room for copies only where the head starts on no 16-byte boundary (a block's output does not)
        self.ws = linear_cross_entropy_workspace(T, head.shape[0], M, head.dtype, head.device,
                                                 aligned=head.data_ptr() % 16 == 0) if self.blocks else None

    def gradients(self, x, target, u=None):
        """(stats, gradients): the head's stats (see linear_cross_entropy) and a gradient for each of `masters`, of its shape.
        u: the draws for blocks with random routing, a tensor that all of them read or a list with an entry for each block
        (None for those without). The gradient of x itself is in `dx` afterwards, for what stands in
        front of the blocks (an embedding)."""
        inputs = []
        draws = u if isinstance(u, (list, tuple)) else [u] * len(self.blocks)
        if len(draws) != len(self.blocks):
            raise ValueError(f"TrainStep: draws for {len(draws)} of {len(self.blocks)} blocks")
        for b, d in zip(self.blocks, draws):
            inputs.append(x)
            if isinstance(b, block.DenseBlock):
                x = b.forward(x)
            else:
                x = b.forward(x, d if b.layer.cfg.random_routing else None)
        _, lse, stats = linear_cross_entropy(x, self.head, target, ignore_index=self.ignore, z_coef=self.z_coef,
                                             ws=self.ws)
        dx, dhead = linear_cross_entropy_backward(x, self.head, target, lse, stats=stats, ignore_index=self.ignore,
                                                  z_coef=self.z_coef, ws=self.ws)
        found = [[dhead]]
        for b, x in zip(reversed(self.blocks), reversed(inputs)):
            if isinstance(b, block.DenseBlock):
                g = b.backward(x, dx)
                dx = g["dx"]
                found.append([g[n] for n in ("W1", "W2", "b1", "b2", "norm_gamma", "norm_beta")])
                continue
            dx, dgamma, dbeta, g = b.backward(x, dx, aux_coef=self.aux_coef, z_coef=self.router_z)
            c = b.layer.cfg
            got = [getattr(g, "d" + n) for n in _MOE_MATRICES]
            if c.n_shared > 1:  # the shared experts' hidden units lie side by side
                got[-1] = got[-1].view(c.M, c.n_shared, c.H_shared).transpose(0, 1).contiguous()
            found.append([t for t in (*got, g.dbias) if t is not None] + [dgamma, dbeta])
        self.dx = dx
        grads = [t for part in reversed(found) for t in part]
        return stats, [t if t.shape == p.shape else t.view(p.shape) for t, (_, p) in zip(grads, self.masters)]

    def step(self, x, target, u=None, lr=None):
        """One step; returns the stats of its forward (float32 [2], on the device)."""
        stats, grads = self.gradients(x, target, u)
        self.opt.step(grads, lr=lr)
        for b, w in zip(self.blocks, self._unpacked):
            if w is not None:
                b.layer.set_weights(w)
        return stats
