"""The operators around the MoE layer in a Transformer block, and blocks made of them.

``layer_norm`` and ``linear`` (with their backward passes) are the C ABI's moe_norm_* and
moe_linear_* on torch tensors: arguments are checked here, outputs that are not given are
allocated, and nothing else happens on the host. ``MoeBlock`` and ``DenseBlock`` are the two
feed-forward halves that alternate in an MoE Transformer: x + MoE(norm(x)) and
x + W2 act(W1 norm(x)).

Matrices are 2-D CUDA tensors of float32 or bfloat16 whose columns are contiguous (any row
stride, any alignment); norm and bias parameters, row statistics and their gradients are
float32. A `stream` other than the current one is the caller's to order, as in `moe`.
"""

from __future__ import annotations

import contextlib
import ctypes
from functools import lru_cache

import torch

from . import _native as N
from . import moe
from .moe import _check, _launch

_DTYPES = {torch.float32: N.MOE_F32, torch.bfloat16: N.MOE_BF16}
_F32 = torch.float32


# The checks run on every call of a serving loop: attributes that cost little (shape, dtype, device
# number, strides), and the message only when one fails.
def _first(t, name, where):
    """Checks the matrix that the others are compared with: (shape, dtype, device number, ld)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{where}: {name} must be a 2-D tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{where}: {name} must be float32 or bfloat16, not {t.dtype}")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{where}: {name} must be on a CUDA device")
    if t.shape[1] < 1:
        raise ValueError(f"{where}: {name} has no columns")
    return t.shape, t.dtype, dev, _ld(t, name, where)


def _ld(t, name, where):
    """The row stride in elements."""
    r, c = t.shape
    s0, s1 = t.stride()
    if s1 == 1 and s0 >= c:
        return s0
    if c > 1 and s1 != 1:
        raise ValueError(f"{where}: the columns of {name} must be contiguous")
    if r > 1 and s0 < c:
        raise ValueError(f"{where}: the rows of {name} overlap (row stride {s0})")
    return max(s0, c) if r > 1 else c


def _matrix(t, name, where, shape, dt, dev):
    """Checks another matrix against a shape, type and device; returns its row stride."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype is not dt or t.get_device() != dev:
        raise ValueError(f"{where}: {name} must be a {dt} tensor of shape {tuple(shape)} on CUDA device {dev}, "
                         f"got {getattr(t, 'dtype', type(t))} {tuple(getattr(t, 'shape', ()))}")
    return _ld(t, name, where)


def _vector(t, name, where, n, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not _F32 or t.shape != (n,) or t.get_device() != dev \
            or not t.is_contiguous():
        raise ValueError(f"{where}: {name} must be a contiguous float32 tensor of {n} elements on CUDA device {dev}")


def _workspace_ok(ws, where, dev):
    if not isinstance(ws, torch.Tensor) or ws.dtype is not torch.uint8 or not ws.is_contiguous() \
            or ws.get_device() != dev:
        raise ValueError(f"{where}: ws must be a contiguous uint8 tensor on CUDA device {dev}")


def _on(stream):
    """Allocations made for a call belong to the stream that the call runs on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


@lru_cache(maxsize=None)
def _device(dev):
    return torch.device("cuda", dev)


def _new(shape, dtype, dev, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=_device(dev))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=_device(dev))


def _p(t):
    return None if t is None else t.data_ptr()


def _scratch(nbytes, dev, stream):
    """A workspace for one call: zeros in its header, the rest as the allocator left it."""
    ws = _new((nbytes,), torch.uint8, dev, stream)
    with _on(stream):
        ws[:256].zero_()
    return ws


# Argument structs by their values; the library reads them during a call only.
@lru_cache(maxsize=512)
def _norm_args(*fields):
    return ctypes.byref(N.MoeNorm(*fields))


@lru_cache(maxsize=512)
def _linear_args(*fields):
    return ctypes.byref(N.MoeLinear(*fields))


# ------------------------------------------------------------------ layer norm
def layer_norm(x, gamma, beta=None, eps=1e-5, residual=None, *, out=None, h=None, mean=None, rstd=None,
               stream=None):
    """(y, h, mean, rstd): h = x (+ residual) and y = (h - mean) * rstd * gamma (+ beta), row by
    row, rstd = 1 / sqrt(var + eps). Without a residual h is x itself, and nothing is stored."""
    w = "layer_norm"
    shape, dt, dev, ldx = _first(x, "x", w)
    T, M = shape
    ldr = M if residual is None else _matrix(residual, "residual", w, shape, dt, dev)
    _vector(gamma, "gamma", w, M, dev)
    if beta is not None:
        _vector(beta, "beta", w, M, dev)
    if out is None:
        out = _new(shape, dt, dev, stream)
    if residual is not None and h is None:
        h = _new(shape, dt, dev, stream)
    if mean is None:
        mean = _new((T,), _F32, dev, stream)
    if rstd is None:
        rstd = _new((T,), _F32, dev, stream)
    ldy = _matrix(out, "out", w, shape, dt, dev)
    ldh = M if h is None else _matrix(h, "h", w, shape, dt, dev)
    _vector(mean, "mean", w, T, dev)
    _vector(rstd, "rstd", w, T, dev)
    _launch("moe_norm_forward", x, stream, _norm_args(T, M, _DTYPES[dt], eps, ldx, ldr, ldh, ldy), x.data_ptr(),
            _p(residual), gamma.data_ptr(), _p(beta), _p(h), out.data_ptr(), mean.data_ptr(), rstd.data_ptr())
    return out, (x if h is None else h), mean, rstd


@lru_cache(maxsize=512)
def _norm_ws_bytes(T, M, dtype):
    b = N.c_size_t()
    _check(N.lib().moe_norm_workspace_bytes(_norm_args(T, M, dtype, 0.0, M, M, M, M), ctypes.byref(b)),
           "moe_norm_workspace_bytes")
    return b.value


def layer_norm_workspace(T, M, dtype=torch.bfloat16, device="cuda"):
    """A zero-filled workspace for layer_norm_backward on [T, M] matrices."""
    return torch.zeros(_norm_ws_bytes(T, M, _DTYPES[dtype]), dtype=torch.uint8, device=device)


def layer_norm_backward(dy, h, gamma, mean, rstd, dh=None, *, need_beta=True, dx=None, dgamma=None,
                        dbeta=None, ws=None, stream=None):
    """(dx, dgamma, dbeta) of layer_norm from the gradient dy of y and, when given, the gradient
    dh that reaches h on its other path; dx is the gradient of x and of the residual alike.
    dbeta is None unless need_beta."""
    w = "layer_norm_backward"
    shape, dt, dev, ldy = _first(dy, "dy", w)
    T, M = shape
    ldx = _matrix(h, "h", w, shape, dt, dev)
    ldr = M if dh is None else _matrix(dh, "dh", w, shape, dt, dev)
    _vector(gamma, "gamma", w, M, dev)
    _vector(mean, "mean", w, T, dev)
    _vector(rstd, "rstd", w, T, dev)
    if dx is None:
        dx = _new(shape, dt, dev, stream)
    with _on(stream):
        if dgamma is None:
            dgamma = torch.empty_like(gamma)
        if need_beta and dbeta is None:
            dbeta = torch.empty_like(gamma)
    if ws is None:
        ws = _scratch(_norm_ws_bytes(T, M, _DTYPES[dt]), dev, stream)
    ldh = _matrix(dx, "dx", w, shape, dt, dev)
    _vector(dgamma, "dgamma", w, M, dev)
    if dbeta is not None:
        _vector(dbeta, "dbeta", w, M, dev)
    _workspace_ok(ws, w, dev)
    _launch("moe_norm_backward", dy, stream, _norm_args(T, M, _DTYPES[dt], 0.0, ldx, ldr, ldh, ldy),
            dy.data_ptr(), h.data_ptr(), gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _p(dh), dx.data_ptr(),
            dgamma.data_ptr(), _p(dbeta), ws.data_ptr(), ws.numel())
    return dx, dgamma, dbeta


# ------------------------------------------------------------------ linear layer
@lru_cache(maxsize=512)
def _linear_ws_bytes(backward, unaligned, *fields):
    b = N.c_size_t()
    _check(N.lib().moe_linear_workspace_bytes(_linear_args(*fields), backward, unaligned, ctypes.byref(b)),
           "moe_linear_workspace_bytes")
    return b.value


def linear_workspace(T, N_out, K, dtype=torch.bfloat16, device="cuda", *, backward=True, aligned=False):
    """A zero-filled workspace for linear (and linear_backward, unless backward is False) with
    x [T, K] and W [N_out, K]. aligned: every matrix starts on a 16-byte boundary and has rows
    of a multiple of 16 bytes, so that no room is needed for copies of them."""
    n = _linear_ws_bytes(int(bool(backward)), int(not aligned), T, N_out, K, N.LIN_ACTS["silu"], _DTYPES[dtype])
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _unaligned(*ts):
    """Whether a matrix starts off a 16-byte boundary: it is copied whatever its stride."""
    return int(any(t.data_ptr() % 16 for t in ts))


def linear(x, W, bias=None, *, act="none", residual=None, save_pre=False, out=None, pre=None, ws=None,
           stream=None):
    """(y, pre): y = act(x W^T + bias) + residual for x [T, K], W [N, K], bias float32 [N],
    residual [T, N]; pre = x W^T + bias is stored when save_pre (or a buffer for it) is given,
    for linear_backward, and None otherwise. act: "none", "relu", "gelu", "gelu_tanh", "silu".
    Without ws the call allocates what it needs (256 bytes, and room for copies of bf16 operands
    on no 16-byte rows); the status word goes with it, so who wants to ask moe.device_status
    whether a wait ran out keeps a workspace of their own."""
    w = "linear"
    code = N.LIN_ACTS.get(act)
    if code is None:
        raise ValueError(f"{w}: act must be one of {sorted(N.LIN_ACTS)}, not {act!r}")
    (T, K), dt, dev, ldx = _first(x, "x", w)
    (n_out, kw), dtw, devw, ldw = _first(W, "W", w)
    if kw != K or dtw is not dt or devw != dev or n_out < 1:
        raise ValueError(f"{w}: W must be a {dt} tensor of shape (any >= 1, {K}) on CUDA device {dev}")
    shape = (T, n_out)
    if bias is not None:
        _vector(bias, "bias", w, n_out, dev)
    ldr = n_out if residual is None else _matrix(residual, "residual", w, shape, dt, dev)
    if out is None:
        out = _new(shape, dt, dev, stream)
    if save_pre and pre is None:
        pre = _new(shape, dt, dev, stream)
    if ws is None:
        ws = _scratch(_linear_ws_bytes(0, _unaligned(x, W), T, n_out, K, code, _DTYPES[dt], ldx, ldw), dev, stream)
    ldy = _matrix(out, "out", w, shape, dt, dev)
    ldp = n_out if pre is None else _matrix(pre, "pre", w, shape, dt, dev)
    _workspace_ok(ws, w, dev)
    _launch("moe_linear_forward", x, stream, _linear_args(T, n_out, K, code, _DTYPES[dt], ldx, ldw, ldy, ldr, ldp),
            x.data_ptr(), W.data_ptr(), _p(bias), _p(residual), out.data_ptr(), _p(pre), ws.data_ptr(), ws.numel())
    return out, pre


def linear_backward(dy, x, W, *, act="none", pre=None, need_x=True, need_W=True, need_bias=True, dx=None,
                    dW=None, dbias=None, ws=None, stream=None):
    """(dx, dW, dbias) of linear from dy [T, N] and the stored pre (not needed for act "none");
    dx and dW in the element type, dbias float32; None for what is not needed. The gradient
    of the residual is dy itself. ws as in linear."""
    w = "linear_backward"
    code = N.LIN_ACTS.get(act)
    if code is None:
        raise ValueError(f"{w}: act must be one of {sorted(N.LIN_ACTS)}, not {act!r}")
    (T, n_out), dt, dev, ldy = _first(dy, "dy", w)
    (tx, K), dtx, devx, ldx = _first(x, "x", w)
    if tx != T or dtx is not dt or devx != dev:
        raise ValueError(f"{w}: x must be a {dt} tensor of {T} rows on CUDA device {dev}")
    ldw = _matrix(W, "W", w, (n_out, K), dt, dev)
    if code and pre is None:
        raise ValueError(f"{w}: act {act!r} needs the forward's pre")
    ldp = n_out if pre is None else _matrix(pre, "pre", w, (T, n_out), dt, dev)
    if need_x and dx is None:
        dx = _new((T, K), dt, dev, stream)
    if need_W and dW is None:
        dW = _new((n_out, K), dt, dev, stream)
    if need_bias and dbias is None:
        dbias = _new((n_out,), _F32, dev, stream)
    if ws is None:
        ws = _scratch(_linear_ws_bytes(1, _unaligned(dy, x, W), T, n_out, K, code, _DTYPES[dt], ldx, ldw, ldy), dev,
                      stream)
    lddx = K if dx is None else _matrix(dx, "dx", w, (T, K), dt, dev)
    lddw = K if dW is None else _matrix(dW, "dW", w, (n_out, K), dt, dev)
    if dbias is not None:
        _vector(dbias, "dbias", w, n_out, dev)
    _workspace_ok(ws, w, dev)
    _launch("moe_linear_backward", dy, stream,
            _linear_args(T, n_out, K, code, _DTYPES[dt], ldx, ldw, ldy, n_out, ldp, lddx, lddw), dy.data_ptr(),
            x.data_ptr(), W.data_ptr(), _p(pre), _p(dx), _p(dW), _p(dbias), ws.data_ptr(), ws.numel())
    return dx, dW, dbias


# ------------------------------------------------------------------ blocks
def _whole_rows(t, stream):
    """t as the MoE layer reads it (by its address alone: contiguous, on a 16-byte boundary), or
    a copy of it made on the stream."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    with _on(stream):
        return t.detach().clone(memory_format=torch.contiguous_format)


class MoeBlock:
    """out = x + MoE(norm(x)): the pre-norm MoE half of a Transformer block, with the routing
    by expert scores when `score` is given (see moe.make_score). weights: those of MoeLayer,
    and "norm_gamma", "norm_beta" (float32 [M])."""

    def __init__(self, cfg: dict, weights: dict, device="cuda", score=None, eps=1e-5):
        self.layer = moe.MoeLayer(cfg, weights, device, score=score)
        c, dev = self.layer.cfg, self.layer.device
        vec = lambda n: weights[n].to(dev, torch.float32).contiguous()
        self.gamma, self.beta, self.eps = vec("norm_gamma"), vec("norm_beta"), eps
        dt = moe.torch_dtype(c)
        self.n = torch.empty((c.S, c.M), dtype=dt, device=dev)
        self.mean, self.rstd = torch.empty((2, c.S), dtype=torch.float32, device=dev).unbind(0)
        self.y = torch.empty((c.S, c.M), dtype=dt, device=dev)

    def forward(self, x, u=None, stream=None):
        layer_norm(x, self.gamma, self.beta, self.eps, out=self.n, mean=self.mean, rstd=self.rstd,
                   stream=stream)
        return self.layer.forward(self.n, u, residual=_whole_rows(x, stream), stream=stream, out=self.y)

    def enable_backward(self, weights: dict):
        self.layer.enable_backward(weights)
        c = self.layer.cfg
        self.norm_ws = layer_norm_workspace(c.S, c.M, self.n.dtype, self.layer.device)

    def backward(self, x, dy, aux_coef=0.0, z_coef=0.0, stream=None):
        """(dx, dgamma, dbeta, grads) for the last forward on x; grads holds the layer's weight
        gradients (its dx is the normalised input's)."""
        n = self.n
        for t, name in ((x, "x"), (dy, "dy")):  # the layer itself checks no shapes
            _matrix(t, name, "MoeBlock.backward", n.shape, n.dtype, n.get_device())
        dy = _whole_rows(dy, stream)
        g = self.layer.backward(n, dy, residual=False, aux_coef=aux_coef, z_coef=z_coef, stream=stream)
        dx, dgamma, dbeta = layer_norm_backward(g.dx, x, self.gamma, self.mean, self.rstd, dh=dy,
                                                ws=self.norm_ws, stream=stream)
        return dx, dgamma, dbeta, g


class DenseBlock:
    """out = x + W2 act(W1 norm(x) + b1) + b2: the dense feed-forward half of the layers without
    experts. weights: W1 [H, M], W2 [M, H] (the element type), b1, b2, norm_gamma, norm_beta
    (float32)."""

    def __init__(self, T: int, weights: dict, act="gelu", dtype=torch.bfloat16, device="cuda", eps=1e-5):
        dev = torch.device(device)
        mat = lambda n: weights[n].to(device=dev, dtype=dtype).contiguous()
        vec = lambda n: weights[n].to(dev, torch.float32).contiguous()
        self.W1, self.W2, self.b1, self.b2 = mat("W1"), mat("W2"), vec("b1"), vec("b2")
        self.gamma, self.beta, self.act, self.eps = vec("norm_gamma"), vec("norm_beta"), act, eps
        H, M = self.W1.shape
        new = lambda *s: torch.empty(s, dtype=dtype, device=dev)
        self.n, self.pre, self.a, self.y = new(T, M), new(T, H), new(T, H), new(T, M)
        self.mean, self.rstd = torch.empty((2, T), dtype=torch.float32, device=dev).unbind(0)
        self.ws1 = linear_workspace(T, H, M, dtype, dev)
        self.ws2 = linear_workspace(T, M, H, dtype, dev)
        self.norm_ws = layer_norm_workspace(T, M, dtype, dev)

    def forward(self, x, stream=None):
        layer_norm(x, self.gamma, self.beta, self.eps, out=self.n, mean=self.mean, rstd=self.rstd,
                   stream=stream)
        linear(self.n, self.W1, self.b1, act=self.act, out=self.a, pre=self.pre, ws=self.ws1, stream=stream)
        return linear(self.a, self.W2, self.b2, residual=x, out=self.y, ws=self.ws2, stream=stream)[0]

    def backward(self, x, dy, stream=None):
        """The gradients of the last forward on x: a dict of dx, W1, b1, W2, b2, norm_gamma and
        norm_beta's."""
        da, dW2, db2 = linear_backward(dy, self.a, self.W2, ws=self.ws2, stream=stream)
        dn, dW1, db1 = linear_backward(da, self.n, self.W1, act=self.act, pre=self.pre, ws=self.ws1,
                                       stream=stream)
        dx, dgamma, dbeta = layer_norm_backward(dn, x, self.gamma, self.mean, self.rstd, dh=dy,
                                                ws=self.norm_ws, stream=stream)
        return dict(dx=dx, W1=dW1, b1=db1, W2=dW2, b2=db2, norm_gamma=dgamma, norm_beta=dbeta)
