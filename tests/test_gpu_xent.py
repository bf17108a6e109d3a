"""The cross entropy of a linear head on the GPU against a 64-bit evaluation: every size class (one
token, few, many; sizes that no tile divides; rows on no 16-byte boundary), vocabularies in one piece
and in several, tokens without a target, targets outside of the vocabulary, gradients, zero tokens,
non-finite values, another stream, a graph.

Tolerances. A logit is a sum of K products: off by at most tl = 2 (K + 3) u sum|x||w| (block_util). An
exponential exp(l - m) = 2^(l log2 e - m log2 e): its argument is off by 2 u (|l| + |m|), the hardware's
exponential and the sums that follow (chains of at most 200 additions) by 256 u, so lse is off by at
most max tl + u (256 + 8 max|l|). Gradients: every d is off by what its logit and exponential are,
|p w| (tl + u (8 + 4 (|l| + |lse|))), bf16 by the rounding of d, 2^-8 relative, beside it; then the sum
of V (or T) products as above and the rounding of the result."""

import pytest
import torch

from block_util import U, assert_within, generator, half_step, strided
from top_gating_expert_gb300 import moe, train

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100


def make(T, V, K, dtype, pad=0, off=0, drop=0.2, scale=2.0, seed=None):
    gen, dt = generator(T + V + K if seed is None else seed), DT[dtype]
    x = strided(T, K, pad, off, dt, gen)
    W = strided(V, K, pad, off, dt, gen, scale=scale * K ** -0.5)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    y = torch.where(torch.rand(T, generator=gen, device="cuda") < drop, IGNORE, y)
    return x, W, y


def logits64(x, W):
    xd, wd = x.double(), W.double()
    return xd @ wd.t(), 2 * (x.shape[1] + 3) * U * (xd.abs() @ wd.abs().t())


def check_forward(x, W, y, z, got):
    loss, lse, stats = got
    T = x.shape[0]
    l, tl = logits64(x, W)
    ref = torch.logsumexp(l, 1)
    keep = y != IGNORE
    at = torch.where(keep, y, 0)[:, None]
    e = tl.amax(1) + U * (256 + 8 * l.abs().amax(1)) + 4 * U * ref.abs()
    assert_within(lse, ref, e, "lse")
    hit = l.gather(1, at)[:, 0]
    rl = torch.where(keep, ref - hit + z * ref * ref, 0.0)
    el = e * (1 + 2 * z * ref.abs()) + tl.gather(1, at)[:, 0] + 4 * U * (ref.abs() + hit.abs() + z * ref * ref)
    el = torch.where(keep, el, 0.0) + 1e-300
    assert_within(loss, rl, el, "loss")
    n = int(keep.sum())
    assert stats[1].item() == n
    mean = rl.sum() / max(1, n)
    assert abs(stats[0].item() - mean.item()) <= el.sum().item() / max(1, n) + 40 * U * rl.abs().sum().item() / max(1, n)
    return ref


def check_backward(x, W, y, z, lse, w, got):
    """w: every token's weight, float64 [T]."""
    dx, dW = got
    dt, V, T = x.dtype, W.shape[0], x.shape[0]
    l, tl = logits64(x, W)
    lse = lse.double()
    keep = y != IGNORE
    w = torch.where(keep, w, 0.0)
    cp = (w * (1 + 2 * z * lse))[:, None]
    p = torch.exp(l - lse[:, None]) * cp
    d = p.clone()
    d.scatter_add_(1, torch.where(keep, y, 0)[:, None], -w[:, None])
    ed = p.abs() * (tl + U * (16 + 4 * (l.abs() + lse.abs()[:, None]))) + 4 * U * d.abs()
    if dt == torch.bfloat16:
        ed = ed + half_step(dt) * (d.abs() + ed) + 1e-38
    for name, out, ref, mag, err, n in (
            ("dx", dx, lambda: d @ W.double(), lambda: d.abs() @ W.double().abs(), lambda: ed @ W.double().abs(), V),
            ("dW", dW, lambda: d.t() @ x.double(), lambda: d.abs().t() @ x.double().abs(),
             lambda: ed.t() @ x.double().abs(), T)):
        if out is None:
            continue
        r = ref()
        tol = err() + 2 * (n + 3) * U * mag()
        assert_within(out, r, tol * (1 + half_step(dt)) + half_step(dt) * r.abs() + 1e-37, name)


SHAPES = [(1, 1, 1), (1, 5, 3), (1, 1000, 64), (2, 128, 8), (3, 129, 72), (17, 300, 5), (40, 4099, 136), (64, 640, 256),
          (65, 127, 64), (100, 2000, 100), (130, 257, 321), (300, 5003, 200), (257, 1024, 1411), (1000, 9001, 328),
          (2048, 4096, 512), (700, 20011, 1024), (4097, 513, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layout", [(0, 0), (3, 1), (8, 8)])
def test_sizes(native_lib, dtype, shape, layout):
    (T, V, K), (pad, off) = shape, layout
    x, W, y = make(T, V, K, dtype, pad, off)
    z = 1e-3 if (T + V) % 2 else 0.0
    got = train.linear_cross_entropy(x, W, y, z_coef=z)
    check_forward(x, W, y, z, got)
    gen = generator(5)
    dx = strided(T, K, pad, off, x.dtype, gen)
    dW = strided(V, K, pad, off, x.dtype, gen)
    back = train.linear_cross_entropy_backward(x, W, y, got[1], stats=got[2], scale=2.0, z_coef=z, dx=dx, dW=dW)
    assert back[0] is dx and back[1] is dW
    n = max(1, int((y != IGNORE).sum()))
    check_backward(x, W, y, z, got[1], torch.full((T,), 2.0 / n, dtype=torch.float64, device="cuda"), back)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1500, 64), (48, 1281, 40), (333, 2049, 96), (1500, 5000, 264), (600, 4097, 513)])
@pytest.mark.parametrize("parts", ["x", "W", "both"])
def test_pieces(native_lib, dtype, shape, parts):
    """Several pieces of the vocabulary, each gradient alone and both; weights of the caller's, some 0."""
    T, V, K = shape
    x, W, y = make(T, V, K, dtype)
    got = train.linear_cross_entropy(x, W, y, z_coef=1e-2, piece=512)
    check_forward(x, W, y, 1e-2, got)
    dloss = torch.randn(T, generator=generator(3), device="cuda")
    dloss[::5] = 0.0
    back = train.linear_cross_entropy_backward(x, W, y, got[1], dloss=dloss, z_coef=1e-2, piece=512,
                                               need_x=parts != "W", need_W=parts != "x")
    assert (back[0] is None) == (parts == "W") and (back[1] is None) == (parts == "x")
    check_backward(x, W, y, 1e-2, got[1], dloss.double(), back)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [5, 500])
def test_gradient_by_differences(native_lib, dtype, T):
    """The mean loss along a direction in x and W, from both sides, against the gradients. Tolerance:
    the loss is smooth, its third derivative along the direction below 8 |delta l|^3; the losses' own
    error is that of the forward's test, bf16 gradients are off by 2^-8 a term."""
    V, K, h = 700, 64, 2.0 ** -5
    x, W, y = make(T, V, K, dtype)
    _, lse, stats = train.linear_cross_entropy(x, W, y, z_coef=1e-2)
    dx, dW = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, z_coef=1e-2)
    gen = generator(9)
    ux = torch.randn(x.shape, generator=gen, device="cuda").to(x.dtype).double()
    uw = (torch.randn(W.shape, generator=gen, device="cuda") * K ** -0.5).to(W.dtype).double()

    def loss(s):
        l = (x.double() + s * ux) @ (W.double() + s * uw).t()
        keep = y != IGNORE
        e = torch.logsumexp(l, 1)
        each = e - l.gather(1, torch.where(keep, y, 0)[:, None])[:, 0] + 1e-2 * e * e
        return (each * keep).sum().item() / max(1, int(keep.sum()))

    # fourth-order central differences: error of order h^4
    num = (8 * (loss(h) - loss(-h)) - (loss(2 * h) - loss(-2 * h))) / (12 * h)
    ana = ((dx.double() * ux).sum() + (dW.double() * uw).sum()).item()
    mag = ((dx.double() * ux).abs().sum() + (dW.double() * uw).abs().sum()).item()
    assert abs(num - ana) <= (2 * half_step(x.dtype) if dtype == "bf16" else 1e-4) * mag + 100 * h ** 4, (num, ana)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 70, 600])
def test_no_targets(native_lib, dtype, T):
    """Only ignored tokens, with NaN and infinities in their rows: losses 0, gradients of x 0."""
    x, W, y = make(T, 900, 128, dtype, drop=2.0)
    x[::2, 3] = float("nan")
    x[1::2, 5] = float("inf")
    loss, lse, stats = train.linear_cross_entropy(x, W, y)
    assert (loss == 0).all() and stats.tolist() == [0.0, 0.0]
    dx, dW = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats)
    assert (dx == 0).all()
    clean = torch.zeros_like(x)
    _, lse, stats = train.linear_cross_entropy(clean, W, y)
    dx, dW = train.linear_cross_entropy_backward(clean, W, y, lse, stats=stats)
    assert (dx == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 90, 700])
def test_outside_of_the_vocabulary(native_lib, dtype, T):
    x, W, y = make(T, 600, 64, dtype, drop=0.0)
    ws = train.linear_cross_entropy_workspace(T, 600, 64, x.dtype)
    good = y.clone()
    for bad in (600, -1, 1 << 40, -(1 << 40), 600 + (1 << 32)):
        y.copy_(good)
        y[1] = bad
        loss, lse, stats = train.linear_cross_entropy(x, W, y, ws=ws)
        assert moe.device_status(ws) == -7 and torch.isnan(loss[1]) and torch.isnan(stats[0])
        assert torch.isfinite(loss[0]) and torch.isfinite(loss[2:]).all()
        dx, dW = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, ws=ws)
        assert moe.device_status(ws) == -7
        y[1] = IGNORE
        want = train.linear_cross_entropy_backward(x, W, y, lse, dloss=torch.full((T,), 1.0 / T, device="cuda"), ws=ws)
        assert moe.device_status(ws) == 0
        w = torch.where(y == IGNORE, 0.0, 1.0 / T)
        check_backward(x, W, y, 0.0, lse, w.double(), (dx, dW))
        check_backward(x, W, y, 0.0, lse, w.double(), want)
    # an ignored number inside of the vocabulary, and one far outside
    for ignore in (7, 1 << 50):
        y.copy_(good)
        y[0] = ignore
        loss, lse, stats = train.linear_cross_entropy(x, W, y, ignore_index=ignore, ws=ws)
        assert loss[0] == 0 and moe.device_status(ws) == 0 and stats[1] == (y != ignore).sum()
        dx, _ = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, ignore_index=ignore, ws=ws)
        assert (dx[0] == 0).all() and moe.device_status(ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 80, 800])
def test_large_and_nonfinite_logits(native_lib, dtype, T):
    x, W, y = make(T, 1300, 64, dtype, drop=0.0, scale=2000.0)
    got = train.linear_cross_entropy(x, W, y)
    check_forward(x, W, y, 0.0, got)
    back = train.linear_cross_entropy_backward(x, W, y, got[1], stats=got[2])
    assert torch.isfinite(back[0]).all() and torch.isfinite(back[1]).all()
    x[T // 2, 7] = float("nan")
    loss, lse, stats = train.linear_cross_entropy(x, W, y)
    nan = torch.isnan(loss)
    assert nan[T // 2] and int(nan.sum()) == 1 and torch.isnan(lse[T // 2]) and torch.isnan(stats[0])
    dx, _ = train.linear_cross_entropy_backward(x, W, y, lse, dloss=torch.ones(T, device="cuda"))
    assert torch.isnan(dx[T // 2]).all() and int(torch.isnan(dx).any(1).sum()) == 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens(native_lib, dtype):
    x, W, y = torch.zeros(0, 64, dtype=DT[dtype], device="cuda"), torch.ones(40, 64, dtype=DT[dtype], device="cuda"), \
        torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse, stats = train.linear_cross_entropy(x, W, y, stats=torch.full((2,), 7.0, device="cuda"))
    assert loss.shape == (0,) and stats.tolist() == [0.0, 0.0]
    dx, dW = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats)
    assert dx.shape == (0, 64) and (dW == 0).all()


def test_offsets_beyond_32_bits(native_lib):
    """A piece of d with more than 2^31 elements, and dW rows beyond it: tokens at both ends."""
    T, V, K = 16640, 131200, 24
    x, W, y = make(T, V, K, "bf16", drop=0.99)
    y[:3] = torch.tensor([0, V - 1, V // 2], device="cuda")
    y[-3:] = torch.tensor([V - 1, 1, V - 2], device="cuda")
    loss, lse, stats = train.linear_cross_entropy(x, W, y)
    w = 1.0 / int((y != IGNORE).sum())
    dx, _ = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, piece=V, need_W=False)
    pick = torch.cat([torch.arange(64), torch.arange(T // 2, T // 2 + 64), torch.arange(T - 64, T)]).cuda()
    lw = torch.full((len(pick),), w, dtype=torch.float64, device="cuda")
    check_backward(x[pick], W, y[pick], 0.0, lse[pick], lw, (dx[pick], None))
    back = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, need_x=False)[1]
    few = (y != IGNORE).nonzero()[:, 0]  # only these have gradients
    check_backward(x[few], W, y[few], 0.0, lse[few], torch.full((len(few),), w, dtype=torch.float64, device="cuda"),
                   (None, back))


@pytest.mark.parametrize("T,V,K", [(8087, 20011, 64), (8087, 20011, 4), (6000, 30001, 8), (20000, 5121, 136)])
def test_many_tiles(native_lib, T, V, K):
    """Products of many tiles with few k-blocks, whose last columns (one by one, slower) are followed by other tiles:
    warps of a tile that run ahead of one another. Every token, several times."""
    x, W, y = make(T, V, K, "bf16")
    for _ in range(3):
        got = train.linear_cross_entropy(x, W, y, z_coef=1e-3)
        check_forward(x, W, y, 1e-3, got)
    dx, _ = train.linear_cross_entropy_backward(x, W, y, got[1], stats=got[2], z_coef=1e-3, need_W=False)
    w = torch.full((T,), 1.0 / int((y != IGNORE).sum()), dtype=torch.float64, device="cuda")
    check_backward(x, W, y, 1e-3, got[1], w, (dx, None))


@pytest.mark.parametrize("dtype,T,V,K", [("bf16", 1, 4096, 256), ("bf16", 50, 3001, 128), ("bf16", 900, 5000, 256),
                                         ("f32", 60, 1500, 64)])
def test_streams_graphs_and_repeats(native_lib, dtype, T, V, K):
    """The same bits from a repeat, two streams at once, and a graph replayed on new inputs."""
    x, W, y = make(T, V, K, dtype)
    ws = [train.linear_cross_entropy_workspace(T, V, K, x.dtype, piece=1024) for _ in range(3)]

    def both(x, y, w, stream=None, out={}):
        loss, lse, stats = train.linear_cross_entropy(x, W, y, z_coef=1e-3, ws=w, piece=1024, stream=stream)
        return loss, lse, stats, *train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, z_coef=1e-3, ws=w,
                                                                      piece=1024, stream=stream)

    want = both(x, y, ws[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [both(x, y, w, s) for w, s in zip(ws, streams)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    xs, ys = x.clone(), y.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(xs, ys, ws[2])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both(xs, ys, ws[2])
    x2, _, y2 = make(T, V, K, dtype, seed=77)
    for nx, ny in ((x2, y2), (x, y), (x2, y2)):
        xs.copy_(nx)
        ys.copy_(ny)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, both(nx, ny, ws[0])))
    assert moe.device_status(ws[0]) == 0


def test_workspace_is_what_is_asked_for(native_lib):
    """The smallest workspace that the query names, its bytes behind the header any: the same results,
    and nothing written behind it."""
    for T, V, K, dtype in ((70, 1500, 64, "bf16"), (600, 2049, 72, "bf16"), (33, 1100, 40, "f32")):
        x, W, y = make(T, V, K, dtype)
        n = train._xent_ws_bytes(1, 0, T, V, K, train._DTYPES[x.dtype], K, K, K, K, IGNORE, 0.0, 512)
        big = torch.full((n + 512,), 255, dtype=torch.uint8, device="cuda")
        ws = big[:n]
        ws[:256] = 0
        loss, lse, stats = train.linear_cross_entropy(x, W, y, piece=512, ws=ws)
        check_forward(x, W, y, 0.0, (loss, lse, stats))
        ws[256:] = 255
        back = train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, piece=512, ws=ws)
        n_y = max(1, int((y != IGNORE).sum()))
        check_backward(x, W, y, 0.0, lse, torch.full((T,), 1.0 / n_y, dtype=torch.float64, device="cuda"), back)
        assert (big[n:] == 255).all()
        with pytest.raises(moe.MoeError):  # the longer of the two needs all of it
            train.linear_cross_entropy(x, W, y, piece=512, ws=big[:n - 256])
            train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, piece=512, ws=big[:n - 256])


@pytest.mark.parametrize("T,V,K", [(600, 5000, 4096), (100, 3000, 8192), (1, 40000, 4096)])
def test_waits_that_run_out(native_lib, T, V, K):
    """With a wait limit of a nanosecond both directions report a timeout and return; with the default again the
    next calls on the same workspace give what they gave before, bit for bit."""
    x, W, y = make(T, V, K, "bf16")
    ws = train.linear_cross_entropy_workspace(T, V, K)

    def both():
        got = train.linear_cross_entropy(x, W, y, ws=ws)
        return [*got, *train.linear_cross_entropy_backward(x, W, y, got[1], stats=got[2], ws=ws)]

    want = both()
    assert moe.device_status(ws) == 0
    for _ in range(3):
        moe.set_wait_limit(ws, 1)
        train.linear_cross_entropy(x, W, y, ws=ws)
        assert moe.device_status(ws) == -5
        train.linear_cross_entropy_backward(x, W, y, want[1], stats=want[2], ws=ws)
        assert moe.device_status(ws) == -5
        moe.set_wait_limit(ws, 0)
        got = both()
        assert moe.device_status(ws) == 0
        assert all(torch.equal(a, b) for a, b in zip(got, want))
