"""The linear layer on the GPU against a 64-bit evaluation: every size class (one token, few,
many; sizes that no tile divides; rows on no 16-byte boundary), activations, residual, stored
pre-activations, gradients, in place, zero tokens, non-finite values, another stream, a graph.

Tolerance of a product of K terms: the products are exact in fp32 for bf16 inputs (and off by u
for fp32); summed in any order, by an accumulator that may truncate (2u a step), the sum is off
by at most 2 (K + 2) u sum|a||b|. An activation with slope at most 1.2 and an evaluation error of
16 u (|v| + 1) follows. bf16 gradients through an activation carry the rounding of d, 2^-8
relative a term."""

import pytest
import torch

from block_util import U, assert_within, generator, half_step, strided
from top_gating_expert_gb300 import block

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def act64(name, v):
    F = torch.nn.functional
    return {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu,
            "gelu_tanh": lambda z: F.gelu(z, approximate="tanh"), "silu": F.silu}[name](v)


def act_slope64(name, v):
    if name == "none":
        return torch.ones_like(v)
    p = v.detach().clone().requires_grad_(True)
    return torch.autograd.grad(act64(name, p).sum(), p)[0]


def check_forward(x, W, bias, act, res, got, dt):
    y, pre = got
    K = x.shape[1]
    xd, wd = x.double(), W.double()
    v = xd @ wd.t()
    s = xd.abs() @ wd.abs().t()
    if bias is not None:
        v = v + bias.double()
        s = s + bias.double().abs()
    tv = 2 * (K + 3) * U * s
    if pre is not None:
        assert_within(pre, v, tv * (1 + half_step(dt)) + half_step(dt) * v.abs() + 1e-38, "pre")
    r = act64(act, v)
    ty = 1.2 * tv + (0 if act in ("none", "relu") else 16 * U * (v.abs() + 1))
    if res is not None:
        r = r + res.double()
        ty = ty + U * (r.abs() + res.double().abs())
    assert_within(y, r, ty * (1 + half_step(dt)) + half_step(dt) * r.abs() + 1e-38, "y")


def make(T, N, K, dtype, pad, off, seed, has_bias=True):
    gen, dt = generator(seed), DT[dtype]
    x = strided(T, K, pad, off, dt, gen)
    W = strided(N, K, pad, off, dt, gen, scale=K ** -0.5)
    bias = torch.randn(N, generator=gen, device="cuda") if has_bias else None
    return gen, dt, x, W, bias


SHAPES = [(1, 1, 1), (1, 64, 64), (1, 5000, 264), (2, 128, 8), (3, 7, 5), (16, 256, 512), (17, 130, 72),
          (33, 200, 1000), (64, 1408, 2048), (65, 128, 64), (100, 100, 100), (128, 256, 192),
          (129, 257, 321), (256, 256, 256), (300, 520, 640), (777, 141, 2049), (513, 2000, 136),
          (2048, 1024, 512), (1000, 4104, 328), (1, 129, 20000), (40, 16, 9000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layout", [(0, 0), (3, 1), (8, 8)])
def test_forward(native_lib, dtype, shape, layout):
    (T, N, K), (pad, off) = shape, layout
    gen, dt, x, W, bias = make(T, N, K, dtype, pad, off, T + N + K)
    act = ACTS[(T + N + K + pad) % 5]
    res = strided(T, N, pad, off, dt, gen)
    out = strided(T, N, pad, off, dt, gen)
    pre = strided(T, N, pad, off, dt, gen)
    got = block.linear(x, W, bias, act=act, residual=res, out=out, pre=pre)
    check_forward(x, W, bias, act, res, got, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", [(1, 512, 256), (48, 512, 256), (600, 512, 256)])
def test_epilogue_parts(native_lib, dtype, act, shape):
    """Every activation with each of bias, residual and stored pre-activation left out in turn."""
    T, N, K = shape
    gen, dt, x, W, bias = make(T, N, K, dtype, 0, 0, 3)
    res = strided(T, N, 0, 0, dt, gen)
    for b, r, p in ((bias, res, True), (None, res, False), (bias, None, True), (None, None, False)):
        got = block.linear(x, W, b, act=act, residual=r, save_pre=p)
        assert (got[1] is not None) == p
        check_forward(x, W, b, act, r, got, dt)


def check_backward(dy, x, W, act, pre, got, dt, has_bias):
    dx, dW, db = got
    T, N = dy.shape
    d = dy.double()
    if act != "none":
        d = d * act_slope64(act, pre.double())
    rel = half_step(torch.bfloat16) if (dt == torch.bfloat16 and act != "none") else 0.0
    # of d itself: slopes within 16 u (|pre| + 1) (their terms reach |pre|), then the rounding
    ed = (0 if act in ("none", "relu") else 16 * U * (pre.double().abs() + 1) * dy.double().abs()) + U * d.abs()
    ed = ed + rel * d.abs() * (1 + 2 * U)
    for name, r, mag, n, err, out in (
            ("dx", d @ W.double(), d.abs() @ W.double().abs(), N, ed @ W.double().abs()
             if torch.is_tensor(ed) else 0, dx),
            ("dW", d.t() @ x.double(), d.abs().t() @ x.double().abs(), T, ed.t() @ x.double().abs(), dW)):
        t = 2 * (n + 3) * U * mag * (1 + rel) + err
        assert_within(out, r, t * (1 + half_step(dt)) + half_step(dt) * r.abs() + 1e-38, name)
    if has_bias:
        edb = (0 if act in ("none", "relu") else 16 * U * (pre.double().abs() + 1) * dy.double().abs()) + U * d.abs()
        assert_within(db, d.sum(0), (T / 8 + 512) * U * d.abs().sum(0) + edb.sum(0) + 1e-38, "dbias")
    else:
        assert db is None


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("layout", [(0, 0), (3, 1)])
def test_backward(native_lib, dtype, shape, layout):
    (T, N, K), (pad, off) = shape, layout
    gen, dt, x, W, _ = make(T, N, K, dtype, pad, off, T + N + K + 1)
    act = ACTS[(T + N + K + pad + 2) % 5]
    dy = strided(T, N, pad, off, dt, gen)
    pre = None if act == "none" else strided(T, N, pad, off, dt, gen, scale=1.5)
    dx, dW = strided(T, K, pad, off, dt, gen), strided(N, K, pad, off, dt, gen)
    got = block.linear_backward(dy, x, W, act=act, pre=pre, need_bias=(T % 2 == 1), dx=dx, dW=dW)
    check_backward(dy, x, W, act, pre, got, dt, T % 2 == 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("side", [1, 9, 16, 17, 32, 33, 64, 65])
@pytest.mark.parametrize("K", [20, 1001, 9000])
@pytest.mark.parametrize("layout", [(0, 0), (3, 1), (8, 8)])
def test_short_sides(native_lib, dtype, side, K, layout):
    """Few tokens or few outputs (and, in the backward, few inputs) against a long other side: the
    tiles along a short side, transposed or not, with K split and not."""
    pad, off = layout
    for T, N in ((side, 700), (700, side)):
        act = ACTS[(side + K + T) % 5]
        gen, dt, x, W, bias = make(T, N, K, dtype, pad, off, side + K)
        res, out, pre = (strided(T, N, pad, off, dt, gen) for _ in range(3))
        got = block.linear(x, W, bias, act=act, residual=res, out=out, pre=pre)
        check_forward(x, W, bias, act, res, got, dt)
        dy = strided(T, N, pad, off, dt, gen)
        p = None if act == "none" else got[1]
        back = block.linear_backward(dy, x, W, act=act, pre=p, need_bias=True)
        check_backward(dy, x, W, act, p, back, dt, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("act", ACTS)
def test_backward_parts(native_lib, dtype, act):
    """Each gradient alone equals the one of the whole call, bit for bit."""
    gen, dt, x, W, _ = make(500, 384, 320, dtype, 0, 0, 9)
    dy = strided(500, 384, 0, 0, dt, gen)
    pre = strided(500, 384, 0, 0, dt, gen)
    whole = block.linear_backward(dy, x, W, act=act, pre=pre)
    check_backward(dy, x, W, act, pre, whole, dt, True)
    for i, need in enumerate(("need_x", "need_W", "need_bias")):
        flags = dict(need_x=False, need_W=False, need_bias=False)
        flags[need] = True
        part = block.linear_backward(dy, x, W, act=act, pre=pre, **flags)
        assert torch.equal(part[i], whole[i])
        assert [p is None for p in part] == [j != i for j in range(3)]


def test_slopes_far_out(native_lib):
    """Activations and their slopes at large arguments, at zero and at the infinities of plain
    relu; the tanh form's cube does not spoil finite arguments."""
    v = torch.tensor([[-3e38, -1e20, -100.0, -20.0, -5.0, -0.0, 0.0, 5.0, 20.0, 100.0, 1e20, 3e38]], device="cuda")
    eye = torch.ones(1, 1, device="cuda")
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        y, _ = block.linear(v.t().contiguous(), eye, act=act)
        ref = act64(act, v.t().double())
        assert_within(y, ref, 32 * U * (ref.abs() + 1), act)
        dx, _, _ = block.linear_backward(torch.ones_like(y), v.t().contiguous(), eye, act=act,
                                         pre=v.t().contiguous())
        far = v.t().abs() > 50
        slope = torch.where(v.t() > 0, 1.0, 0.0)
        assert torch.equal(dx[far], slope[far]), act
    pre = torch.tensor([[0.0, -0.0, float("nan")]], device="cuda")
    dx, _, _ = block.linear_backward(torch.ones(1, 3, device="cuda"), torch.ones(1, 1, device="cuda"),
                                     torch.eye(3, device="cuda")[:, :1].contiguous(), act="relu", pre=pre)
    assert dx.item() == 0.0  # relu'(0) = 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [2, 40, 300])
def test_non_finite_rows_stay_in_their_rows(native_lib, dtype, T):
    gen, dt, x, W, bias = make(T, 260, 200, dtype, 0, 0, 5)
    clean, _ = block.linear(x, W, bias)
    x[T // 2, 3] = float("nan")
    x[0, 5] = float("inf")
    y, _ = block.linear(x, W, bias)
    assert torch.isnan(y[T // 2]).all()
    assert torch.equal(y[0], (clean[0] * 0 + float("inf")) * torch.sign(W[:, 5])) or T // 2 == 0
    rest = [t for t in range(T) if t not in (0, T // 2)]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_tokens(native_lib, dtype):
    dt = DT[dtype]
    x, W = torch.empty(0, 64, device="cuda", dtype=dt), torch.randn(32, 64, device="cuda").to(dt)
    y, pre = block.linear(x, W, act="gelu", save_pre=True)
    assert y.shape == pre.shape == (0, 32)
    dW = torch.full((32, 64), 3.0, device="cuda", dtype=dt)
    dx, dW2, db = block.linear_backward(y, x, W, act="gelu", pre=pre, dW=dW)
    assert dx.shape == (0, 64) and not dW2.any() and not db.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 20, 257, 1024])
def test_residual_in_place(native_lib, dtype, T):
    gen, dt, x, W, bias = make(T, 264, 320, dtype, 0, 0, 6)
    res = strided(T, 264, 0, 0, dt, gen)
    y, _ = block.linear(x, W, bias, act="silu", residual=res)
    y2, _ = block.linear(x, W, bias, act="silu", residual=res, out=res)
    assert y2 is res and torch.equal(y, y2)


def test_aligned_workspace(native_lib):
    """A workspace without room for copies serves aligned operands and refuses others."""
    from top_gating_expert_gb300 import moe
    gen, dt, x, W, bias = make(100, 256, 128, "bf16", 0, 0, 7)
    ws = block.linear_workspace(100, 256, 128, aligned=True, backward=False)
    y, _ = block.linear(x, W, bias, ws=ws)
    assert torch.equal(y, block.linear(x, W, bias)[0])
    xo = strided(100, 128, 0, 1, dt, gen)
    with pytest.raises(moe.MoeError):
        block.linear(xo, W, bias, ws=ws)
    assert moe.device_status(ws) == 0


def test_repeatable_on_another_stream_and_in_a_graph(native_lib):
    gen, dt, x, W, bias = make(1500, 768, 513, "bf16", 0, 0, 10)
    dy = strided(1500, 768, 0, 0, dt, gen)
    ws = block.linear_workspace(1500, 768, 513)

    def step(**kw):
        y, pre = block.linear(x, W, bias, act="gelu", save_pre=True, ws=ws, **kw)
        return (y, pre) + block.linear_backward(dy, x, W, act="gelu", pre=pre, ws=ws, **kw)

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = step()
    for _ in range(2):
        graph.replay()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_large_offsets(native_lib):
    """Rows more than 2^31 elements into their buffers."""
    T, N, K = 9, 64, 64
    ld = 1 << 28
    big = torch.empty(8 * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((T, K), (ld, 1))
    x.copy_(torch.randn(T, K, generator=generator(1), device="cuda"))
    W = (torch.randn(N, K, generator=generator(2), device="cuda") / 8).to(torch.bfloat16)
    y, _ = block.linear(x, W)
    check_forward(x, W, None, "none", None, (y, None), torch.bfloat16)
    gamma = torch.ones(K, device="cuda")
    n = block.layer_norm(x, gamma)[0]
    assert torch.equal(n, block.layer_norm(x.contiguous(), gamma)[0])


@pytest.mark.parametrize("T,N,K,residual", [(600, 1024, 2048, False), (20, 4096, 2048, True), (2600, 1800, 1912, True)])
def test_stalled_pipeline_reports_a_timeout(native_lib, T, N, K, residual):
    """A wait limit of 1 ns: the kernel gives up (or finishes at once), frees what it holds and
    the next call with the default limit is right."""
    from top_gating_expert_gb300 import moe
    gen, dt, x, W, bias = make(T, N, K, "bf16", 0, 0, 12)
    res = strided(T, N, 0, 0, dt, gen) if residual else None
    good, _ = block.linear(x, W, bias, residual=res)
    ws = block.linear_workspace(T, N, K)
    for _ in range(3):
        moe.set_wait_limit(ws, 1)
        block.linear(x, W, bias, residual=res, ws=ws)
        assert moe.device_status(ws) in (0, -5)
        moe.set_wait_limit(ws, 0)
        y, _ = block.linear(x, W, bias, residual=res, ws=ws)
        assert moe.device_status(ws) == 0 and torch.equal(y, good)


@pytest.mark.parametrize("shape", [(2600, 1800, 1912), (2511, 1803, 1901), (4096, 2304, 1280), (20000, 136, 2056)])
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_many_tiles(native_lib, shape, act):
    """Products whose 256 x 256 tiles fill the GPU, in both directions; ragged last tiles."""
    T, N, K = shape
    gen, dt, x, W, bias = make(T, N, K, "bf16", 0, 0, 21)
    res = strided(T, N, 0, 0, dt, gen)
    y, pre = block.linear(x, W, bias, act=act, residual=res, save_pre=True)
    check_forward(x, W, bias, act, res, (y, pre), dt)
    y2, _ = block.linear(x, W, bias, act=act, residual=res, out=res)
    assert torch.equal(y, y2)
    dy = strided(T, N, 0, 0, dt, gen)
    got = block.linear_backward(dy, x, W, act=act, pre=pre)
    check_backward(dy, x, W, act, pre, got, dt, True)


@pytest.mark.parametrize("T", [2, 70])
@pytest.mark.parametrize("off", [0, 1])
def test_copied_operands_end_with_their_rows(native_lib, T, off):
    """bf16 rows of every length up to three pieces, even and odd starts, between NaNs: the copies
    hold the rows and zeros, whatever lies beside them."""
    gen = generator(T + off)

    def between_nans(rows, cols, pad):
        full = torch.full((rows * (cols + pad) + off + 9,), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = full[off:].as_strided((rows, cols), (cols + pad, 1))
        return v.copy_(torch.randn((rows, cols), generator=gen, device="cuda"))

    for K in range(1, 26):
        for pad in (1, 2, 5):
            x, W = between_nans(T, K, pad), between_nans(9, K, pad)
            got = block.linear(x, W, save_pre=True)
            check_forward(x, W, None, "none", None, got, torch.bfloat16)
            dy = between_nans(T, 9, pad)
            dx, dW, _ = block.linear_backward(dy, x, W, need_bias=False)
            dd, xd, wd = dy.double(), x.double(), W.double()
            h = half_step(torch.bfloat16)
            for g, ref, s, n in ((dx, dd @ wd, dd.abs() @ wd.abs(), 9), (dW, dd.t() @ xd, dd.abs().t() @ xd.abs(), T)):
                assert_within(g, ref, 2 * (n + 3) * U * s * (1 + h) + h * ref.abs() + 1e-38)


@pytest.mark.parametrize("dtype,N", [("f32", 66), ("f32", 130), ("f32", 20), ("bf16", 66)])
def test_more_rows_than_a_grid_axis_has_tiles(native_lib, dtype, N):
    """65536 tiles of 128 rows and one row more, either side of the output the long one."""
    T, K = 65536 * 128 + 1, 3
    gen, dt = generator(N), DT[dtype]
    x = torch.randn((T, K), generator=gen, device="cuda").to(dt)
    W, b = torch.randn((N, K), generator=gen, device="cuda").to(dt), torch.randn(N, generator=gen, device="cuda")
    out = torch.full((T, N), float("nan"), dtype=dt, device="cuda")
    block.linear(x, W, b, act="relu", out=out)
    assert not torch.isnan(out).any()
    for at in (slice(0, 700), slice(65535 * 128 - 300, 65535 * 128 + 300), slice(T - 300, T)):
        check_forward(x[at], W, b, "relu", None, (out[at], None), dt)
    if dtype == "f32":  # dx's rows are the tokens too
        wide = torch.randn((2, N), generator=gen, device="cuda")
        dx, _, _ = block.linear_backward(x[:, :2], out, wide, need_W=False, need_bias=False, dx=out)
        for at in (slice(0, 700), slice(65535 * 128 - 300, 65535 * 128 + 300), slice(T - 300, T)):
            ref, s = x[at, :2].double() @ wide.double(), x[at, :2].double().abs() @ wide.double().abs()
            assert_within(dx[at], ref, 2 * 5 * U * s + U * ref.abs() + 1e-38)


@pytest.mark.parametrize("T,N,K,dtype,pad,off,room", [
    (1, 512, 256, "bf16", 0, 0, 0), (1, 511, 257, "bf16", 3, 1, 0), (8, 100, 300, "f32", 3, 1, 0),
    (300, 512, 256, "bf16", 0, 0, 0), (300, 512, 256, "bf16", 8, 8, 0), (300, 100, 257, "bf16", 0, 0, 400 * 264 * 2)])
def test_forward_without_a_workspace_allocates_little(native_lib, T, N, K, dtype, pad, off, room):
    """Operands on 16-byte rows, and few tokens, need the header alone; others room for their copies."""
    gen, dt, x, W, bias = make(T, N, K, dtype, pad, off, T + N)
    out = torch.empty((T, N), dtype=dt, device="cuda")
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = block.linear(x, W, bias, out=out)
    assert torch.cuda.max_memory_allocated() - before <= 512 + room + 1024 * bool(room)
    check_forward(x, W, bias, "none", None, got, dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K,pad,off", [(1, 70, 129, 3, 1), (200, 256, 512, 0, 0), (333, 130, 257, 3, 1),
                                           (64, 1408, 2048, 8, 0), (1500, 768, 513, 0, 0)])
def test_workspaces_hold_all_that_is_written(native_lib, dtype, T, N, K, pad, off):
    """A workspace of exactly the bytes asked for, arbitrary beyond its header: the bytes after it stay
    as they are and the results do not change."""
    gen, dt, x, W, bias = make(T, N, K, dtype, pad, off, T + K)
    dy, pre = strided(T, N, pad, off, dt, gen), strided(T, N, pad, off, dt, gen)

    def results(ws_of):
        y, p = block.linear(x, W, bias, act="silu", save_pre=True, ws=ws_of(0))
        return (y, p, *block.linear_backward(dy, x, W, act="silu", pre=pre, ws=ws_of(1)))

    want = results(lambda back: None)
    for stale in (0xFF, 0x3C):
        whole = []

        def ws_of(back):
            n = block.linear_workspace(T, N, K, dt, backward=bool(back)).numel()
            whole.append((torch.full((n + 8192,), stale, dtype=torch.uint8, device="cuda"), n))
            whole[-1][0][:256] = 0
            return whole[-1][0][:n]

        for a, b in zip(results(ws_of), want):
            assert torch.equal(a, b)
        for t, n in whole:
            assert bool((t[n:] == stale).all())
