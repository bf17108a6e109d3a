"""The cross entropy of a linear head on the GPU where its parts meet: the warps of a tile that hand their column sums
to one of them, pieces of the vocabulary, the split reduction of dx, groups of tokens. Tolerances as in
test_gpu_xent.py."""

import pytest
import torch

from block_util import U, assert_within
from test_gpu_xent import IGNORE, check_backward, check_forward, logits64, make
from top_gating_expert_gb300 import train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,V,K", [(4103, 40001, 8), (2500, 65792, 16), (12289, 9999, 72)])
def test_handed_over_sums(native_lib, T, V, K):
    """Dozens of tiles a pair of SMs whose products are shorter than the hand-over of their sums between
    warps: two buffers in turn, each written again only when it was read. Every token, and the same bits every time."""
    x, W, y = make(T, V, K, "bf16")
    first = train.linear_cross_entropy(x, W, y)
    check_forward(x, W, y, 0.0, first)
    for _ in range(20):
        again = train.linear_cross_entropy(x, W, y)
        assert all(torch.equal(a, b) for a, b in zip(again, first))


def up(n, m):
    return -(-n // m) * m


@pytest.mark.parametrize("T,V,K,piece,parts", [
    (1024, 65000, 512, 32768, (2, 32488, 9)),  # the last piece shorter by less than a k-block
    (4800, 61456, 512, 4096, (16, 16, 2)),     # the last piece one k-block: fewer parts
    (700, 20011, 1024, 0, (1, 20011, 6))])
def test_split_reduction_of_pieces(native_lib, T, V, K, piece, parts):
    """dx summed over pieces of the vocabulary, each piece's share in parts: (pieces, entries of the last, parts)."""
    pieces, last, splits = parts
    each = (V - last) // (pieces - 1) if pieces > 1 else V
    room = up(T * up(each, 8) * 2, 256) + up(splits * T * K * 4, 256) + (up(T * K * 4, 256) if pieces > 1 else 0)
    assert train.linear_cross_entropy_workspace(T, V, K, aligned=True, piece=piece).numel() == 256 + room
    x, W, y = make(T, V, K, "bf16")
    loss, lse, stats = train.linear_cross_entropy(x, W, y, z_coef=1e-3, piece=piece)
    w = torch.full((T,), 2.0 / int((y != IGNORE).sum()), dtype=torch.float64, device="cuda")
    back = lambda **kw: train.linear_cross_entropy_backward(x, W, y, lse, stats=stats, scale=2.0, z_coef=1e-3, piece=piece,
                                                            **kw)
    dx, dW = back()
    check_backward(x, W, y, 1e-3, lse, w, (dx, dW))
    again, _ = back(need_W=False)
    assert torch.equal(again, dx)
    dloss = torch.linspace(-1.0, 1.0, T, device="cuda")
    dx, _ = train.linear_cross_entropy_backward(x, W, y, lse, dloss=dloss, z_coef=1e-3, need_W=False, piece=piece)
    check_backward(x, W, y, 1e-3, lse, dloss.double(), (dx, None))


def test_forward_in_groups_of_tokens(native_lib):
    """A vocabulary so large that the columns' sums of all tokens take more than their room: groups of 1024 tokens
    one after another, the last of 76, every token's loss and lse, and the mean over all."""
    T, V, K, z = 1100, 1 << 22, 8, 1e-3
    room = up(1024 * (V // 128) * 8, 256) + 1024 * 4 + up(up(T, 32) // 32 * 8 + 2 * 8, 256)
    assert train.linear_cross_entropy_workspace(T, V, K, backward=False, aligned=True).numel() == 256 + room
    x, W, y = make(T, V, K, "bf16")
    y[1020:1028] = torch.tensor([0, V - 1, IGNORE, 5, V - 2, IGNORE, 1, V // 2], device="cuda")
    first = train.linear_cross_entropy(x, W, y, z_coef=z)
    total, slack, n = 0.0, 0.0, int((y != IGNORE).sum())
    for a in range(0, T, 100):
        r = slice(a, a + 100)
        l, tl = logits64(x[r], W)
        ref, keep = torch.logsumexp(l, 1), y[r] != IGNORE
        at = torch.where(keep, y[r], 0)[:, None]
        e = tl.amax(1) + U * (256 + 8 * l.abs().amax(1)) + 4 * U * ref.abs()
        assert_within(first[1][r], ref, e, f"lse {a}")
        hit = l.gather(1, at)[:, 0]
        want = torch.where(keep, ref - hit + z * ref * ref, 0.0)
        el = e * (1 + 2 * z * ref.abs()) + tl.gather(1, at)[:, 0] + 4 * U * (ref.abs() + hit.abs() + z * ref * ref)
        assert_within(first[0][r], want, torch.where(keep, el, 0.0) + 1e-300, f"loss {a}")
        total, slack = total + want.sum().item(), slack + (el * keep + 40 * U * want.abs()).sum().item()
    assert first[2][1].item() == n and abs(first[2][0].item() - total / n) <= slack / n
    for _ in range(3):  # the count of finished groups starts again
        again = train.linear_cross_entropy(x, W, y, z_coef=z)
        assert all(torch.equal(p, q) for p, q in zip(again, first))
