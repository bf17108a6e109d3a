"""The cross entropy of a linear head on the GPU where its parts meet: the warps of a tile that hand their column sums
to one of them, pieces of the vocabulary, the split reduction of dx, groups of tokens. Tolerances as in
test_gpu_xent.py."""

import pytest
import torch

from test_gpu_xent import check_forward, make
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
