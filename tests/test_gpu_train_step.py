"""What TrainStep makes of the weights, draws and inputs that it is given."""

import pytest
import torch

from block_util import generator
from test_gpu_train import MOE, SCORE, dense_weights, moe_weights
from top_gating_expert_gb300 import block, train

pytestmark = pytest.mark.gpu


def test_masters_are_the_values_given(native_lib):
    """Blocks in bf16 made from float32 weights, as a resumed run has them: the masters are those, experts' and
    dense ones alike, and the weights that the forward reads their rounding."""
    w, x = moe_weights(MOE, 5)
    w = {n: t if t is None or not torch.is_tensor(t) or t.dtype is not torch.bfloat16 else
         t.float() * (1 + 2.0 ** -12) for n, t in w.items()}
    d = dense_weights(MOE["M"], 256, 6, torch.float32)
    head = torch.randn(1003, MOE["M"], generator=generator(7), device="cuda").bfloat16()
    blocks = [block.MoeBlock(MOE, w, score=SCORE), block.DenseBlock(MOE["S"], d)]
    before = blocks[0].forward(x).clone()
    step = train.TrainStep(blocks, [w, d], head, lr=1e-3)
    values = {f"{i}.{n}": t for i, v in enumerate((w, d)) for n, t in v.items() if torch.is_tensor(t)}
    values["head"] = head
    assert len(step.masters) == 17
    for (n, p), c in zip(step.masters, step.opt.copies):
        assert p.dtype is torch.float32 and torch.equal(p, values[n].to("cuda", torch.float32)), n
        assert c is None or torch.equal(c, p.bfloat16()), n
        assert (c is None) == (values[n].dim() == 1), n
    step.blocks[0].layer.set_weights(step._unpacked[0])
    assert torch.equal(blocks[0].forward(x), before)
