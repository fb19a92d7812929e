"""The example with blocks at widths that 64 does not divide."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [200, 264])
def test_runs(dim):
    from memory_lean_optimizer_gb300 import lm_example
    losses = lm_example.train(steps=3, vocab=500, dim=dim, rows=3, length=70, blocks=1)
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)


def test_without_blocks_any_width_will_do():
    from memory_lean_optimizer_gb300 import lm_example
    model = lm_example.TinyLM(300, 100)
    tokens = torch.randint(300, (2, 20), device="cuda")
    model(tokens, tokens).backward()
    assert all(bool(p.grad.isfinite().all()) for p in model.parameters())
