"""AdamW groups of empty tensors alone: every call works and does nothing."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("states", ["u8", "fp32"])
@pytest.mark.parametrize("shapes", [[(0,)], [(0, 8), (3, 0)]])
def test_nothing_to_do(states, shapes):
    from memory_lean_optimizer_gb300 import engine, lmopt
    group = engine.AdamWGroup([torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes], states=states)
    group.step([torch.empty_like(w) for w in group.weights], dict(lr=1e-3))
    assert group.unpacked_numel() == 0
    for x in group.unpack_states() + group.unpack_states(stream=torch.cuda.Stream()):
        assert x.shape == (0,)
    assert lmopt.optim_query_nonfinite(group.handle) == 0
    group.close()
