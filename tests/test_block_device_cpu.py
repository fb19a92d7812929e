"""A block that is moved takes its rotary plan along."""
import copy
import math

import pytest
import torch

from memory_lean_optimizer_gb300 import block


def test_a_moved_block_moves_its_plan():
    b = block.TransformerBlock(128, 2, device="cpu")
    plan, turns = b.rotary, b.rotary.turns.clone()
    assert b.to("meta") is b and b.rotary.turns.device.type == "meta" and plan.turns.device.type == "cpu"
    b.to_empty(device="cpu")             # parameters without values; the plan has its own
    assert torch.equal(b.rotary.turns, turns) and b.rotary.factor == plan.factor and b.rotary.rotary_dim == 64
    assert "turns" not in " ".join(b.state_dict()) and len(list(b.buffers())) == 0


def test_other_types_and_copies_leave_it():
    plan = block.RotaryPlan(64, interleaved=True, scaling="yarn", factor=4.0, original_length=128, device="cpu")
    m = torch.nn.ModuleList(block.TransformerBlock(128, 2, rotary=plan, device="cpu") for _ in range(2))
    m.float().double().to(torch.bfloat16).cpu()
    assert all(x.rotary is plan for x in m) and plan.turns.dtype is torch.int64
    c = copy.deepcopy(m)
    assert torch.equal(c[0].rotary.turns, plan.turns) and c[0].rotary is c[1].rotary


def test_a_plan_on_another_device():
    plan = block.RotaryPlan(48, interleaved=True, scaling="yarn", factor=4.0, original_length=128, device="cpu")
    assert plan.to("cpu") is plan
    there = plan.to("meta")
    assert there.turns.shape == plan.turns.shape and there.turns.device.type == "meta" and there.interleaved
    back = there.to("cpu")
    assert torch.equal(back.turns, plan.turns) and back.factor == plan.factor == 1 + 0.1 * math.log(4)


@pytest.mark.gpu
def test_a_block_made_on_the_host_runs_on_the_gpu():
    torch.manual_seed(0)
    b = block.TransformerBlock(128, 2, device="cpu")
    with torch.no_grad():
        b.proj.copy_(torch.randn_like(b.proj))
    x, pos = torch.randn(50, 128, device="cuda").to(torch.bfloat16), torch.arange(50, device="cuda")
    with pytest.raises((ValueError, RuntimeError)):
        b(x, pos)
    b.cuda()
    here = block.TransformerBlock(128, 2)
    here.load_state_dict(b.state_dict())
    assert torch.equal(b(x, pos), here(x, pos))
