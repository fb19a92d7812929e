"""The example that runs the norm, the loss and the optimizer together: it learns, its first loss is the one that
torch computes from the logits, and two runs agree bit for bit."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_example_learns(states):
    from memory_lean_optimizer_gb300 import lm_example
    losses = lm_example.train(steps=60, vocab=1000, dim=128, rows=8, length=256, states=states)
    # logits of unit variance over 1000 words: log 1000 + 1/2 at the start, up to the spread of a mean of 1800 rows
    assert abs(losses[0] - (math.log(1000) + 0.5)) < 0.3
    assert losses[-1] < 0.25 * losses[0]


def test_example_is_deterministic_without_atomics_of_its_own():
    """The embedding's gradient is torch's; from equal gradients on, everything is reproducible: the tail alone."""
    from memory_lean_optimizer_gb300 import head
    out = []
    for _ in range(2):
        torch.manual_seed(3)
        tail = head.LMTail(96, 700)
        h = torch.randn(300, 96, device="cuda").to(torch.bfloat16).requires_grad_()
        t = torch.randint(700, (300,), device="cuda")
        tail(h, t).backward()
        out.append([h.grad] + [p.grad for p in tail.parameters()])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_tail_equals_torch():
    """Loss and gradients of the tail against torch's layer norm, matrix product and cross entropy in fp32.  bf16
    roundings on the way (the norm's output, E, the gradients: 2^-8 each of what they round, and the
    second's and third's go through products) stay within 2^-5 of the largest gradient; the loss sees
    only the norm output's, averaged over 96 columns: 2^-8."""
    from memory_lean_optimizer_gb300 import head
    torch.manual_seed(1)
    tail = head.LMTail(96, 700)
    h = torch.randn(4, 75, 96, device="cuda").to(torch.bfloat16).requires_grad_()
    t = torch.randint(700, (4, 75), device="cuda")
    t[0, :20] = -100
    loss = tail(h, t)
    loss.backward()
    p = [x.detach().float().requires_grad_() for x in (h, tail.norm_weight, tail.norm_bias, tail.weight)]
    y = torch.nn.functional.layer_norm(p[0], (96,), p[1], p[2], 1e-5)
    ref = torch.nn.functional.cross_entropy((y @ p[3].t()).view(-1, 700), t.view(-1))
    ref.backward()
    assert abs(float(loss.detach()) - float(ref.detach())) < 2.0 ** -8
    for got, want in zip((h, tail.norm_weight, tail.norm_bias, tail.weight), p):
        assert float((got.grad.float() - want.grad).abs().max()) <= 2.0 ** -5 * float(want.grad.abs().max())


def test_frozen_parts_cost_no_gradient():
    """Autograd asks for what is needed: a frozen output matrix, frozen norm weights, a leaf hidden state without grad."""
    from memory_lean_optimizer_gb300 import head
    torch.manual_seed(2)
    h = torch.randn(50, 96, device="cuda").to(torch.bfloat16)
    t = torch.randint(700, (50,), device="cuda")
    tail = head.LMTail(96, 700)
    h.requires_grad_()
    tail(h, t).backward()
    full = [h.grad] + [p.grad for p in tail.parameters()]
    for keep in range(4):
        ps = [h] + list(tail.parameters())
        for i, p in enumerate(ps):
            p.grad = None
            p.requires_grad_(i == keep)
        tail(h, t).backward()
        for i, p in enumerate(ps):
            assert (p.grad is None) == (i != keep)
        assert torch.equal(ps[keep].grad, full[keep])


def test_no_second_derivatives():
    from memory_lean_optimizer_gb300 import head
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(head.layer_norm(x, w).pow(2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
