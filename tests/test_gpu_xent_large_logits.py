"""Cross entropy of logits far from zero, up to fp32's largest: the softmax depends on their differences alone.

Each logit is one exact product of two bf16 values, and one word's lies above all others by a tenth of its
magnitude, so that the probabilities are 0 and 1: lse, loss and the gradients are exact numbers, each rounded
once (the loss is a difference of two numbers that fp32 holds)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def build(rows, vocab, power, sign, seed=0):
    """hidden [rows, 8] = (sign 2^a, 0, ...), weight [vocab, 8] = (2^b f, 0, ...), a + b = power, f in (0.5, 0.9) but
    for word `top`, whose logit is the largest."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    a = power // 2
    h = torch.zeros(rows, 8, dtype=BF, device="cuda")
    h[:, 0] = sign * 2.0 ** a
    f = torch.rand(vocab, generator=g, device="cuda") * 0.3 + 0.6
    top = vocab // 3
    f[top] = 1.0 if sign > 0 else 0.5
    w = torch.zeros(vocab, 8, dtype=BF, device="cuda")
    w[:, 0] = (f.to(BF).float() * 2.0 ** (power - a)).to(BF)
    t = torch.randint(vocab, (rows,), generator=g, device="cuda")
    t[0] = top
    return h, w, t, top


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("power", [17, 24, 30, 33, 40, 64, 100, 126, 127])
@pytest.mark.parametrize("rows,vocab", [(40, 700), (300, 1500)])
def test_differences_decide(rows, vocab, power, sign):
    from memory_lean_optimizer_gb300 import head
    h, w, t, top = build(rows, vocab, power, sign)
    loss, lse = head.xent_forward(h, w, t)
    logits = w[:, 0].double() * float(h[0, 0])
    assert float(logits[top]) == float(logits.max())
    assert torch.equal(lse, logits[top].float().expand(rows))
    assert torch.equal(loss, (logits[top] - logits[t]).float())
    dh, dw = head.xent_backward(h, w, t, lse, torch.ones(rows, device="cuda"))
    want = w[top, 0].double() - w[t, 0].double()
    assert torch.equal(dh[:, 0], want.to(BF)) and not dh[:, 1:].any()
    count = torch.zeros(vocab, dtype=torch.float64, device="cuda")
    count[top] += rows
    count -= torch.bincount(t, minlength=vocab)
    assert torch.equal(dw[:, 0], (count * float(h[0, 0])).to(BF)) and not dw[:, 1:].any()
