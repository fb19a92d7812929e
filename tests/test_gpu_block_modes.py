"""The gated MLP outside of an ordinary backward pass, on the kernels."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def inputs():
    torch.manual_seed(0)
    return [torch.randn(*s, device="cuda").to(BF) for s in ((5, 64), (192, 64), (64, 96))]


def test_forward_mode_is_refused():
    from memory_lean_optimizer_gb300 import block
    x, w1, w2 = inputs()
    for grad in (True, False):
        with torch.set_grad_enabled(grad), forward_ad.dual_level():
            dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))
            for call in (lambda: block.swiglu(dual(x)), lambda: block.gated_mlp(dual(x), w1, w2), lambda: block.gated_mlp(x, dual(w1), w2),
                         lambda: block.gated_mlp(x, w1, dual(w2))):
                with pytest.raises((NotImplementedError, RuntimeError)):
                    call()


def test_without_grad_mode_the_result_is_the_same():
    from memory_lean_optimizer_gb300 import block
    x, w1, w2 = (t.requires_grad_() for t in inputs())
    y, h = block.gated_mlp(x, w1, w2), block.swiglu(x)
    with torch.no_grad():
        a, b = block.gated_mlp(x, w1, w2), block.swiglu(x)
    assert torch.equal(a, y) and torch.equal(b, h) and not a.requires_grad and not b.requires_grad and y.requires_grad and h.requires_grad


def test_autocast():
    """Under autocast the gated MLP runs in its type, as the two linear layers around the activation would: the same as on inputs cast by
    hand, gradients in the parameters' own types."""
    from memory_lean_optimizer_gb300 import block
    a = [t.float().requires_grad_() for t in inputs()]
    b = [t.detach().clone().requires_grad_() for t in a]
    dy = torch.randn(5, 64, device="cuda").to(BF)
    with torch.autocast("cuda", BF):
        y = block.gated_mlp(*a)
        again = torch.nn.functional.linear(torch.ones(2, 64, device="cuda"), a[1])      # the weight's cast elsewhere still has its gradient
    want = block.gated_mlp(*(t.to(BF) for t in b))
    assert y.dtype == BF and torch.equal(y, want)
    y.backward(dy)
    want.backward(dy)
    for s, t in zip(a, b):
        assert s.grad.dtype == torch.float32 and torch.equal(s.grad, t.grad)
    assert again.requires_grad and bool(torch.autograd.grad(again.sum(), a[1])[0].any())
    # fp32 leaves outside, bf16 ones inside: nothing to cast
    c = inputs()
    with torch.autocast("cuda", BF):
        assert torch.equal(block.gated_mlp(*c), block.gated_mlp(*inputs()))
    with torch.autocast("cuda", torch.float16), pytest.raises(TypeError):
        block.gated_mlp(*a)
