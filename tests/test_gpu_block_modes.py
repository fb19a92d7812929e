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
