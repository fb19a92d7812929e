"""What the autograd side of the transformer block's operators does outside of an ordinary backward pass.  The kernels' calls are
replaced by torch formulas on the host, so that no GPU is needed."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

from memory_lean_optimizer_gb300 import block


@pytest.fixture
def on_host(monkeypatch):
    """The kernels' calls of the gated MLP as formulas that, like the kernels, write into new memory; returns the list of calls."""
    calls = []

    def swiglu_forward(gate_up, keep=True):
        calls.append("swiglu_keep" if keep else "swiglu")
        n = gate_up.shape[-1] // 2
        with torch.no_grad():
            h = torch.empty(*gate_up.shape[:-1], n).copy_(torch.nn.functional.silu(gate_up[..., :n]) * gate_up[..., n:])
        shape = torch.Size((*gate_up.shape[:-1], 2, n))
        return h, block.PackedActivation._of(torch.zeros(1, dtype=torch.uint8), shape, gate_up.dtype) if keep else None

    def pack_activation(x):
        calls.append("pack")
        return block.PackedActivation._of(torch.zeros(1, dtype=torch.uint8), x.shape, x.dtype)
    monkeypatch.setattr(block, "swiglu_forward", swiglu_forward)
    monkeypatch.setattr(block, "pack_activation", pack_activation)
    return calls


@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(on_host, grad):
    """A result without its tangent would be a wrong derivative: the calls raise, as layer_norm's and attention's do.  Without grad mode
    too, for that does not end forward mode."""
    x, w1, w2 = torch.randn(3, 4), torch.randn(16, 4), torch.randn(4, 8)
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        dual = lambda t: forward_ad.make_dual(t, torch.ones_like(t))
        for call in (lambda: block.swiglu(dual(torch.randn(3, 16))), lambda: block.gated_mlp(dual(x), w1, w2), lambda: block.gated_mlp(x, dual(w1), w2),
                     lambda: block.gated_mlp(x, w1, dual(w2))):
            with pytest.raises((NotImplementedError, RuntimeError)):
                call()
        # what carries no tangent runs
        assert block.swiglu(torch.randn(3, 16)).shape == (3, 8) and block.gated_mlp(x, w1, w2).shape == (3, 4)


@pytest.mark.parametrize("needs", [(), (0,), (1,), (2,), (0, 1, 2)])
def test_only_what_a_backward_pass_needs_is_packed(on_host, needs):
    """gated_mlp keeps gate and up if any input wants a gradient, x if w_in does; nothing without grad mode or without such an input."""
    ts = [t.requires_grad_(i in needs) for i, t in enumerate((torch.randn(3, 4), torch.randn(16, 4), torch.randn(4, 8)))]
    y = block.gated_mlp(*ts)
    assert on_host == (["swiglu_keep"] if needs else ["swiglu"]) + (["pack"] if 1 in needs else [])
    assert y.requires_grad == bool(needs)
    on_host.clear()
    with torch.no_grad():
        block.gated_mlp(*ts)
    assert on_host == ["swiglu"]
