"""The heads that the example's blocks get: what a block accepts, for every width that it can accept at all."""
import pytest


@pytest.mark.parametrize("dim,heads,kv", [(64, 1, 1), (128, 2, 1), (256, 4, 2), (512, 8, 4), (96, 1, 1), (192, 3, 3), (264, 3, 3), (200, 5, 5), (8, 1, 1),
                                          (136, 17, 17)])
def test_heads_of_a_width(dim, heads, kv):
    from memory_lean_optimizer_gb300 import lm_example
    assert lm_example.block_heads(dim) == (heads, kv)


def test_every_width_that_a_block_accepts():
    from memory_lean_optimizer_gb300 import block, lm_example
    for dim in range(8, 1025, 8):
        heads, kv = lm_example.block_heads(dim)
        if dim <= 264:
            block.TransformerBlock(dim, heads, kv, hidden=8, device="cpu")
        assert dim % heads == 0 and dim // heads % 8 == 0 and 8 <= dim // heads <= 128 and heads % kv == 0


@pytest.mark.parametrize("dim", [1, 4, 100, 257])
def test_widths_without_heads_are_refused(dim):
    from memory_lean_optimizer_gb300 import lm_example
    with pytest.raises(ValueError, match="does not make heads"):
        lm_example.block_heads(dim)
    with pytest.raises(ValueError, match="does not make heads"):
        lm_example.TinyLM(50, dim, blocks=1)
