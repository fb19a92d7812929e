"""What a transformer block holds between its forward and its backward pass."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def requested():
    """Bytes of the tensors that live: as asked for (the allocator's own count has up to 1 MiB more for each, where it does not split a block)."""
    return torch.cuda.memory_stats()["requested_bytes.all.current"]


@pytest.mark.parametrize("heads,kv", [(8, 4), (8, 8), (8, 1)])
def test_block_keeps_what_its_backward_pass_reads(heads, kv):
    """A token's bytes: both norms' outputs' sources and statistics, the first norm's output, rotated q and k, v, attention's output and lse, the sum
    behind it, x, gate and up in 8 bits, and the block's output.  Not q and k as they were before they were turned."""
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(0)
    tokens, dim, hidden = 4096, 512, 512
    d = dim // heads
    b = block.TransformerBlock(dim, heads, kv, hidden)
    x = torch.randn(tokens, dim, device="cuda").to(BF).requires_grad_()
    pos = torch.arange(tokens, device="cuda")
    b(x, pos)                            # library workspaces
    torch.cuda.synchronize()
    before = requested()
    y = b(x, pos)
    kept = requested() - before
    norms = 2 * dim + 2 * 8 + 2 * dim            # the first one's output, both's statistics, the second one's input
    attention = 2 * d * (heads + 2 * kv) + 2 * dim + 4 * heads
    mlp = (dim + 2 * hidden) * 33 / 32
    assert kept <= tokens * (norms + attention + mlp + 2 * dim) + (1 << 20)
    y.sum().backward()


def test_results_are_those_of_the_calls():
    from memory_lean_optimizer_gb300 import block, head
    torch.manual_seed(1)
    b = block.TransformerBlock(256, 4, 2, 64)
    with torch.no_grad():
        b.proj.copy_(torch.randn_like(b.proj))
    x = torch.randn(300, 256, device="cuda").to(BF).requires_grad_()
    pos, cu = torch.arange(300, device="cuda"), torch.tensor([0, 100, 290], dtype=torch.int32, device="cuda")
    y = b(x, pos, cu)
    with torch.no_grad():
        assert torch.equal(b(x, pos, cu), y)
    qkv = torch.nn.functional.linear(head.layer_norm(x, b.norm1, None, b.eps), b.qkv).view(300, 8, 64)
    q, k = block.rotary(qkv[:, :4], qkv[:, 4:6], pos, b.rotary)
    z = x + torch.nn.functional.linear(block.attention(q, k, qkv[:, 6:], cu).flatten(1), b.proj)
    z = z + block.gated_mlp(head.layer_norm(z, b.norm2, None, b.eps), b.w_in, b.w_out)
    assert torch.equal(y, z)
    dy = torch.randn_like(y)
    for g, w in zip(torch.autograd.grad(y, [x, *b.parameters()], dy), torch.autograd.grad(z, [x, *b.parameters()], dy)):
        assert torch.equal(g, w)
