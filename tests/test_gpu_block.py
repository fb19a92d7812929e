"""The operators of a transformer block run together: the block against the same formulas in fp32, its gradients against
differences, and the example that trains it."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def make(dim=128, heads=4, kv=2, hidden=192, interleaved=False, scaling=None):
    from memory_lean_optimizer_gb300 import block
    plan = block.RotaryPlan(dim // heads, interleaved=interleaved, scaling=scaling, factor=4.0 if scaling else 1.0, original_length=256)
    b = block.TransformerBlock(dim, heads, kv, hidden, plan)
    with torch.no_grad():        # the output matrices start at zero: give them something
        b.proj.copy_(torch.randn_like(b.proj.float()) * dim ** -0.5)
        b.w_out.copy_(torch.randn_like(b.w_out.float()) * hidden ** -0.5)
        b.norm1.copy_(1 + 0.2 * torch.randn_like(b.norm1.float()))
    return b


def formula(b, p, x, positions, lengths):
    """The block in the parameters p (fp32 or fp64), from its formulas."""
    from memory_lean_optimizer_gb300 import block
    h, kv, d = b.heads, b.kv_heads, b.head_dim
    norm = lambda t, w: torch.nn.functional.layer_norm(t, (t.shape[-1],), w, None, b.eps)
    qkv = (norm(x, p["norm1"]) @ p["qkv"].t()).view(x.shape[0], h + 2 * kv, d)
    plan = b.rotary
    f = torch.tensor([t / 2 ** 64 * 2 * math.pi for t in (t % 2 ** 64 for t in plan.turns.tolist())], dtype=torch.float64, device=x.device)
    a = positions.double()[:, None, None] * f
    c, s = (a.cos() * plan.factor).to(x.dtype), (a.sin() * plan.factor).to(x.dtype)
    r = plan.rotary_dim
    i, j = (slice(0, r, 2), slice(1, r, 2)) if plan.interleaved else (slice(0, r // 2), slice(r // 2, r))

    def turn(t):
        y = t.clone()
        y[..., i], y[..., j] = t[..., i] * c - t[..., j] * s, t[..., j] * c + t[..., i] * s
        return y
    q, k, v = turn(qkv[:, :h]), turn(qkv[:, h:h + kv]), qkv[:, h + kv:]
    seq = torch.repeat_interleave(torch.arange(len(lengths), device=x.device), torch.tensor(lengths, device=x.device))
    see = (seq[:, None] == seq[None, :]) & torch.ones(len(seq), len(seq), dtype=torch.bool, device=x.device).tril()
    w = (torch.einsum("ihd,jhd->hij", q, k.repeat_interleave(h // kv, 1)) * d ** -0.5).masked_fill(~see, -math.inf).softmax(2)
    y = torch.einsum("hij,jhd->ihd", w, v.repeat_interleave(h // kv, 1)).flatten(1)
    x = x + y @ p["proj"].t()
    gu = norm(x, p["norm2"]) @ p["w_in"].t()
    n = gu.shape[1] // 2
    return x + (torch.nn.functional.silu(gu[:, :n]) * gu[:, n:]) @ p["w_out"].t()


@pytest.mark.parametrize("interleaved,scaling", [(False, None), (True, "yarn")])
def test_block_equals_its_formulas(interleaved, scaling):
    """Output and gradients in the 2-norm: some twenty roundings to bf16 (2^-8 at most, a third of that on average) and the 8-bit values
    (2^-7 at most of a block's largest), each relative to what they round and uncorrelated: within 2^-5."""
    torch.manual_seed(0)
    b = make(interleaved=interleaved, scaling=scaling)
    lengths = [130, 1, 69, 200]
    n = sum(lengths)
    x = torch.randn(n, 128, device="cuda").to(BF).requires_grad_()
    pos = torch.cat([torch.arange(m) for m in lengths]).cuda()
    cu = torch.tensor([0, 130, 131, 200, 400], dtype=torch.int32, device="cuda")
    dy = torch.randn(n, 128, device="cuda").to(BF)
    y = b(x, pos, cu)
    names = [k for k, _ in b.named_parameters()]
    got = torch.autograd.grad(y, [x, *b.parameters()], dy)
    p = {k: v.detach().double().requires_grad_() for k, v in b.named_parameters()}
    xr = x.detach().double().requires_grad_()
    ref = formula(b, p, xr, pos, lengths)
    want = torch.autograd.grad(ref, [xr, *(p[k] for k in names)], dy.double())
    assert float((y.double() - ref).norm()) <= 2.0 ** -5 * float(ref.norm())
    for name, g, w in zip(["x", *names], got, want):
        assert float((g.double() - w).norm()) <= 2.0 ** -5 * float(w.norm()), name


def test_gradient_of_the_block_against_differences():
    """<dy, block(x)> along a direction in 64 bits, against the gradients' product with it."""
    torch.manual_seed(1)
    b = make()
    lengths = [90, 60]
    x = torch.randn(150, 128, device="cuda").to(BF).requires_grad_()
    pos = torch.cat([torch.arange(m) for m in lengths]).cuda()
    cu = torch.tensor([0, 90, 150], dtype=torch.int32, device="cuda")
    dy = torch.randn(150, 128, device="cuda").to(BF)
    g, gq = torch.autograd.grad(b(x, pos, cu), (x, b.qkv), dy)
    p = {k: v.detach().double() for k, v in b.named_parameters()}
    loss = lambda x, p: float((formula(b, p, x, pos, lengths) * dy.double()).sum())
    for grad, at in ((g, None), (gq, "qkv")):
        step = torch.randn_like(grad, dtype=torch.float64)
        step = step / step.norm() + grad.double() / grad.double().norm()     # partly along the gradient: far from 0
        h = 1e-3

        def moved(s):
            return loss(x.detach().double() + s * step, p) if at is None else loss(x.detach().double(), {**p, at: p[at] + s * step})
        slope = (moved(h) - moved(-h)) / (2 * h)
        assert abs(float((grad.double() * step).sum()) - slope) <= 2.0 ** -5 * float(grad.double().norm()) * float(step.norm())


def test_block_starts_as_the_identity_and_packs_like_single_sequences():
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(2)
    b = block.TransformerBlock(128, 2)
    x = torch.randn(70, 128, device="cuda").to(BF)
    assert torch.equal(b(x, torch.arange(70, device="cuda")), x)
    b = make()
    pos = torch.cat((torch.arange(30), torch.arange(40))).cuda()
    cu = torch.tensor([0, 30, 70], dtype=torch.int32, device="cuda")
    with torch.no_grad():
        y = b(x, pos, cu)
        a, c = b(x[:30], pos[:30]), b(x[30:], pos[30:])
    # the attention does not see its neighbours; cuBLAS may take other kernels for other row counts (roundings of bf16)
    assert float((torch.cat((a, c)).double() - y.double()).abs().max()) <= 2.0 ** -5 * float(y.double().abs().max())


def test_memory_kept_for_the_backward_pass():
    """The gated MLP keeps x, gate and up at a byte an element and a 32nd of one, and nothing else of their size."""
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(3)
    x = torch.randn(4096, 256, device="cuda").to(BF)
    w1, w2 = (torch.randn(*s, device="cuda").to(BF).requires_grad_() for s in ((2048, 256), (256, 1024)))
    block.gated_mlp(x, w1, w2)           # library workspaces
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    y = block.gated_mlp(x, w1, w2)
    kept = torch.cuda.memory_allocated() - before - y.numel() * 2
    assert kept <= 4096 * (2048 + 256) * (1 + 1 / 32) + (1 << 20)
    y.sum().backward()


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_example_with_blocks_runs(states):
    from memory_lean_optimizer_gb300 import lm_example
    losses = lm_example.train(steps=4, vocab=500, dim=128, rows=4, length=96, states=states, blocks=2)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
    # identity at first: the first loss is that without blocks
    assert abs(losses[0] - (math.log(500) + 0.5)) < 0.5


def test_example_model_gradients():
    """The example's model, blocks included, against the same formulas in 64 bits."""
    from memory_lean_optimizer_gb300 import lm_example
    torch.manual_seed(4)
    model = lm_example.TinyLM(300, 128, blocks=1)
    with torch.no_grad():
        for w in (model.blocks[0].proj, model.blocks[0].w_out):
            w.copy_(torch.randn_like(w.float()) * w.shape[1] ** -0.5)
    tokens = torch.randint(300, (3, 50), device="cuda")
    target = torch.randint(300, (3, 50), device="cuda")
    loss = model(tokens, target)
    loss.backward()
    p = {k: v.detach().double().requires_grad_() for k, v in model.named_parameters()}
    b = {k.removeprefix("blocks.0."): v for k, v in p.items() if k.startswith("blocks.0.")}
    x = p["embed.weight"][tokens.flatten()]
    x = formula(model.blocks[0], b, x, torch.arange(50, device="cuda").repeat(3), [50] * 3)
    x = torch.nn.functional.layer_norm(x, (128,), p["tail.norm_weight"], p["tail.norm_bias"], 1e-5)
    ref = torch.nn.functional.cross_entropy(x @ p["tail.weight"].t(), target.flatten())
    ref.backward()
    assert abs(float(loss.detach()) - float(ref.detach())) < 2.0 ** -5
    for k, v in model.named_parameters():
        assert float((v.grad.double() - p[k].grad).norm()) <= 2.0 ** -4 * float(p[k].grad.norm()), k


def test_block_of_no_tokens():
    b = make()
    x = torch.zeros(0, 128, device="cuda", dtype=BF).requires_grad_()
    pos = torch.zeros(0, dtype=torch.int64, device="cuda")
    for cu in (None, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")):
        y = b(x, pos, cu)
        assert y.shape == (0, 128)
        g = torch.autograd.grad(y, [x, *b.parameters()], torch.zeros_like(y))
        assert all(not t.any() for t in g)


def test_operators_with_their_gradients_in_a_graph():
    """Rotary, attention and the gated activation with autograd, captured and replayed with other inputs and borders: bit for bit
    what they give outside a graph.  (No eager autograd graph of the same leaves is alive at the capture.)"""
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(5)
    plan = block.RotaryPlan(64)
    x = torch.randn(150, 8 * 64, device="cuda").to(BF).requires_grad_()
    pos = torch.arange(150, device="cuda")
    cu = torch.tensor([0, 90, 150], dtype=torch.int32, device="cuda")
    dy = torch.randn(150, 2 * 64, device="cuda").to(BF)

    def step():
        qkv = x.view(150, 8, 64)
        q, k = block.rotary(qkv[:, :4], qkv[:, 4:6], pos, plan)
        y = block.swiglu(block.attention(q, k, qkv[:, 6:], cu).flatten(1))
        return y.detach(), torch.autograd.grad(y, x, dy)[0]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    with torch.no_grad():
        x.copy_(torch.randn(150, 8 * 64, device="cuda").to(BF))
    cu.copy_(torch.tensor([0, 20, 140], dtype=torch.int32))
    pos.copy_(torch.randperm(150))
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))
