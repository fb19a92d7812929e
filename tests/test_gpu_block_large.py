"""Offsets past 32 bits: rows far apart, and more than 2^31 elements."""
import pytest
import torch

from memory_lean_optimizer_gb300 import lmopt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FAR = 1 << 27                 # elements from one row to the next: 40 rows span 5.4e9


@pytest.fixture
def far():
    torch.cuda.empty_cache()
    buf = torch.zeros(40 * FAR, dtype=BF, device="cuda")          # 10.7 GB
    yield lambda first, heads, dim: buf.as_strided((40, heads, dim), (FAR, dim, 1), first)
    del buf
    torch.cuda.empty_cache()


def test_attention_on_rows_far_apart(far):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(0)
    near = [torch.randn(40, h, 64, device="cuda").to(BF) for h in (4, 2, 2, 4)]
    views = [far(1024 * i, t.shape[1], 64) for i, t in enumerate(near)]
    for v, t in zip(views, near):
        v.copy_(t)
    cu = torch.tensor([0, 17, 40], dtype=torch.int32, device="cuda")
    q, k, v, do = near
    out, lse = block.attention_forward(q, k, v, cu)
    grads = block.attention_backward(do, q, k, v, out, lse, cu)
    q, k, v, do = views
    got, got_lse = block.attention_forward(q, k, v, cu)
    assert torch.equal(got, out) and torch.equal(got_lse, lse)
    assert all(torch.equal(a, b) for a, b in zip(block.attention_backward(do, q, k, v, got, lse, cu), grads))
    # outputs far apart too, by the library call
    side = lambda t: (t.data_ptr(), t.stride(0), t.stride(1))
    o, dq, dk, dv = (far(8192 + 1024 * i, h, 64) for i, h in enumerate((4, 4, 2, 2)))
    sizes = (cu.data_ptr(), 2, 40, 4, 2, 64, 0.125)
    s = torch.cuda.current_stream().cuda_stream
    lmopt.attn_forward(side(q), side(k), side(v), side(o), got_lse.data_ptr(), *sizes, s)
    n = lmopt.attn_workspace(*sizes[:-1])
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    lmopt.attn_backward(side(do), side(q), side(k), side(v), side(o), got_lse.data_ptr(), side(dq), side(dk), side(dv), *sizes,
                        work.data_ptr(), n, s)
    assert torch.equal(o, out) and torch.equal(dq, grads[0]) and torch.equal(dk, grads[1]) and torch.equal(dv, grads[2])


def test_rotary_on_rows_far_apart(far):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(1)
    q, k = (torch.randn(40, h, 64, device="cuda").to(BF) for h in (4, 2))
    pos, plan = torch.randint(1 << 20, (40,), device="cuda"), block.RotaryPlan(64)
    want = block.rotary_forward(q, k, pos, plan)
    a, b = far(0, 4, 64), far(4096, 2, 64)
    a.copy_(q)
    b.copy_(k)
    assert all(torch.equal(x, y) for x, y in zip(block.rotary_forward(a, b, pos, plan), want))
    s = torch.cuda.current_stream().cuda_stream
    side = lambda t: (t.data_ptr(), FAR, 64, t.data_ptr(), FAR, 64, t.shape[1])      # in place
    lmopt.rope_apply(side(a), side(b), pos.data_ptr(), plan.turns.data_ptr(), 40, 64, 64, 1.0, False, False, lmopt.OPTIM_BF16, s)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("cols", [32768, 32767])
def test_activations_of_more_elements_than_31_bits(cols):
    """65600 rows: the last of them lie past 2^31 elements."""
    from memory_lean_optimizer_gb300 import block
    torch.cuda.empty_cache()
    rows = 65600
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    for part in x.split(8192):
        part.copy_(torch.randn(part.shape[0], cols, device="cuda", dtype=BF))
    p = block.pack_activation(x)
    y = block.unpack_activation(p)
    for s in (slice(0, 40), slice(40000, 40040), slice(rows - 40, rows)):
        q = block.pack_activation(x[s])
        assert torch.equal(p.codes[s], q.codes) and torch.equal(p.exponents[s], q.exponents)
        assert torch.equal(y[s], block.unpack_activation(q))
    del y, p
    half = cols // 2
    gu = x[:, :2 * half]
    h, p = block.swiglu_forward(gu)
    dh = h                                 # any gradient
    d, again = block.swiglu_backward(dh, p, need_h=True)
    for s in (slice(0, 40), slice(rows - 40, rows)):
        a, q = block.swiglu_forward(gu[s])
        b, c = block.swiglu_backward(dh[s], q, need_h=True)
        assert torch.equal(h[s], a) and torch.equal(d[s], b) and torch.equal(again[s], c)
    del x, gu, h, p, dh, d, again
    torch.cuda.empty_cache()
