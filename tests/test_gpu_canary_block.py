"""Guard bytes around every buffer of the attention, rotary and 8-bit activation calls: after each call the 512 bytes
before and after every buffer still hold their value, inputs are unchanged, and the results equal those on ordinary
buffers.  Sizes lie on both sides of tiles and blocks (16, 32, 64, 128, 256); buffers start on the widest path's alignment or at the
smallest they accept."""
import pytest
import torch

from memory_lean_optimizer_gb300 import lmopt
from test_gpu_canary_tail import Buffers, stream

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def kind(dtype):
    return lmopt.OPTIM_BF16 if dtype == BF else lmopt.OPTIM_F32


@pytest.mark.parametrize("rows,heads,kv,dim,lengths", [(1, 1, 1, 8, [1]), (37, 4, 2, 64, [37]), (129, 2, 1, 80, [129]), (300, 2, 2, 128, [256, 40]),
                                                       (257, 3, 1, 72, [64, 0, 65, 100]), (1030, 8, 1, 128, [1025])])
def test_attention(rows, heads, kv, dim, lengths):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(rows)
    q, do = (torch.randn(rows, heads, dim, device="cuda").to(BF) for _ in range(2))
    k, v = (torch.randn(rows, kv, dim, device="cuda").to(BF) for _ in range(2))
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    ref = block.attention_forward(q, k, v, cu)
    grads = block.attention_backward(do, q, k, v, *ref, cu)
    b = Buffers()
    side = lambda p, h: (p, h * dim, dim)
    pq, pk, pv, pdo, pcu = (b.put(t) for t in (q, k, v, do, cu))
    po, out = b.out((rows, heads, dim), BF)
    pl, lse = b.out((heads, rows), F32)
    sizes = (pcu, len(lengths), rows, heads, kv, dim, dim ** -0.5)
    lmopt.attn_forward(side(pq, heads), side(pk, kv), side(pv, kv), side(po, heads), pl, *sizes, stream())
    b.check()
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    got = [b.out((rows, h, dim), BF) for h in (heads, kv, kv)]
    n = lmopt.attn_workspace(*sizes[:-1])
    pw, _ = b.out((n,), torch.uint8)
    lmopt.attn_backward(side(pdo, heads), side(pq, heads), side(pk, kv), side(pv, kv), side(po, heads), pl, side(got[0][0], heads),
                        side(got[1][0], kv), side(got[2][0], kv), *sizes, pw, n, stream())
    b.check()
    assert all(torch.equal(g[1], w) for g, w in zip(got, grads))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,kv,dim,rotary", [(1, 1, 1, 1, 0), (3, 2, 1, 6, 2), (33, 4, 2, 64, 64), (9, 3, 3, 81, 36), (300, 2, 1, 128, 96)])
def test_rotary(rows, heads, kv, dim, rotary, interleaved, dtype, shift):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(rows)
    q, k = (torch.randn(rows, h, dim, device="cuda").to(dtype) for h in (heads, kv))
    pos = torch.randint(1 << 20, (rows,), device="cuda")
    plan = block.RotaryPlan(rotary, interleaved=interleaved)
    ref = block.rotary_forward(q, k, pos, plan)
    b = Buffers()
    pq, pk = b.put(q, shift), b.put(k, shift)
    ppos, pt = b.put(pos), b.put(plan.turns) if rotary else None
    (oq, yq), (ok, yk) = (b.out((rows, h, dim), dtype, shift) for h in (heads, kv))
    lmopt.rope_apply((pq, heads * dim, dim, oq, heads * dim, dim, heads), (pk, kv * dim, dim, ok, kv * dim, dim, kv), ppos, pt, rows, dim,
                     rotary, 1.0, interleaved, False, kind(dtype), stream())
    b.check()
    assert torch.equal(yq, ref[0]) and torch.equal(yk, ref[1])


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 15), (2, 32), (5, 33), (40, 80), (7, 511), (130, 64), (2, 4100)])
def test_activations(rows, cols, dtype, shift):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(rows + cols)
    x, gu, dh = (torch.randn(rows, c, device="cuda").to(dtype) for c in (cols, 2 * cols, cols))
    ref = block.pack_activation(x)
    blocks = -(-cols // 32)
    b = Buffers()
    px = b.put(x, shift)
    pc, codes = b.out((rows, 32 * blocks), torch.int8)
    pe, exps = b.out((rows, blocks), torch.uint8, shift)
    lmopt.act_pack_i8(px, cols, pc, 32 * blocks, pe, blocks, rows, cols, kind(dtype), stream())
    b.check()
    assert torch.equal(codes, ref.codes) and torch.equal(exps, ref.exponents)
    py, y = b.out((rows, cols), dtype, shift)
    lmopt.act_unpack_i8(pc, 32 * blocks, pe, blocks, py, cols, rows, cols, kind(dtype), stream())
    b.check()
    assert torch.equal(y, block.unpack_activation(ref))
    h_ref, p_ref = block.swiglu_forward(gu)
    b = Buffers()
    pg, pd = b.put(gu, shift), b.put(dh, shift)
    ph, h = b.out((rows, cols), dtype, shift)
    pc, codes = b.out((2 * rows, 32 * blocks), torch.int8)
    pe, exps = b.out((2 * rows, blocks), torch.uint8, shift)
    lmopt.act_swiglu_forward(pg, 2 * cols, ph, cols, pc, 32 * blocks, pe, blocks, rows, cols, kind(dtype), stream())
    b.check()
    assert torch.equal(h, h_ref) and torch.equal(codes, p_ref.codes) and torch.equal(exps, p_ref.exponents)
    po, d = b.out((rows, 2 * cols), dtype, shift)
    pa, again = b.out((rows, cols), dtype, shift)
    lmopt.act_swiglu_backward(pd, cols, pc, 32 * blocks, pe, blocks, po, 2 * cols, pa, cols, rows, cols, kind(dtype), stream())
    b.check()
    want = block.swiglu_backward(dh, p_ref, need_h=True)
    assert torch.equal(d, want[0]) and torch.equal(again, want[1])
