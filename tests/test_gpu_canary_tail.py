"""Guard bytes around every buffer of the layer norm, cross entropy and AdamW calls: after each call the 512
bytes before and after every buffer still hold their value, inputs are unchanged, and the results equal
those on ordinary buffers.  Sizes lie on both sides of vector widths, tiles (32, 64, 128, 256) and
blocks (256); buffers start on the alignment that the widest path asks for or at the smallest they accept."""
import numpy as np
import pytest
import torch

from memory_lean_optimizer_gb300 import lmopt
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def stream():
    return torch.cuda.current_stream().cuda_stream


class Buffers:
    def __init__(self):
        self.all = []

    def put(self, x, shift=0):
        g = Guarded(x.numel() * x.element_size(), shift * x.element_size())
        v = g.view(x.dtype, x.shape)
        v.copy_(x)
        self.all.append((g, v, x.clone()))
        return g.ptr()

    def out(self, shape, dtype, shift=0):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        g = Guarded(n, shift * torch.empty(0, dtype=dtype).element_size())
        self.all.append((g, g.view(dtype, shape), None))
        return g.ptr(), self.all[-1][1]

    def check(self):
        torch.cuda.synchronize()
        for g, v, before in self.all:
            assert g.intact()
            if before is not None:
                assert torch.equal(v.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,dim", [(1, 1), (5, 31), (9, 64), (3, 511), (17, 513), (6, 1024), (5, 2047), (4, 4096), (3, 8200),
                                      (2, 20001)])
def test_layer_norm(rows, dim, dtype, shift):
    from memory_lean_optimizer_gb300 import head
    torch.manual_seed(rows + dim)
    x, dy = (torch.randn(rows, dim, device="cuda").to(dtype) for _ in range(2))
    w, b = (torch.randn(dim, device="cuda").to(dtype) for _ in range(2))
    ref = head.layer_norm_forward(x, w, b)
    bufs = Buffers()
    t = lmopt.OPTIM_BF16 if dtype == BF else lmopt.OPTIM_F32
    px, pw, pb, pg = (bufs.put(a, shift) for a in (x, w, b, dy))
    py, y = bufs.out((rows, dim), dtype, shift)
    pm, mean = bufs.out((rows,), torch.float32, shift)
    pr, rstd = bufs.out((rows,), torch.float32, shift)
    lmopt.norm_layer_forward(px, dim, pw, pb, py, dim, pm, pr, rows, dim, 1e-5, t, t, stream())
    n = lmopt.norm_layer_workspace(rows, dim)
    pws, _ = bufs.out((n,), torch.uint8)
    pd, dx = bufs.out((rows, dim), dtype, shift)
    pdw, dw = bufs.out((dim,), dtype, shift)
    pdb, db = bufs.out((dim,), dtype, shift)
    lmopt.norm_layer_backward(pg, dim, px, dim, pw, pm, pr, pd, dim, pdw, pdb, rows, dim, t, t, pws, n, stream())
    bufs.check()
    # another alignment may sum in another order: a few roundings of fp32, and one of the type, apart
    tol = (2.0 ** -7 if dtype == BF else 2.0 ** -20)
    want = ref + head.layer_norm_backward(dy, x, w, *ref[1:])
    for got, ref_t in zip((y, mean, rstd, dx, dw, db), want):
        scale = float(ref_t.float().abs().max()) + 1e-6
        assert float((got.float() - ref_t.float()).abs().max()) <= (tol if got.dtype == dtype else 2.0 ** -20) * max(scale, 1.0) * 4


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("rows,dim,vocab", [(1, 1, 1), (3, 33, 65), (127, 64, 255), (129, 72, 513), (200, 257, 1000), (64, 520, 3001),
                                            (300, 130, 257)])
def test_cross_entropy(rows, dim, vocab, shift):
    from memory_lean_optimizer_gb300 import head
    torch.manual_seed(rows + dim + vocab)
    h = torch.randn(rows, dim, device="cuda").to(BF)
    w = (torch.randn(vocab, dim, device="cuda") * dim ** -0.5).to(BF)
    t = torch.randint(vocab, (rows,), device="cuda")
    t[torch.rand(rows, device="cuda") < 0.2] = -100
    c = torch.rand(rows, device="cuda")
    ref = head.xent_forward(h, w, t)
    ref_grads = head.xent_backward(h, w, t, ref[1], c)
    bufs = Buffers()
    ph, pw, pt, pc = bufs.put(h, shift), bufs.put(w, shift), bufs.put(t), bufs.put(c, shift)
    pl, loss = bufs.out((rows,), torch.float32, shift)
    pe, lse = bufs.out((rows,), torch.float32, shift)
    for backward in (False, True):
        n = lmopt.loss_xent_workspace(rows, dim, vocab, pw, dim, backward)
        pws, _ = bufs.out((n + 256,), torch.uint8)
        at = (pws + 255) // 256 * 256
        if not backward:
            lmopt.loss_xent_forward(ph, dim, pw, dim, pt, rows, dim, vocab, -100, pl, pe, at, n, stream())
            continue
        pdh, dh = bufs.out((rows, dim), BF, shift)
        pdw, dw = bufs.out((vocab, dim), BF, shift)
        lmopt.loss_xent_backward(ph, dim, pw, dim, pt, pe, pc, rows, dim, vocab, -100, pdh, dim, pdw, dim, at, n, stream())
    bufs.check()
    for a, b in zip((loss, lse, dh, dw), ref + ref_grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_adamw(states, shift):
    from memory_lean_optimizer_gb300 import engine
    rng = np.random.default_rng(0)
    sizes = [1, 7, 255, 257, 4095, 4096, 4097, 4353, 16383, 16385, 65537]
    masters = [torch.from_numpy((rng.standard_normal(n) * 0.02).astype(np.float32)).cuda() for n in sizes]
    plain = engine.AdamWGroup.from_masters(masters, states=states)
    guards, descs, views, keep = [], [], [], []
    for x in masters:
        n = x.numel()
        hi, lo = engine.kahan_split(x)
        size = engine.u8_state_bytes(n) if states == "u8" and n > 4096 else 4 * n
        gw, gr = Guarded(2 * n, 2 * shift), Guarded(2 * n, 2 * shift)
        gm, gv = Guarded(size, 4 * shift), Guarded(size, 4 * shift)
        gw.view(BF, (n,)).copy_(hi)
        gr.view(torch.int16, (n,)).copy_(lo)
        for s in (gm, gv):
            s.view(torch.uint8, (size,)).zero_()
        d = lmopt.TensorDesc(w_bf16=gw.ptr(), res_u16=gr.ptr(), m=gm.ptr(), v=gv.ptr(), numel=n, ndim=1)
        d.shape[0] = n
        descs.append(d)
        guards += [gw, gr, gm, gv]
        views.append((gw.view(BF, (n,)), gr.view(torch.int16, (n,)), gm.view(torch.uint8, (size,)), gv.view(torch.uint8, (size,))))
    handle = lmopt.optim_group_create(descs, lmopt.OPTIM_KIND_ADAMW_U8 if states == "u8" else lmopt.OPTIM_KIND_ADAMW)
    hp = dict(lr=1e-3, weight_decay=0.01)
    for step in (1, 2, 3):
        grads = [torch.from_numpy((rng.standard_normal(n) * 1e-3).astype(np.float32)).to(BF).cuda() for n in sizes]
        gg = []
        for g in grads:
            b = Guarded(2 * g.numel(), 2 * shift)
            b.view(BF, g.shape).copy_(g)
            gg.append(b)
        plain.step(grads, hp)
        lmopt.optim_step_adamw(handle, [b.ptr() for b in gg], step,
                               lmopt.AdamWHparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01), None, stream())
        torch.cuda.synchronize()
        assert all(g.intact() for g in guards + gg)
        for b, g in zip(gg, grads):
            assert torch.equal(b.view(BF, g.shape), g)
        for i, (w, r, m, v) in enumerate(views):
            assert torch.equal(w, plain.weights[i]) and torch.equal(r, plain.res[i])
            for a, b in ((m, plain.m[i]), (v, plain.v[i])):
                n = sizes[i]
                if states == "u8" and n > 4096:       # the padding between codes and constants is nobody's
                    codes, q = engine.u8_state_views(a, n)
                    codes2, q2 = engine.u8_state_views(b, n)
                    assert torch.equal(codes, codes2) and torch.equal(q, q2)
                else:
                    assert torch.equal(a.view(torch.float32), b)
    total = sum((n + 63) // 64 * 64 for n in sizes)
    fm, fv = Guarded(4 * total, 4 * shift), Guarded(4 * total, 4 * shift)
    lmopt.optim_group_unpack_state(handle, fm.ptr(), fv.ptr(), stream())
    torch.cuda.synchronize()
    assert fm.intact() and fv.intact()
    m, v = plain.unpack_states()
    at = 0
    for n in sizes:
        assert torch.equal(fm.view(torch.float32, (total,))[at:at + n], m[at:at + n])
        assert torch.equal(fv.view(torch.float32, (total,))[at:at + n], v[at:at + n])
        at += (n + 63) // 64 * 64
    lmopt.optim_group_destroy(handle)
