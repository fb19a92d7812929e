"""Guard bytes directly before and behind workspaces of exactly the size that the workspace calls name, for the layer
norm's and the cross entropy's calls, over tile edges, split sums, copied weights and several pieces."""
import pytest
import torch

from memory_lean_optimizer_gb300 import lmopt
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def workspace(nbytes, align):
    g = Guarded(nbytes, 0)
    assert g.ptr() % align == 0
    return g


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("rows,dim,vocab", [(1, 1, 1), (3, 33, 65), (127, 64, 255), (128, 256, 512), (129, 72, 513), (200, 257, 1000),
                                            (64, 520, 3001), (300, 130, 257), (16, 1024, 30000), (1000, 64, 40000), (20, 4095, 33000),
                                            (20000, 64, 20500), (4096, 512, 32769)])
def test_cross_entropy(rows, dim, vocab, shift):
    from memory_lean_optimizer_gb300 import head
    torch.manual_seed(rows + dim + vocab)
    h = torch.randn(rows, dim, device="cuda").to(BF)
    store = torch.empty(vocab * dim + shift, dtype=BF, device="cuda")
    w = store[shift:].view(vocab, dim)
    w.copy_(torch.randn(vocab, dim, device="cuda") * dim ** -0.5)
    t = torch.randint(vocab, (rows,), device="cuda")
    t[torch.rand(rows, device="cuda") < 0.2] = -100
    c = torch.rand(rows, device="cuda")
    loss, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty(vocab, dim, dtype=BF, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    for backward in (False, True):
        n = lmopt.loss_xent_workspace(rows, dim, vocab, w.data_ptr(), dim, backward)
        ws = workspace(n, 256)
        if backward:
            lmopt.loss_xent_backward(h.data_ptr(), dim, w.data_ptr(), dim, t.data_ptr(), lse.data_ptr(), c.data_ptr(), rows, dim, vocab,
                                     -100, dh.data_ptr(), dim, dw.data_ptr(), dim, ws.ptr(), n, s)
        else:
            lmopt.loss_xent_forward(h.data_ptr(), dim, w.data_ptr(), dim, t.data_ptr(), rows, dim, vocab, -100, loss.data_ptr(),
                                    lse.data_ptr(), ws.ptr(), n, s)
        torch.cuda.synchronize()
        assert ws.intact()
    ref = head.xent_forward(h, w, t)
    for a, b in zip((loss, lse, dh, dw), ref + head.xent_backward(h, w, t, ref[1], c)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,dim", [(1, 1), (5, 31), (9, 64), (3, 511), (700, 513), (3000, 1024), (5, 2047), (4, 4096), (300, 8200),
                                      (2, 20001), (65, 20001)])
def test_layer_norm(rows, dim, dtype):
    from memory_lean_optimizer_gb300 import head
    torch.manual_seed(rows + dim)
    x, dy = (torch.randn(rows, dim, device="cuda").to(dtype) for _ in range(2))
    w = torch.randn(dim, device="cuda").to(dtype)
    _, mean, rstd = head.layer_norm_forward(x, w)
    want = head.layer_norm_backward(dy, x, w, mean, rstd)
    n = lmopt.norm_layer_workspace(rows, dim)
    ws = workspace(n, 16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    k = lmopt.OPTIM_BF16 if dtype == BF else lmopt.OPTIM_F32
    lmopt.norm_layer_backward(dy.data_ptr(), dim, x.data_ptr(), dim, w.data_ptr(), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), dim,
                              dw.data_ptr(), db.data_ptr(), rows, dim, k, k, ws.ptr(), n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert ws.intact()
    for a, b in zip((dx, dw, db), want):
        assert torch.equal(a, b)
