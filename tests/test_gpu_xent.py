"""Softmax cross entropy from hidden states, forward and backward, against the formulas in 64 bits.

Tolerances.  A logit is a sum of `dim` exact products of bf16 values, each addition at most 2^-23 off
(whether it rounds or truncates): dl <= dim 2^-23 sum |h w|.  lse and loss are off by at most the largest dl
of the row (twice, for the target's), plus 2^-20 (1 + |lse|) for exponentials, their sum and the logarithm.
An entry of E is off by p (2 dl + 2^-18) |c| and then rounded to bf16, 2^-8 of its magnitude; a gradient is a
sum of K of them with at most 2^-23 of the sum of magnitudes lost per addition.  The last rounding, to an
output's type, is monotone: the output lies between the rounded ends of the interval these bounds give."""
import numpy as np
import pytest
import torch

from memory_lean_optimizer_gb300 import lmopt

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
IGN = -100


def inputs(rows, dim, vocab, seed=0, ignored=0.0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    w = (r(vocab, dim) * scale / dim ** 0.5).to(BF)
    h = r(rows, dim).to(BF)
    t = torch.randint(vocab, (rows,), generator=g, device="cuda")
    if ignored:
        t[torch.rand(rows, generator=g, device="cuda") < ignored] = IGN
    c = torch.rand(rows, generator=g, device="cuda") + 0.1
    return h, w, t, c


def within(got, want, tol):
    lo, hi = ((want + s * tol).float().to(got.dtype) for s in (-1, 1))
    return bool(((got >= lo) & (got <= hi)).all())


def check(h, w, t, c, ignore=IGN):
    from memory_lean_optimizer_gb300 import head
    loss, lse = head.xent_forward(h, w, t, ignore_index=ignore)
    dh, dw = head.xent_backward(h, w, t, lse, c, ignore_index=ignore)
    keep = torch.nonzero(t != ignore)[:, 0]
    out = torch.nonzero(t == ignore)[:, 0]
    assert not loss[out].any() and not lse[out].any() and not dh[out].any()
    H, W, C, T = h[keep].double(), w.double(), c[keep].double()[:, None], t[keep]
    dim, vocab = W.shape[1], W.shape[0]
    logits = H @ W.t()
    dl = (dim * 2.0 ** -23 * (H.abs() @ W.abs().t())).amax(1, keepdim=True) if len(keep) else logits.sum(1, keepdim=True)
    ref = torch.logsumexp(logits, 1, keepdim=True)
    tol = (dl + 2.0 ** -20 * (1 + ref.abs()))[:, 0]
    assert bool(((lse[keep].double() - ref[:, 0]).abs() <= tol).all())
    want = ref[:, 0] - logits.gather(1, T[:, None])[:, 0]
    assert bool(((loss[keep].double() - want).abs() <= 2 * tol).all())
    p = torch.exp(logits - ref)
    dp = p * (2 * dl + 2.0 ** -18) * C.abs()
    E = p.clone()
    E.scatter_add_(1, T[:, None], torch.full_like(T[:, None], -1, dtype=E.dtype))
    E *= C
    dE = dp + 2.0 ** -8 * E.abs() + 2.0 ** -8 * dp
    assert within(dh[keep], E @ W, dE @ W.abs() + vocab * 2.0 ** -23 * (E.abs() @ W.abs()))
    assert within(dw, E.t() @ H, dE.t() @ H.abs() + len(keep) * 2.0 ** -23 * (E.abs().t() @ H.abs()))
    return loss, lse, dh, dw


@pytest.mark.parametrize("rows,dim,vocab", [
    (1, 8, 1), (1, 64, 2), (1, 64, 256), (2, 1, 3), (3, 100, 257), (127, 65, 255), (128, 64, 1000), (129, 512, 2049),
    (256, 256, 512), (300, 72, 5000), (64, 1290, 3001), (257, 129, 700), (5, 4096, 20000), (1000, 256, 33000),
    (513, 2056, 1025), (16, 640, 50021)])
def test_sizes(rows, dim, vocab):
    check(*inputs(rows, dim, vocab))


@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("dim", [32, 33, 96, 160, 257, 288, 320, 400, 520, 776, 1032])
def test_columns_shared_between_tiles(rows, dim):
    check(*inputs(rows, dim, 1300))


@pytest.mark.parametrize("scale", [0.0, 30.0])
def test_flat_and_peaked_distributions(scale):
    check(*inputs(200, 256, 3000, scale=scale))


def test_large_logits_of_one_sign():
    h, w, t, c = inputs(100, 128, 1500, scale=8.0)
    check(h.abs(), w.abs(), t, c)
    check(h.abs(), -w.abs(), t, c)


@pytest.mark.parametrize("ignored", [0.3, 0.97])
@pytest.mark.parametrize("rows", [50, 1200])
def test_ignored_rows(rows, ignored):
    check(*inputs(rows, 192, 2000, ignored=ignored))


def test_all_rows_ignored_and_other_index():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(70, 96, 400)
    t[:] = 7
    loss, lse, dh, dw = check(h, w, t, c, ignore=7)
    assert not dw.any() and not dh.any()
    out = head.linear_cross_entropy(h.requires_grad_(), w.requires_grad_(), t, ignore_index=7)
    out.backward()
    assert float(out) == 0.0 and not h.grad.any() and not w.grad.any()


def test_non_finite_ignored_rows_reach_nothing():
    h, w, t, c = inputs(300, 160, 900, ignored=0.4)
    clean = check(h, w, t, c)
    h2, c2 = h.clone(), c.clone()
    off = torch.nonzero(t == IGN)[:, 0]
    h2[off[0::3]], h2[off[1::3]], c2[off] = float("nan"), float("inf"), float("nan")
    from memory_lean_optimizer_gb300 import head
    loss, lse = head.xent_forward(h2, w, t)
    dh, dw = head.xent_backward(h2, w, t, lse, c2)
    for a, b in zip(clean, (loss, lse, dh, dw)):
        assert torch.equal(a, b)


def test_rows_without_weight_are_left_out():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(200, 96, 700)
    lse = head.xent_forward(h, w, t)[1]
    c[::2] = 0.0
    dh, dw = head.xent_backward(h, w, t, lse, c)
    h2, lse2 = h.clone(), lse.clone()
    h2[::4], lse2[::4] = float("nan"), float("nan")
    dh2, dw2 = head.xent_backward(h2, w, t, lse2, c)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2) and not dh[::2].any()
    t2 = t.clone()
    t2[::2] = IGN
    assert torch.equal(head.xent_backward(h, w, t2, lse, c)[1], dw)


@pytest.mark.parametrize("bad", [-1, 700, 1 << 40])
def test_target_outside_the_vocabulary_is_loud(bad):
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(40, 96, 700)
    t[11] = bad
    loss, lse = head.xent_forward(h, w, t)
    assert bool(loss[11].isnan()) and int(loss.isnan().sum()) == 1 and bool(lse.isfinite().all())
    dh, dw = head.xent_backward(h, w, t, lse, c)
    assert bool(dh[11].isnan().all()) and int(dh.isnan().any(1).sum()) == 1 and bool(dw.isnan().all())


def test_non_finite_hidden_row_stays_in_its_row():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(40, 96, 700)
    clean = head.xent_forward(h, w, t)[0]
    h[5, 3] = float("nan")
    loss = head.xent_forward(h, w, t)[0]
    assert bool(loss[5].isnan())
    keep = [i for i in range(40) if i != 5]
    assert torch.equal(loss[keep], clean[keep])


def test_strides_and_alignment():
    """Rows of hidden and of the weight cut from wider matrices, on and off 16-byte boundaries."""
    h, w, t, c = inputs(150, 264, 1300)
    base = check(h[:, :256].contiguous(), w[:, :256].contiguous(), t, c)
    same = check(h[:, :256], w[:, :256], t, c)
    for a, b in zip(base, same):
        assert torch.equal(a, b)
    check(h[:, 1:257], w[:, 1:257], t, c)
    check(h[:, 3:250], w[:, 3:250], t, c)
    check(h[:, :256], w[:, 5:261], t, c)


def test_several_pieces_of_the_vocabulary():
    check(*inputs(20000, 64, 20500, ignored=0.1))


def test_leading_dimensions_and_single_gradients():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(60, 128, 999)
    loss, lse = head.xent_forward(h, w, t)
    loss3, lse3 = head.xent_forward(h.view(3, 20, 128), w, t.view(3, 20))
    assert loss3.shape == (3, 20) and torch.equal(loss3.view(-1), loss)
    dh, dw = head.xent_backward(h, w, t, lse, c)
    dh3, none = head.xent_backward(h.view(3, 20, 128), w, t.view(3, 20), lse3, c.view(3, 20), need_weight=False)
    assert none is None and torch.equal(dh3.view(-1, 128), dh)
    none, only = head.xent_backward(h, w, t, lse, c, need_hidden=False)
    assert none is None and torch.equal(only, dw)


def test_no_rows():
    from memory_lean_optimizer_gb300 import head
    w = torch.randn(300, 64, device="cuda").to(BF)
    h, t = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = head.xent_forward(h, w, t)
    dh, dw = head.xent_backward(h, w, t, lse, loss)
    assert loss.shape == (0,) and dh.shape == (0, 64) and not dw.any()


def test_deterministic_and_other_stream():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(700, 320, 9000, ignored=0.2)
    loss, lse = head.xent_forward(h, w, t)
    grads = head.xent_backward(h, w, t, lse, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = head.xent_forward(h, w, t, stream=side)
    more = head.xent_backward(h, w, t, again[1], c, stream=side)
    side.synchronize()
    for a, b in zip((loss, lse) + grads, again + more):
        assert torch.equal(a, b)


def test_gradient_against_differences():
    """Autograd's gradients of the mean loss against central differences of the 64-bit formula (step 1e-4 of
    directions of order one: truncation 1e-8) along random directions; E's rounding to bf16 and the outputs'
    allow 2^-7 of the sum of magnitudes."""
    from memory_lean_optimizer_gb300 import head
    h, w, t, _ = inputs(48, 96, 500, ignored=0.25)
    h.requires_grad_()
    w.requires_grad_()
    head.linear_cross_entropy(h, w, t).backward()
    keep = t != IGN

    def f(H, W):
        return float(torch.nn.functional.cross_entropy((H @ W.t())[keep], t[keep]))
    p = [h.detach().double(), w.detach().double()]
    for i, grad in enumerate((h.grad, w.grad)):
        d = torch.randn_like(p[i])
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-4 * d, p[i] - 1e-4 * d
        slope = (f(*hi) - f(*lo)) / 2e-4
        assert abs(float((grad.double() * d).sum()) - slope) <= 2.0 ** -7 * float((grad.double() * d).abs().sum()) + 1e-7


def test_reductions():
    from memory_lean_optimizer_gb300 import head
    h, w, t, _ = inputs(90, 64, 300, ignored=0.3)
    loss = head.xent_forward(h, w, t)[0]
    assert torch.equal(head.linear_cross_entropy(h, w, t, reduction="none"), loss)
    assert torch.equal(head.linear_cross_entropy(h, w, t, reduction="sum"), loss.sum())
    assert torch.equal(head.linear_cross_entropy(h, w, t), loss.sum() / (t != IGN).sum())
    with pytest.raises(ValueError):
        head.linear_cross_entropy(h, w, t, reduction="max")


def test_refusals_of_tensors():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(10, 64, 100)
    with pytest.raises(TypeError):
        head.xent_forward(h.float(), w, t)
    with pytest.raises(TypeError):
        head.xent_forward(h, w.half(), t)
    with pytest.raises(ValueError):
        head.xent_forward(h, w[:, :32], t)
    with pytest.raises(ValueError):
        head.xent_forward(h, w, t[:5])
    with pytest.raises(ValueError):
        head.xent_forward(h, w, t.int())
    with pytest.raises(ValueError):
        head.xent_forward(h.cpu(), w, t)
    with pytest.raises(ValueError):
        head.xent_backward(h, w, t, c[:3], c)
