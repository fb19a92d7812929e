"""Layer norm, forward and backward, against the formulas in 64 bits.

Tolerances, with u = 2^-24: a row's sum is at most dim/32 sequential additions in a thread and then a tree,
so a mean of values x_i is within c = (dim/32 + 32) u of mean |x_i|; the remaining operations add a few
u each, which the 32 covers.  mu enters xh as an absolute error c r mean|x|, the variance as a relative
one.  Column sums are bounded by (rows + 32) u of the sum of magnitudes.  The one rounding to an output's
type is monotone, so the output lies between the rounded ends of the interval that these bounds give the
fp32 value: no tolerance stands for it."""
import numpy as np
import pytest
import torch

from memory_lean_optimizer_gb300 import lmopt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (F32, F32), (F32, BF), (BF, F32)]


def inputs(rows, dim, xt, wt, seed=0, pad=0, offset=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    x = (r(rows, dim + pad) * 2 + offset + r(rows, 1)).to(xt)[:, :dim]
    dy = r(rows, dim + pad).to(xt)[:, :dim]
    return x, (1 + 0.3 * r(dim)).to(wt), r(dim).to(wt), dy


def within(got, want, tol):
    """got is a rounding of some value in want +- tol (both ends rounded the same way, through fp32)."""
    lo, hi = ((want + s * tol).float().to(got.dtype) for s in (-1, 1))
    return bool(((got >= lo) & (got <= hi)).all())


def check(x, w, b, dy, eps=1e-5):
    from memory_lean_optimizer_gb300 import head
    rows, dim = x.shape
    y, mean, rstd = head.layer_norm_forward(x, w, b, eps)
    X, W, B, G = x.double(), w.double(), b.double(), dy.double()
    mu = X.mean(1, keepdim=True)
    r = 1 / ((X - mu).pow(2).mean(1, keepdim=True) + eps).sqrt()
    xh = (X - mu) * r
    c = (dim / 32 + 32) * U
    ax = X.abs().mean(1, keepdim=True)
    dxh = c * (r * (ax + X.abs()) + xh.abs())             # error of xh in fp32
    assert bool(((mean.double()[:, None] - mu).abs() <= c * ax).all())
    # the mean's own error moves the variance by its square; relative to r: c + (r dmu)^2 / 2
    assert bool(((rstd.double()[:, None] - r).abs() <= r * (c + (r * c * ax) ** 2 + 4 * U)).all())
    want = xh * W + B
    assert within(y, want, W.abs() * dxh + 4 * U * B.abs())
    dx, dw, db = head.layer_norm_backward(dy, x, w, mean, rstd)
    a = G * W
    m1, m2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
    want = r * (a - m1 - xh * m2)
    aa = a.abs().mean(1, keepdim=True)
    e2 = c * (a * xh).abs().mean(1, keepdim=True) + (a.abs() * dxh).mean(1, keepdim=True)
    tol = r * (4 * U * a.abs() + c * aa + xh.abs() * e2 + dxh * m2.abs() + c * (a.abs() + aa + (xh * m2).abs()))
    assert within(dx, want, 2 * tol)
    k = (rows + 32) * U
    want = (G * xh).sum(0)
    tol = k * (G * xh).abs().sum(0) + (G.abs() * dxh).sum(0)
    assert within(dw, want, tol)
    want = G.sum(0)
    assert within(db, want, k * G.abs().sum(0))
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("xt,wt", TYPES)
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 2), (5, 31), (33, 64), (300, 257), (7, 1000), (130, 1024), (1, 4096),
                                      (257, 4096), (40, 4100), (70, 8192), (9, 20001), (3, 33000), (2000, 40)])
def test_sizes_and_types(rows, dim, xt, wt):
    check(*inputs(rows, dim, xt, wt))


@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("pad", [1, 2, 8, 24])
def test_row_strides(xt, pad):
    check(*inputs(65, 512, xt, xt, pad=pad))
    check(*inputs(65, 513, xt, xt, pad=pad))


@pytest.mark.parametrize("xt", [BF, F32])
def test_unaligned_start(xt):
    x, w, b, dy = inputs(20, 1025, xt, xt)
    check(x[:, 1:], w[1:], b[1:], dy[:, 1:])


def test_offset_far_above_the_spread():
    check(*inputs(17, 2048, F32, F32, offset=3000.0))


def test_constant_rows_and_zero_gradient():
    from memory_lean_optimizer_gb300 import head
    x = torch.full((4, 600), 3.0, device="cuda", dtype=BF)
    w, b = torch.ones(600, device="cuda", dtype=BF), torch.full((600,), 0.5, device="cuda", dtype=BF)
    y, mean, rstd = head.layer_norm_forward(x, w, b, 1e-5)
    assert bool((y == 0.5).all()) and bool((mean == 3.0).all())
    dx, dw, db = head.layer_norm_backward(torch.zeros_like(x), x, w, mean, rstd)
    assert not dx.any() and not dw.any() and not db.any()


def test_non_finite_rows_stay_in_their_rows():
    from memory_lean_optimizer_gb300 import head
    x, w, b, dy = inputs(12, 3000, BF, BF)
    clean = head.layer_norm_forward(x, w, b)[0]
    x[3, 7], x[8, 0] = float("nan"), float("inf")
    y, mean, rstd = head.layer_norm_forward(x, w, b)
    keep = [i for i in range(12) if i not in (3, 8)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[3].isnan().all()) and bool(y[8].isnan().any())
    dx = head.layer_norm_backward(dy, x, w, mean, rstd)[0]
    assert bool(dx[keep].isfinite().all()) and bool(dx[3].isnan().all())


def test_no_rows():
    from memory_lean_optimizer_gb300 import head
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = head.layer_norm_forward(x, w)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dw, db = head.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_shapes_and_views():
    """Leading dimensions, a transposed matrix, a broadcast row and a missing bias give what a plain matrix gives."""
    from memory_lean_optimizer_gb300 import head
    x, w, b, dy = inputs(24, 96, F32, F32)
    y = head.layer_norm_forward(x, w, b)[0]
    assert torch.equal(head.layer_norm_forward(x.view(2, 3, 4, 96), w, b)[0].view(24, 96), y)
    assert torch.equal(head.layer_norm_forward(x.t().contiguous().t(), w, b)[0], y)
    assert torch.equal(head.layer_norm_forward(x[:1].expand(5, 96), w, b)[0], y[:1].expand(5, 96))
    assert torch.equal(head.layer_norm_forward(x, w)[0], head.layer_norm_forward(x, w, torch.zeros_like(b))[0])


def test_deterministic_in_place_and_other_stream():
    from memory_lean_optimizer_gb300 import head
    x, w, b, dy = inputs(3000, 1111, BF, BF)
    first = head.layer_norm_forward(x, w, b)
    grads = head.layer_norm_backward(dy, x, w, *first[1:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = head.layer_norm_forward(x, w, b, stream=side)
    side_grads = head.layer_norm_backward(dy, x, w, *again[1:], stream=side)
    side.synchronize()
    for p, q in zip(first + grads, again + side_grads):
        assert torch.equal(p, q)
    s = torch.cuda.current_stream().cuda_stream
    n = lmopt.norm_layer_workspace(3000, 1111)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    g = dy.clone()
    dw, db = torch.empty_like(w), torch.empty_like(w)
    lmopt.norm_layer_backward(g.data_ptr(), 1111, x.data_ptr(), 1111, w.data_ptr(), first[1].data_ptr(),
                              first[2].data_ptr(), g.data_ptr(), 1111, dw.data_ptr(), db.data_ptr(), 3000, 1111,
                              lmopt.OPTIM_BF16, lmopt.OPTIM_BF16, work.data_ptr(), n, s)
    assert torch.equal(g, grads[0]) and torch.equal(dw, grads[1]) and torch.equal(db, grads[2])
    z = x.clone()
    lmopt.norm_layer_forward(z.data_ptr(), 1111, w.data_ptr(), b.data_ptr(), z.data_ptr(), 1111, None, None, 3000, 1111,
                             1e-5, lmopt.OPTIM_BF16, lmopt.OPTIM_BF16, s)
    assert torch.equal(z, first[0])


@pytest.mark.parametrize("want", ["dx", "dweight", "dbias"])
def test_single_outputs(want):
    from memory_lean_optimizer_gb300 import head
    x, w, b, dy = inputs(100, 520, BF, BF)
    y, mean, rstd = head.layer_norm_forward(x, w, b)
    full = dict(zip(("dx", "dweight", "dbias"), head.layer_norm_backward(dy, x, w, mean, rstd)))
    n = lmopt.norm_layer_workspace(100, 520)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(full[want])
    p = {k: (out.data_ptr() if k == want else None) for k in full}
    lmopt.norm_layer_backward(dy.data_ptr(), 520, x.data_ptr(), 520, w.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
                              p["dx"], 520, p["dweight"], p["dbias"], 100, 520, lmopt.OPTIM_BF16, lmopt.OPTIM_BF16,
                              work.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, full[want])


def test_gradient_against_differences():
    """Autograd's gradients of sum(y c) against central differences of the 64-bit formula along random
    directions: step h = 1e-4 leaves a truncation error of h^2 times third derivatives of order one."""
    from memory_lean_optimizer_gb300 import head
    x, w, b, c = (t.requires_grad_() for t in inputs(6, 300, F32, F32))
    (head.layer_norm(x, w, b) * c.detach()).sum().backward()

    def f(X, W, B):
        xc = X - X.mean(1, keepdim=True)
        return float(((xc / (xc.pow(2).mean(1, keepdim=True) + 1e-5).sqrt() * W + B) * c.detach().double()).sum())
    p = [t.detach().double() for t in (x, w, b)]
    h = 1e-4
    for i, t in enumerate((x, w, b)):
        d = torch.randn_like(p[i])
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + h * d, p[i] - h * d
        slope = (f(*hi) - f(*lo)) / (2 * h)
        got = float((t.grad.double() * d).sum())
        scale = float((t.grad.double() * d).abs().sum())
        assert abs(got - slope) <= 1e-5 * scale + 1e-6


def test_rows_past_2_31_elements():
    from memory_lean_optimizer_gb300 import head
    rows, dim = 65600, 32768
    x = torch.empty(rows, dim, dtype=BF, device="cuda")
    pick = [0, 1, 65534, 65535, 65536, rows - 1]
    base, w, b, dy = inputs(len(pick), dim, BF, BF)
    x.fill_(1.0)
    x[pick] = base
    y, mean, rstd = head.layer_norm_forward(x, w, b)
    small = head.layer_norm_forward(base, w, b)
    assert torch.equal(y[pick], small[0]) and torch.equal(mean[pick], small[1])
    g = torch.zeros_like(x)
    g[pick] = dy
    del y
    dx, dw, db = head.layer_norm_backward(g, x, w, mean, rstd)
    ref = head.layer_norm_backward(dy, base, w, *small[1:])
    assert torch.equal(dx[pick], ref[0])
    # the other rows add exact zeros; the order of the six sums may differ
    xh = (base.double() - small[1].double()[:, None]) * small[2].double()[:, None]
    tol = 64 * U * (dy.double() * xh).abs().sum(0)
    want = (dy.double() * xh).sum(0)
    assert within(dw, want, tol)


def test_refusals():
    from memory_lean_optimizer_gb300 import head
    x, w, b, dy = inputs(4, 64, BF, BF)
    mean = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        head.layer_norm_forward(x.half(), w)
    with pytest.raises(ValueError):
        head.layer_norm_forward(x, w[:32])
    with pytest.raises(ValueError):
        head.layer_norm_forward(x, w, b.float())
    with pytest.raises(ValueError):
        head.layer_norm_forward(x.cpu(), w)
    with pytest.raises(ValueError):
        head.layer_norm_backward(dy[:3], x, w, mean, mean)
    with pytest.raises(ValueError):
        head.layer_norm_backward(dy, x, w, mean[:2], mean)
    P = x.data_ptr()
    ok = dict(x=P, ldx=64, weight=w.data_ptr(), bias=None, y=P, ldy=64, mean=None, rstd=None, rows=4, dim=64, eps=1e-5,
              x_type=0, w_type=0)
    for bad, code in ((dict(rows=-1), lmopt.OPTIM_EINVAL), (dict(dim=0), lmopt.OPTIM_EINVAL),
                      (dict(ldx=63), lmopt.OPTIM_EINVAL), (dict(ldy=1), lmopt.OPTIM_EINVAL),
                      (dict(x=None), lmopt.OPTIM_EINVAL), (dict(weight=None), lmopt.OPTIM_EINVAL),
                      (dict(x_type=2), lmopt.OPTIM_EINVAL), (dict(eps=-1.0), lmopt.OPTIM_EINVAL),
                      (dict(eps=float("nan")), lmopt.OPTIM_EINVAL), (dict(y=P + 1), lmopt.OPTIM_EALIGN),
                      (dict(mean=P + 2), lmopt.OPTIM_EALIGN)):
        with pytest.raises(lmopt.LmoptError) as e:
            lmopt.norm_layer_forward(**{**ok, **bad})
        assert e.value.code == code, bad
    with pytest.raises(lmopt.LmoptError):            # no workspace for the weight's gradient
        lmopt.norm_layer_backward(P, 64, P, 64, P, mean.data_ptr(), mean.data_ptr(), None, 64, P, None, 4, 64, 0, 0,
                                  None, 0)
    with pytest.raises(lmopt.LmoptError):
        lmopt.norm_layer_backward(P, 64, P, 64, P, mean.data_ptr(), mean.data_ptr(), None, 64, P, None, 4, 64, 0, 0,
                                  P, 16)
