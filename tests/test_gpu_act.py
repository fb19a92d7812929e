"""Activations in 8 bits and the gated activation, against their definitions in 64 bits.

The codes are exact: powers of two and one rounding to nearest even, the same in 64 bits.  The gated activation in fp32:
s(g) = 1 / (1 + e^-g) is off by at most k u (u = 2^-24) of its value for bounded g, where k covers the exponential's
argument (|g| u in bf16's approximate form: |g| + 4) and the few roundings behind it; g s u adds two roundings and
the gradient's polynomial s (1 + g (1 - s)) at most (3 k + 6) u (1 + |g|).  The rounding to the output's type is monotone."""
import pytest
import torch

from test_gpu_norm import within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (3, 2), (5, 31), (2, 32), (7, 33), (300, 64), (9, 80), (40, 1000), (3, 2047), (17, 4096), (2, 20001)]


def kept64(x):
    """(codes, exponent bytes) of a matrix in 64 bits; finite values."""
    n, c = x.shape
    y = torch.zeros(n, -(-c // 32) * 32, dtype=torch.float64, device=x.device)
    y[:, :c] = x
    y = y.view(n, -1, 32)
    top = y.abs().amax(2)
    e = (torch.frexp(top)[1] - 1 + 127).clamp(min=0)
    e = torch.where(top > 0, e, torch.zeros_like(e))
    code = lambda e: torch.round(y * torch.exp2(133.0 - e.double())[..., None])
    e = torch.where(code(e).abs().amax(2) > 127, e + 1, e).clamp(max=254)
    return code(e).clamp(-127, 127), e


def matrix(rows, cols, dtype, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows + cols)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-30, 30, (rows, cols + pad), generator=g, device="cuda").float() / 4)
    return x.to(dtype)[:, :cols]


def check_pack(x):
    from memory_lean_optimizer_gb300 import block
    p = block.pack_activation(x)
    code, e = kept64(x)
    assert torch.equal(p.codes.double(), code.flatten(1)) and torch.equal(p.exponents.int(), e.int())
    y = block.unpack_activation(p)
    want = (code * torch.exp2(e.double() - 133)[..., None]).flatten(1)[:, :x.shape[1]]
    assert y.shape == x.shape and y.dtype == x.dtype and torch.equal(y.double(), want)
    return p


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack(rows, cols, dtype):
    check_pack(matrix(rows, cols, dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [1, 2, 4, 8])
def test_pack_strides(pad, dtype):
    check_pack(matrix(9, 96, dtype, pad=pad))
    x = matrix(9, 96, dtype, pad=pad)
    check_pack(x[:, 1:90])
    check_pack(x.t())
    check_pack(x[:1].expand(4, 96))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pack_every_exponent_and_border(dtype):
    """Blocks whose largest magnitude is each power of two from the smallest subnormal to the largest finite value, and the
    values on both sides of where the exponent goes up."""
    tops = [2.0 ** e for e in range(-149 if dtype == F32 else -133, 128)]
    mant = [1.0, 1.5, 127.0 / 64, 127.5 / 64] + ([1.9921874, 2 - 2.0 ** -23] if dtype == F32 else [])
    x = torch.zeros(len(tops) * len(mant), 32, dtype=torch.float64, device="cuda")
    x[:, 5] = torch.tensor([t * m for t in tops for m in mant], dtype=torch.float64)
    x[:, 6] = -x[:, 5]
    steps = torch.arange(26, device="cuda").double()
    x[:, 6:] = -x[:, 5:6] * (1 - steps / 51)        # ties and others between the codes
    x = x.to(dtype)
    check_pack(x[x.isfinite().all(1)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pack_zero_and_non_finite_blocks(dtype):
    from memory_lean_optimizer_gb300 import block
    x = matrix(6, 96, dtype)
    x[0, :32] = 0
    x[1, 40], x[2, 70], x[3, 0] = float("nan"), float("inf"), -float("inf")
    y = block.unpack_activation(block.pack_activation(x))
    bad = torch.zeros(6, 3, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 2] = bad[3, 0] = True
    assert torch.equal(y.view(6, 3, 32).isnan(), bad[:, :, None].expand(6, 3, 32))
    assert not y[0, :32].any()
    clean = block.unpack_activation(block.pack_activation(torch.where(x.isfinite(), x, torch.ones_like(x))))
    keep = ~bad[:, :, None].expand(6, 3, 32).reshape(6, 96)
    assert torch.equal(y[keep], clean[keep])


def test_pack_shapes_and_no_rows():
    from memory_lean_optimizer_gb300 import block
    x = matrix(6, 50, BF).view(2, 3, 50)
    p = block.pack_activation(x)
    assert p.codes.shape == (6, 64) and p.exponents.shape == (6, 2)
    assert block.unpack_activation(p).shape == (2, 3, 50)
    assert not p.codes[:, 50:].any()
    assert block.unpack_activation(block.pack_activation(x[:0])).shape == (0, 3, 50)


def swiglu64(g, u):
    return g * torch.sigmoid(g) * u


def check_swiglu(x, dh):
    from memory_lean_optimizer_gb300 import block
    c = dh.shape[1]
    h, p = block.swiglu_forward(x)
    assert torch.equal(block.swiglu_forward(x, keep=False)[0], h)
    pairs = block.pack_activation(x.reshape(-1, 2, c) if x.is_contiguous() else x.contiguous().view(-1, 2, c))
    assert torch.equal(p.codes, pairs.codes) and torch.equal(p.exponents, pairs.exponents)

    def k(g):
        return (g.abs() + 8) * U
    G, W = x[:, :c].double(), x[:, c:].double()
    tiny = 2.0 ** -126                                                      # where the approximate functions flush
    assert within(h, swiglu64(G, W), (k(G) + 4 * U) * swiglu64(G, W).abs() + tiny * (1 + W.abs()) * (1 + G.abs()))
    d, again = block.swiglu_backward(dh, p, need_h=True)
    kept = block.unpack_activation(p).view(-1, 2, c).double()
    G, W, D = kept[:, 0], kept[:, 1], dh.double()
    s = torch.sigmoid(G)
    assert within(again, swiglu64(G, W), (k(G) + 4 * U) * swiglu64(G, W).abs() + tiny * (1 + W.abs()) * (1 + G.abs()))
    slope = s * (1 + G * torch.sigmoid(-G))
    tol = (D * W).abs() * ((3 * k(G) + 6 * U) * s * (1 + G.abs()) + tiny * (1 + G.abs()))
    assert within(d[:, :c], D * W * slope, tol)
    assert within(d[:, c:], D * G * s, (k(G) + 4 * U) * (D * G * s).abs() + tiny * (1 + G.abs()) * (1 + D.abs()))
    assert torch.equal(block.swiglu_backward(dh, p)[0], d) and block.swiglu_backward(dh, p)[1] is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_swiglu(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = (torch.randn(rows, 2 * cols, generator=g, device="cuda") * 3).to(dtype)
    check_swiglu(x, torch.randn(rows, cols, generator=g, device="cuda").to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_swiglu_strides_and_far_gates(dtype):
    torch.manual_seed(0)
    wide = torch.randn(11, 200, device="cuda").to(dtype)
    check_swiglu(wide[:, 3:131], torch.randn(11, 80, device="cuda").to(dtype)[:, 5:69])
    x = torch.randn(8, 128, device="cuda")
    x[:, :64] = torch.linspace(-80, 80, 64, device="cuda")
    check_swiglu(x.to(dtype), torch.randn(8, 64, device="cuda").to(dtype))


def test_swiglu_extremes_stay_finite():
    from memory_lean_optimizer_gb300 import block
    for dtype in (BF, F32):
        x = torch.tensor([[-1e4, 1e4, -300.0, 0.0, 2.0, 3.0, -1.0, 5.0]], device="cuda").to(dtype)
        h, p = block.swiglu_forward(x)
        assert h[0, 0] == 0 and h[0, 1].float() == (x[0, 1] * x[0, 5]).float() and h[0, 2] == 0 and h[0, 3] == 0
        d, _ = block.swiglu_backward(torch.ones_like(h), p)
        assert bool(d.isfinite().all())


def test_swiglu_autograd_matches_the_calls():
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(1)
    x = torch.randn(4, 5, 96, device="cuda").to(BF).requires_grad_()
    dh = torch.randn(4, 5, 48, device="cuda").to(BF)
    h = block.swiglu(x)
    grad, = torch.autograd.grad(h, x, dh)
    want, packed = block.swiglu_forward(x.detach())
    assert torch.equal(h, want) and torch.equal(grad, block.swiglu_backward(dh, packed)[0])
    with torch.no_grad():
        assert torch.equal(block.swiglu(x), want)
    assert torch.equal(torch.autograd.grad(block.swiglu(x).sum(), x)[0], block.swiglu_backward(torch.ones_like(dh), packed)[0])


def test_gated_mlp_gradients():
    """Against the same products of what the calls give, and against 64 bits with the error of the 8-bit values."""
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(2)
    x, w1, w2 = (torch.randn(*s, device="cuda") * a for s, a in (((3, 50, 64), 1), ((192, 64), 0.2), ((64, 96), 0.2)))
    dy = torch.randn(3, 50, 64, device="cuda")
    for t in (x, w1, w2):
        t.requires_grad_()
    y = block.gated_mlp(x, w1, w2)
    with torch.no_grad():
        assert torch.equal(block.gated_mlp(x, w1, w2), y)
    grads = torch.autograd.grad(y, (x, w1, w2), dy, retain_graph=True)
    ref = [t.detach().double().requires_grad_() for t in (x, w1, w2)]
    gu = ref[0] @ ref[1].t()
    out = (torch.nn.functional.silu(gu[..., :96]) * gu[..., 96:]) @ ref[2].t()
    assert float((y.double() - out).abs().max()) < 1e-4 * float(out.abs().max())
    for got, want in zip(grads, torch.autograd.grad(out, ref, dy.double())):
        # each kept value is off by 2^-7 of its block's largest at most and by a third of that on average (a uniform
        # error has sqrt(1/3) of its bound): products of sums of many stay within 2^-6 in the 2-norm
        assert float((got.double() - want).norm()) < 2.0 ** -6 * float(want.norm())
    only = torch.autograd.grad(y, w2, dy)[0]
    assert torch.equal(only, grads[2])


def test_streams_and_graphs():
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(3)
    x, dh = torch.randn(60, 128, device="cuda").to(BF), torch.randn(60, 64, device="cuda").to(BF)
    h, p = block.swiglu_forward(x)
    d, again = block.swiglu_backward(dh, p, need_h=True)
    kept = block.unpack_activation(p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h2, p2 = block.swiglu_forward(x, stream=s)
    d2, again2 = block.swiglu_backward(dh, p2, need_h=True, stream=s)
    kept2 = block.unpack_activation(block.pack_activation(x.view(60, 2, 64), stream=s), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in ((h, h2), (d, d2), (again, again2), (kept, kept2)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h2, p2 = block.swiglu_forward(x)
        d2, _ = block.swiglu_backward(dh, p2)
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    h, p = block.swiglu_forward(x)
    assert torch.equal(h2, h) and torch.equal(d2, block.swiglu_backward(dh, p)[0])


def test_packed_from_codes_and_exponents():
    """A packed activation made from another's codes and exponents (a saved one) is the same; empty ones too."""
    from memory_lean_optimizer_gb300 import block
    x = torch.randn(3, 5, 70, device="cuda").to(BF)
    p = block.pack_activation(x)
    q = block.PackedActivation(p.codes.cpu(), p.exponents.cpu(), (3, 5, 70), BF)
    with pytest.raises(ValueError):
        block.unpack_activation(q)                       # not on the GPU
    q = block.PackedActivation(p.codes.clone(), p.exponents.t().contiguous().t(), p.shape, p.dtype)
    assert torch.equal(block.unpack_activation(q), block.unpack_activation(p))
    assert torch.equal(q.codes, p.codes) and torch.equal(q.exponents, p.exponents)
    e = block.pack_activation(x[:0])
    assert block.PackedActivation(e.codes, e.exponents, e.shape, e.dtype).data.numel() == 0
    assert block.unpack_activation(e).shape == (0, 5, 70)
