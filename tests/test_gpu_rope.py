"""Rotary positions, forward and backward, against the formulas in 64 bits.

Tolerances, with u = 2^-24: sine and cosine are taken of an angle within an eighth of a turn that is rounded once
(0.79 u at most in either), to 1 ulp each (2 u), and multiplied by the factor (1 u); products and the sum round
once each: 2 u of |a| + |b|.  8 u (|a| + |b|) factor holds all of it.  The rounding to the output's type is monotone, so the
output lies between the rounded ends of that interval."""
from fractions import Fraction

import pytest
import torch

from test_gpu_norm import within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
DRAWN = dict(none=dict(), linear=dict(scaling="linear", factor=4.0), ntk=dict(scaling="ntk", factor=4.0),
             yarn=dict(scaling="yarn", factor=4.0, original_length=4096))


def turned(x, angle, factor, interleaved):
    """x turned in 64 bits, and |a| + |b| of each pair in both of its places."""
    r = 2 * angle.shape[-1]
    f = x.double()
    c, s = angle.cos()[:, None] * factor, angle.sin()[:, None] * factor
    first, second = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    a, b = f[..., first], f[..., second]
    y, size = f.clone(), torch.zeros_like(f)
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    size[..., first] = size[..., second] = a.abs() + b.abs()
    return y, size


def check(q, k, pos, plan, angle):
    from memory_lean_optimizer_gb300 import block
    for fn, sign in ((block.rotary_forward, 1), (block.rotary_backward, -1)):
        for x, y in zip((q, k), fn(q, k, pos, plan)):
            want, size = turned(x, sign * angle, plan.factor, plan.interleaved)
            assert y.shape == x.shape and y.dtype == x.dtype and y.is_contiguous()
            assert within(y, want, 8 * U * plan.factor * size)
            assert torch.equal(y[..., plan.rotary_dim:], x[..., plan.rotary_dim:])


def angles(pos, plan_args):
    from memory_lean_optimizer_gb300 import block
    freq, _ = block.rotary_frequencies(**plan_args)
    return pos.double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,heads,kv,dim,rotary", [(1, 1, 1, 2, 2), (5, 3, 1, 64, 64), (33, 4, 2, 80, 40), (7, 2, 2, 81, 36),
                                                      (130, 5, 1, 128, 128), (3, 1, 1, 6, 2), (9, 2, 1, 48, 0), (2, 2, 1, 1024, 1024),
                                                      (20000, 2, 1, 64, 32)])
def test_sizes(rows, heads, kv, dim, rotary, dtype, interleaved):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(rows + dim)
    q, k = (torch.randn(rows, h, dim, device="cuda").to(dtype) for h in (heads, kv))
    pos = torch.randint(1 << 20, (rows,), device="cuda")
    check(q, k, pos, block.RotaryPlan(rotary, interleaved=interleaved), angles(pos, dict(rotary_dim=rotary)))


@pytest.mark.parametrize("scaling", sorted(DRAWN))
def test_scalings(scaling):
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(1)
    q, k = (torch.randn(50, h, 64, device="cuda") for h in (4, 2))
    pos = torch.randint(1 << 15, (50,), device="cuda")
    check(q, k, pos, block.RotaryPlan(64, **DRAWN[scaling]), angles(pos, dict(rotary_dim=64, **DRAWN[scaling])))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad,start", [(0, 0), (8, 0), (7, 0), (2, 1), (4, 2), (16, 4)])
def test_strides_and_alignment(pad, start, dtype, interleaved):
    """q and k cut from one projection's rows, off every vector width."""
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(2)
    x = torch.randn(21, 6 * 64 + pad + start, device="cuda").to(dtype)
    q, k = x[:, start:start + 256].view(21, 4, 64), x[:, start + 256:start + 384].view(21, 2, 64)
    pos = torch.arange(21, device="cuda").flip(0)[::1]
    check(q, k, pos, block.RotaryPlan(64, interleaved=interleaved), angles(pos, dict(rotary_dim=64)))
    # heads outside tokens, and one head shown to all
    q, k = q.transpose(0, 1).contiguous().transpose(0, 1), k[:, :1].expand(21, 3, 64)
    check(q, k, pos, block.RotaryPlan(64, interleaved=interleaved), angles(pos, dict(rotary_dim=64)))


def test_far_and_negative_positions():
    """Angles in exact rational arithmetic: positions up to 2^31 and beyond, and negative ones."""
    from memory_lean_optimizer_gb300 import block
    where = [0, 1, -1, 4096, 10 ** 6, 2 ** 31 - 1, 2 ** 31, -2 ** 31, 2 ** 40 + 12345, 999999937]
    freq, _ = block.rotary_frequencies(64)
    two_pi = 2 * block._PI
    angle = torch.tensor([[float((p * Fraction(f) / two_pi) % 1 * two_pi) for f in freq] for p in where], dtype=torch.float64,
                         device="cuda")
    torch.manual_seed(3)
    q, k = (torch.randn(len(where), h, 64, device="cuda") for h in (2, 1))
    check(q, k, torch.tensor(where, device="cuda"), block.RotaryPlan(64), angle)


def test_backward_is_the_transpose_and_autograd_runs_it():
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(4)
    plan = block.RotaryPlan(32, interleaved=True, scaling="yarn", factor=8.0, original_length=128)
    q, k = (torch.randn(17, h, 48, device="cuda", requires_grad=True) for h in (4, 2))
    pos = torch.randint(1000, (17,), device="cuda")
    a, b = block.rotary(q, k, pos, plan)
    ga, gb = torch.randn_like(a), torch.randn_like(b)
    dq, dk = torch.autograd.grad((a, b), (q, k), (ga, gb))
    # <R q, g> = <q, R^T g>: both sides summed in 64 bits; each element is off by 8 u of its pair's size
    for x, y, g, d in ((q, a, ga, dq), (k, b, gb, dk)):
        left, right = (y.double() * g.double()).sum(), (x.double() * d.double()).sum()
        bound = 2 * 8 * U * plan.factor * 2 * float(x.detach().abs().max()) * float(g.double().abs().sum())
        assert abs(float(left - right)) <= bound
    # one of the two without a gradient
    a, _ = block.rotary(q, k.detach(), pos, plan)
    assert torch.equal(torch.autograd.grad(a, q, ga)[0], dq)


def test_no_tokens_no_key_heads_and_in_place():
    from memory_lean_optimizer_gb300 import block, lmopt
    plan = block.RotaryPlan(64)
    q, k = block.rotary_forward(torch.zeros(0, 2, 64, device="cuda"), torch.zeros(0, 1, 64, device="cuda"),
                                torch.zeros(0, dtype=torch.int64, device="cuda"), plan)
    assert q.shape == (0, 2, 64)
    torch.manual_seed(5)
    x, pos = torch.randn(12, 2, 64, device="cuda"), torch.arange(12, device="cuda")
    q, k = block.rotary_forward(x, x[:, :0], pos, plan)
    assert k.shape == (12, 0, 64)
    p = x.data_ptr()
    lmopt.rope_apply((p, 128, 64, p, 128, 64, 2), (None, 0, 0, None, 0, 0, 0), pos.data_ptr(), plan.turns.data_ptr(), 12, 64, 64,
                     1.0, False, False, lmopt.OPTIM_F32, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(x, q)


def test_another_stream_and_a_graph():
    from memory_lean_optimizer_gb300 import block
    torch.manual_seed(6)
    plan = block.RotaryPlan(64)
    q, k, pos = torch.randn(40, 4, 64, device="cuda"), torch.randn(40, 2, 64, device="cuda"), torch.arange(40, device="cuda")
    want = block.rotary_forward(q, k, pos, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = block.rotary_forward(q, k, pos, plan, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = block.rotary_forward(q, k, pos, plan)
    q.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0] * 2) and torch.equal(got[1], want[1])
