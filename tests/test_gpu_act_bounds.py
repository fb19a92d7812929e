"""How far an activation in 8 bits is off: half a step of its block, and what that is of the block's largest magnitude."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(x):
    """x [rows, 32 n], finite: the bounds that pack_activation states, in exact arithmetic (powers of two and differences in 64 bits)."""
    from memory_lean_optimizer_gb300 import block
    p = block.pack_activation(x)
    y = x.double().view(x.shape[0], -1, 32)
    error = (block.unpack_activation(p).double().view_as(y) - y).abs().amax(2)
    top, e = y.abs().amax(2), p.exponents.double()
    step = torch.exp2(e - 133)
    last = (e == 254) & (top >= 127.5 * step)               # the step cannot grow
    assert bool((error <= step / 2)[~last].all()) and bool((error < step)[last].all())
    inside = (e >= 1) & ~last
    assert bool((error * 127.5 <= top)[inside].all())
    return error, top, inside


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_exponent(dtype):
    g = torch.Generator(device="cuda").manual_seed(0)
    top = torch.exp2(torch.arange(-149 if dtype == F32 else -133, 128, device="cuda").double())
    mant = torch.cat((torch.tensor([1.0, 127.0 / 64, 127.5 / 64, 2 - 2.0 ** -8, 1.9921874, 2 - 2.0 ** -23], device="cuda").double(),
                      1 + torch.rand(20, generator=g, device="cuda").double()))
    x = torch.rand(len(top) * len(mant), 32, generator=g, device="cuda").double() * 2 - 1
    x[:, 7] = 1
    # the other codes' middles, among them 1 under 127.5: half a step of 2
    x[:, 8], x[:, 9], x[:, 10] = 1 / 127.5, -3 / 127.5, 0.5 / 63.75
    x = (x * (top[:, None] * mant).reshape(-1, 1)).to(dtype)
    check(x[x.isfinite().all(1)])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_bound_is_reached(dtype):
    """127.5 and 1: the step is 2, and 1 lies half of it from either code; more than 2^-7 of the largest."""
    x = torch.zeros(1, 32, device="cuda", dtype=dtype)
    x[0, 0], x[0, 1] = 127.5, 1.0
    error, top, inside = check(x)
    assert bool(inside.all()) and float(error) == 1.0 and float(error) > 2.0 ** -7 * float(top)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_ordinary_values(dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    check((torch.randn(4000, 512, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (4000, 1), generator=g, device="cuda").float())).to(dtype))
