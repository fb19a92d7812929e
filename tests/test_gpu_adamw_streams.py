"""AdamW groups used on a stream that is not the current one, with one of the two kept busy: nothing that a call makes
on its way may run on the other stream, and what it reads is not given away before it is done."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, weight_decay=0.01)
SIZES = [100, 5000, 300001]
BUSY = 200_000_000     # clock ticks, about a tenth of a second


def masters():
    g = torch.Generator(device="cuda").manual_seed(0)
    return [torch.randn(n, generator=g, device="cuda") * 0.02 for n in SIZES]


def gradients(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * 1e-3).to(torch.bfloat16) for n in SIZES]


def state(group):
    return group.weights + group.res + group.m + group.v


def take_free_memory(value):
    """Writes what the current stream's allocator gives out: small, middle and large pieces, more than was freed."""
    out = [torch.full((n,), value, device="cuda") for n in [1] * 64 + [50, 2500, 150001, 300001, 600002] * 24]
    return out


@pytest.fixture
def side():
    s = torch.cuda.Stream()
    yield s
    torch.cuda.synchronize()


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_unpacked_states_are_not_cleared_behind_the_call(states, side):
    from memory_lean_optimizer_gb300 import engine
    group = engine.AdamWGroup.from_masters(masters(), states=states)
    group.step(gradients(1), HP)
    want = [x.clone() for x in group.unpack_states()]
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)                     # the current stream; the call's own is free
    got = group.unpack_states(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_group_made_and_stepped_on_another_stream(states, side):
    from memory_lean_optimizer_gb300 import engine
    # masters that have to be laid out first
    wide = [torch.stack((x, x), 1) for x in masters()]
    grads = gradients(1)
    want = engine.AdamWGroup.from_masters([x[:, 0] for x in wide], states=states)
    want.step(grads, HP)
    del_me = take_free_memory(7.0)              # what is freed holds nothing that would pass for a master
    del del_me
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    group = engine.AdamWGroup.from_masters([x[:, 0] for x in wide], stream=side, states=states)
    group.step(grads, HP, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(state(group), state(want)):
        assert torch.equal(a, b)


def test_gradients_freed_after_the_call_are_still_read_whole(side):
    from memory_lean_optimizer_gb300 import engine
    a, b = (engine.AdamWGroup.from_masters(masters()) for _ in range(2))
    a.step(gradients(1), HP, grad_scale=torch.full((1,), 0.5, device="cuda"))
    grads, scale = gradients(1), torch.full((1,), 0.5, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    b.step(grads, HP, stream=side, grad_scale=scale)
    del grads, scale
    junk = take_free_memory(7.0)
    torch.cuda.synchronize()
    for x, y in zip(state(a), state(b)):
        assert torch.equal(x, y)
    del junk


def test_buffers_freed_after_unpacking_are_written_whole(side):
    from memory_lean_optimizer_gb300 import engine
    group = engine.AdamWGroup.from_masters(masters())
    group.step(gradients(1), HP)
    flats = [torch.zeros(group.unpacked_numel(), device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    group.unpack_states(*flats, stream=side)
    del flats
    fresh = take_free_memory(7.0)
    torch.cuda.synchronize()
    assert all(bool((x == 7.0).all()) for x in fresh)
