"""The bounded waits inside the attention kernels, made to run out: one tile stops copying or keeps its weights back
(host-set, LMOPT_FAULT_INJECT=stall_attention*), so that what waits for it gives up after a tenth of a second.  The kernel
returns, the rows it held up are NaN, every other element is what it is without the injection, and the next call
is unharmed.  Nothing faults, traps or hangs: each wait ends by its own limit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


# 700 rows of 2 key heads leave SMs over: the tiles of keys are shared by clusters; 40 sequences do not
@pytest.mark.parametrize("lengths", [[700], [150] * 40], ids=["clusters", "alone"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("what", ["copy", "softmax"])
@pytest.mark.parametrize("kernel", ["", "_dq", "_dkv"])
def test_a_wait_that_runs_out_gives_nan_and_returns(kernel, what, dim, lengths, monkeypatch):
    from memory_lean_optimizer_gb300 import block
    rows = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(rows)
    q, k, v, do = (torch.randn(rows, h, dim, generator=g, device="cuda").to(torch.bfloat16) for h in (8, 2, 2, 8))
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    out, lse = block.attention_forward(q, k, v, cu)
    call = (lambda: block.attention_forward(q, k, v, cu)) if not kernel else (lambda: block.attention_backward(do, q, k, v, out, lse, cu))
    want = call()
    monkeypatch.setenv("LMOPT_FAULT_INJECT", f"stall_attention{kernel}_{what}")
    got = call()
    torch.cuda.synchronize()
    monkeypatch.delenv("LMOPT_FAULT_INJECT")
    tile = min(lengths[0], 256 if not kernel else 128)
    for i, (x, y) in enumerate(zip(got, want)):
        bad = x.isnan()
        assert torch.equal(x[~bad], y[~bad])
        if not kernel and i == 1:
            x = x.t()[:, :, None]
            bad = x.isnan()
        # the queries' kernel forms the deltas that the keys' gradients take
        reached = {"": (0, 1), "_dq": (0, 1), "_dkv": (1, 2)}[kernel]
        assert bool(bad.any()) == (i in reached)
        if i in reached:           # whole rows of the tile, of its head alone
            assert not bad[tile:].any() and not bad[:, 1:].any() and bool(bad[:tile, 0].any())
            if kernel:
                assert bool(bad[:tile, 0].all())
    for x, y in zip(call(), want):
        assert torch.equal(x, y)
