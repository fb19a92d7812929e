"""The bounded waits inside the cross entropy's product kernels, made to run out: one cluster stops copying or keeps
its accumulators (host-set, LMOPT_FAULT_INJECT=stall_*), so that what waits for it gives up after a tenth of a
second.  The kernel returns, whatever it held up is NaN, every other element is what it is without
the injection, and the next call is unharmed.  Nothing faults, traps or hangs: each wait ends by its
own limit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# 600 rows take pairs of CTAs, 100 single ones; a cluster that only keeps its accumulators is noticed at its third
# tile, which the sizes give the first cluster in the cases listed
CASES = [(role, what, rows) for rows in (600, 100) for role in ("stats", "grad", "hidden", "weight") for what in ("copy", "peer")
         if rows == 600 or what == "copy"]
CASES += [("stats", "free", 600), ("grad", "free", 600), ("weight", "free", 600), ("weight", "free", 100)]


@pytest.mark.parametrize("role,what,rows", CASES)
def test_a_wait_that_runs_out_gives_nan_and_returns(role, what, rows, monkeypatch):
    from memory_lean_optimizer_gb300 import head
    g = torch.Generator(device="cuda").manual_seed(rows)
    h = torch.randn(rows, 512, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(30000, 512, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    t = torch.randint(30000, (rows,), generator=g, device="cuda")
    c = torch.rand(rows, generator=g, device="cuda") + 0.5
    lse = head.xent_forward(h, w, t)[1]
    call = (lambda: head.xent_forward(h, w, t)) if role == "stats" else (lambda: head.xent_backward(h, w, t, lse, c))
    want = call()
    monkeypatch.setenv("LMOPT_FAULT_INJECT", f"stall_{role}_{what}")
    got = call()
    torch.cuda.synchronize()
    monkeypatch.delenv("LMOPT_FAULT_INJECT")
    spoilt = [x.isnan() for x in got]
    for x, y, bad in zip(got, want, spoilt):
        assert torch.equal(x[~bad], y[~bad])
    if role in ("hidden", "weight"):      # the other gradient does not wait for it
        assert bool(spoilt[role == "weight"].any()) and not spoilt[role != "weight"].any()
    else:
        assert all(bool(bad.any()) for bad in spoilt)
    for x, y in zip(call(), want):
        assert torch.equal(x, y)
