"""Cross entropy at sizes that make a call take the vocabulary in several pieces in every way it can: with a weight
that is copied piece by piece, with dH's K split over the pieces, with a last piece so narrow that a split of
it is empty.  Against 64 bits, with the tolerances of test_gpu_xent.py."""
import pytest
import torch

from test_gpu_xent import BF, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,extra", [(20, 1), (20, 232), (300, 5000)])
def test_copied_weight_in_several_pieces(rows, extra):
    """4095 columns are copied to 4096, 32768 words to 256 MiB: forward and backward take two pieces."""
    check(*inputs(rows, 4095, 32768 + extra, ignored=0.2))


@pytest.mark.parametrize("extra", [1, 700])
def test_split_k_over_several_pieces(extra):
    """4096 rows hold 32768 words of E in 256 MiB, 512 columns are 32 tiles for 76 pairs of CTAs: two pieces, two
    splits; one word more leaves the second split of the last piece empty."""
    check(*inputs(4096, 512, 32768 + extra))


def test_copied_weight_and_split_k_over_several_pieces():
    h, w, t, c = inputs(4096, 512, 33000, ignored=0.5)
    check(h[:, 1:511], w[:, 1:511], t, c)


def test_three_pieces_of_a_copied_weight_deterministic():
    from memory_lean_optimizer_gb300 import head
    h, w, t, c = inputs(130, 8191, 3 * 16384 - 100)          # 16384 words to a piece
    first = head.xent_forward(h, w, t)
    grads = head.xent_backward(h, w, t, first[1], c)
    for a, b in zip(first + grads, head.xent_forward(h, w, t) + head.xent_backward(h, w, t, first[1], c)):
        assert torch.equal(a, b)
    wide = torch.zeros(w.shape[0], 8192, dtype=BF, device="cuda")     # the same matrix, addressed in place: one piece
    wide[:, :8191] = w
    loss, lse = head.xent_forward(h, wide[:, :8191], t)
    assert torch.equal(loss, first[0]) and torch.equal(lse, first[1])


def test_long_sums_of_one_sign_do_not_drift():
    """The tensor cores cut an accumulator towards zero at each of its additions (16 products): at most 2^-23 of what it
    holds, which grows evenly when all products have one sign.  An accumulator of 1024 products, 64 additions, loses
    32 * 2^-23 of its sum at most; sums of accumulators are rounded.  One accumulator of all 4096 would lose up to four
    times that, and more than this bound if its cuts are evenly spread (0.72 of the most, over magnitudes, halved)."""
    from memory_lean_optimizer_gb300 import head
    g = torch.Generator(device="cuda").manual_seed(5)
    h = torch.randn(256, 4096, generator=g, device="cuda").abs().to(BF)
    w = (torch.randn(3000, 4096, generator=g, device="cuda").abs() * 0.02).to(BF)
    t = torch.zeros(256, dtype=torch.int64, device="cuda")
    lse = head.xent_forward(h, w, t)[1].double()
    ref = torch.logsumexp(h.double() @ w.double().t(), 1)
    drift = float(((lse - ref) / ref).mean())
    print(f"mean relative error of lse {drift:.3g}")
    assert abs(drift) <= 32 * 2.0 ** -23 + 4 * 2.0 ** -24
