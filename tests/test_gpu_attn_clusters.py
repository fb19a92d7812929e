"""Tiles of keys that several CTAs share (a cluster, whose sums are joined over distributed shared memory): against the formulas in 64 bits, with
non-finite values in masked places and in seen ones; and gradients of sequences longer than a few tiles."""
import pytest
import torch

from test_gpu_attn import BF, borders, check, inputs

pytestmark = pytest.mark.gpu


def shared_by(rows, heads, kv, lengths, sms):
    """CTAs that share each tile of keys (the rule of csrc/attn_backward.cu), tile by tile of every sequence."""
    units, most = (rows // 128 + len(lengths) + 2) * kv, -(-rows // 64) * (heads // kv)
    splits = 1
    while splits < 8 and 2 * units * splits <= sms and most >= 2 * splits * 12:
        splits *= 2
    return [min(splits, max(1, -(-(n - at) // 64) * (heads // kv) // 12)) for n in lengths for at in range(0, n, 128)]


def cover(rows, heads, kv, lengths, want):
    """The shape is one that a GPU of this many SMs shares as meant."""
    assert set(want) <= set(shared_by(rows, heads, kv, lengths, torch.cuda.get_device_properties(0).multi_processor_count))


@pytest.mark.parametrize("dim", [64, 72, 128])
@pytest.mark.parametrize("lengths,want", [([1025], {1, 2, 3, 4, 6, 7, 8}), ([500, 1, 520], {1, 2, 3, 4, 5, 6}), ([960], {2, 4, 6, 7, 8})],
                         ids=["one", "several", "whole_blocks"])
def test_against_the_formulas(lengths, want, dim):
    rows = sum(lengths)
    cover(rows, 8, 1, lengths, want)
    check(*inputs(rows, 8, 1, dim), lengths)


def test_rows_of_no_sequence():
    lengths = [900, 70]
    q, k, v, do = inputs(1025, 8, 1, 64)
    cover(1025, 8, 1, lengths, {8})
    clean = check(q, k, v, do, lengths, 3)
    for t in (q, k, v, do):
        t[:3] = float("nan")
        t[973:] = float("inf")
    got = check(q, k, v, do, lengths, 3)
    assert all(torch.equal(got[n], clean[n]) for n in clean)


def test_masked_values_do_not_reach():
    """NaN and infinities of one row, on both sides of the tiles' borders and in the last block, which is not whole: nothing that does not
    see them changes."""
    from memory_lean_optimizer_gb300 import block
    lengths = [940, 85]
    q, k, v, do = inputs(1025, 8, 1, 80)
    cover(1025, 8, 1, lengths, {8})
    cu = borders(lengths)
    out, lse = block.attention_forward(q, k, v, cu)
    grads = block.attention_backward(do, q, k, v, out, lse, cu)
    for at in (0, 63, 64, 127, 128, 500, 895, 896, 930, 939, 940, 1003, 1004, 1024):
        start, end = (0, 940) if at < 940 else (940, 1025)
        other = [i for i in range(1025) if not start <= i < end]
        for bad in (float("nan"), float("inf"), -float("inf")):
            for which in range(3):
                t = [x.clone() for x in (q, k, v)]
                t[which][at] = bad
                o, l = block.attention_forward(*t, cu)
                dq, dk, dv = block.attention_backward(do, *t, o, l, cu)
                keep = [i for i in range(1025) if not at <= i < end] if which else [i for i in range(1025) if i != at]
                assert torch.equal(o[keep], out[keep]) and torch.equal(dq[keep], grads[0][keep]), (at, bad, which)
                free = other + ([i for i in range(at + 1, end)] if which == 0 else [])
                assert torch.equal(dk[free], grads[1][free]) and torch.equal(dv[free], grads[2][free]), (at, bad, which)
            g = do.clone()
            g[at] = bad
            dq, dk, dv = block.attention_backward(g, q, k, v, out, lse, cu)
            keep, free = [i for i in range(1025) if i != at], [i for i in range(1025) if not start <= i <= at]
            assert torch.equal(dq[keep], grads[0][keep]) and not dq[at].isfinite().any()
            assert torch.equal(dk[free], grads[1][free]) and torch.equal(dv[free], grads[2][free])
            assert not dk[start:at + 1].isfinite().any() and not dv[start:at + 1].isfinite().any()


@pytest.mark.parametrize("at", [0, 40, 127, 300, 959, 1000, 1024])
def test_one_infinite_gradient_stays_in_its_column(at):
    """What a block with masked places has cleared comes back for the keys that the row sees, once, whichever CTA had the block."""
    from memory_lean_optimizer_gb300 import block
    q, k, v, do = inputs(1025, 8, 1, 64)
    cover(1025, 8, 1, [1025], {8})
    out, lse = block.attention_forward(q, k, v)
    want = block.attention_backward(do, q, k, v, out, lse)[2]
    for bad in (float("inf"), -float("inf")):
        g = do.clone()
        g[at, 5, 7] = bad
        dv = block.attention_backward(g, q, k, v, out, lse)[2]
        other = [i for i in range(64) if i != 7]
        assert torch.equal(dv[..., other], want[..., other]) and torch.equal(dv[at + 1:], want[at + 1:])
        assert bool((dv[:at + 1, 0, 7] == bad).all())
    g[at, 2, 7] = float("inf")                    # another head's, of the other sign
    dv = block.attention_backward(g, q, k, v, out, lse)[2]
    assert bool(dv[:at + 1, 0, 7].isnan().all()) and torch.equal(dv[at + 1:], want[at + 1:])


@pytest.mark.parametrize("rows,heads,kv,dim", [(3000, 4, 2, 128), (1025, 8, 1, 64)])
def test_nothing_finite(rows, heads, kv, dim):
    """All of the gradients say so."""
    from memory_lean_optimizer_gb300 import block
    for bad in (float("nan"), float("inf")):
        q, k, v, do = (torch.full_like(t, bad) for t in inputs(rows, heads, kv, dim))
        out, lse = block.attention_forward(q, k, v)
        assert not lse.isfinite().any()
        assert not any(t.isfinite().any() for t in (out, *block.attention_backward(do, q, k, v, out, lse)))


@pytest.mark.parametrize("rows,heads,kv,dim", [(4200, 2, 1, 64), (3300, 4, 4, 128), (2500, 3, 1, 80)])
def test_long_sequences(rows, heads, kv, dim):
    check(*inputs(rows, heads, kv, dim), [rows])
