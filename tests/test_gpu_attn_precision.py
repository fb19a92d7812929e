"""How far the gradients of attention are off in the 2-norm, for weights of every kind: flat rows, rows whose weights lie on a few keys far into a
sequence, and keys and values with a mean of their own (as a projection with a bias has).  Attention's gradients do not change when a vector is added to all
keys of a sequence (sum_j dS_ij = 0), so neither out's rounding, which the delta that is formed from out carries, nor dS's must
reach them times such a vector, however long the rows.

Bounds.  A gradient is rounded once at its end, `own`: the distance of the formula's value from its rounding, which the test forms.  What the kernels
round before is formed too, from the formula's p and dS: a rounding of a weight a_ij that multiplies x_j, uncorrelated from the others, adds
|e_ij| |x_j| in quadrature.  For dq, x_j is k_j less the row's mean of the keys, for the rounded dS are made to sum to nothing, and for heads of
up to 80, which take dS in two parts, there is none of it.  Scores and dP in fp32 leave some 2^-20 of a weight and a dS, out's rounding
2^-9 of a correction that is itself 2^-8 of delta: together below 2^-11 of the gradient beside those.  A tenth for the quadrature's spread."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rounding(t):
    return t.to(BF).double() - t


def measure(q, k, v, do, lengths):
    """{gradient: (error, bound, size)} of rows behind the first 64 of their sequences (dq), and of all (dk, dv)."""
    from memory_lean_optimizer_gb300 import block
    rows, heads, d = q.shape
    kv = k.shape[1]
    g, scale = heads // kv, d ** -0.5
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    out, lse = block.attention_forward(q, k, v, cu)
    got = dict(zip(("dq", "dk", "dv"), block.attention_backward(do, q, k, v, out, lse, cu)))
    want = {n: torch.zeros(t.shape, dtype=torch.float64, device="cuda") for n, t in got.items()}
    var = dict.fromkeys(want, 0.0)
    at, far = 0, torch.zeros(rows, dtype=torch.bool, device="cuda")
    for n in lengths:
        s_, at = slice(at, at + n), at + n
        far[s_.start + 64:s_.stop] = True
        see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(heads):
            j = h // g
            Q, K, V, D = q[s_, h].double(), k[s_, j].double(), v[s_, j].double(), do[s_, h].double()
            p = ((Q @ K.t()) * scale).masked_fill(~see, -math.inf).softmax(1)
            dp = D @ V.t()
            ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
            want["dq"][s_, h] = ds @ K
            want["dk"][s_, j] += ds.t() @ Q
            want["dv"][s_, j] += p.t() @ D
            e = rounding(ds)
            var["dk"] += float((e.pow(2).t() @ Q.pow(2)).sum())
            var["dv"] += float((rounding(p).pow(2).t() @ D.pow(2)).sum())
            if d > 80:
                mean = p @ K
                two = e.pow(2)[64:]
                var["dq"] += float((two @ K.pow(2) - 2 * (two @ K) * mean[64:] + two.sum(1, keepdim=True) * mean[64:].pow(2)).sum())
    res = {}
    for n in got:
        rows_ = far if n == "dq" else slice(None)
        w = want[n][rows_]
        bound = 1.1 * math.sqrt(float(rounding(w).norm()) ** 2 + var[n]) + 2.0 ** -11 * float(w.norm())
        res[n] = float((got[n][rows_].double() - w).norm()), bound, float(w.norm())
    return res


def inputs(rows, heads, kv, dim, size, mean):
    gen = torch.Generator(device="cuda").manual_seed(rows + dim)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    return ((r(rows, heads, dim) * size).to(BF), (r(rows, kv, dim) + mean * r(1, kv, dim)).to(BF), (r(rows, kv, dim) + mean * r(1, kv, dim)).to(BF),
            (r(rows, heads, dim) * 0.1).to(BF))


@pytest.mark.parametrize("dim", [64, 80, 96, 128])
@pytest.mark.parametrize("size,mean", [(1, 0), (4, 0), (8, 0), (0.5, 1), (1, 4)], ids=["flat", "sharp", "sharper", "means", "large_means"])
def test_gradients_whatever_the_weights(size, mean, dim):
    for lengths in ([512], [300, 77, 640]):
        res = measure(*inputs(sum(lengths), 4, 2, dim, size, mean), lengths)
        print(dim, size, mean, lengths, {n: f"{e / s:.2e} of {b / s:.2e}" for n, (e, b, s) in res.items()})
        for n, (error, bound, _) in res.items():
            assert error <= bound, (n, lengths)


@pytest.mark.parametrize("dim", [64, 128])
def test_long_flat_rows_over_means(dim):
    """A mean of the keys beside thousands of weights: dq is small beside what the mean alone would give."""
    res = measure(*inputs(4100, 2, 1, dim, 0.5, 1), [4100])
    print(dim, {n: f"{e / s:.2e} of {b / s:.2e}" for n, (e, b, s) in res.items()})
    for n, (error, bound, _) in res.items():
        assert error <= bound, n
