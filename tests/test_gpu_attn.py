"""Causal attention over packed sequences, forward and backward, against the formulas in 64 bits.

Tolerances, element by element, with u = 2^-24 and b = 2^-8 (bf16's rounding).  A product of d terms in the tensor cores, which cut low
bits, is within d 2 u of the sum of magnitudes: a score within es = scale d 2 u |q||k| + 4 u |s| (the change of base), so
p within r = es + |error of the reference| + 8 u of its value (approximate exponential: 4 u), and b more as it is rounded.
out: sum p |v| (b + 2 r + n 2 u), the 2 for the sum in the denominator.  Backward, with the given out and lse, whose distance from the exact
ones is known: delta within |dO| |out - o| + d u |dO||out|, dP within d 2 u |dO||v|, dS within p times those and |dP - delta| r, and
b |dS|; dq, dk, dv the sums of what these give, and n 2 u of the sums of magnitudes.  Second-order terms: a quarter more.
Weights below 2^-126, fp32's smallest normal value, are taken as 0 (the approximate exponential flushes, and so may a product with
them): p and dS are off by at most 2^-126 (1 and 1 + |dP - delta|) more, which counts where a key has only such weights.
The rounding to the output's type is monotone, so outputs lie between the rounded ends of the intervals."""
import math

import pytest
import torch

from test_gpu_norm import within

pytestmark = pytest.mark.gpu
U, B, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -126
BF = torch.bfloat16


def borders(lengths, first=0):
    return torch.tensor([first + sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def inputs(rows, heads, kv, dim, seed=0, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + rows)
    r = lambda h, a=1.0: (torch.randn(rows, h, dim, generator=g, device="cuda") * a).to(BF)
    return r(heads, size), r(kv, size), r(kv), r(heads, 0.1)


def reference(q, k, v, do, lengths, first, scale, out, lse):
    """Yields (what, rows, head, exact, tolerance) for every sequence and head."""
    rows, heads, d = q.shape
    kv = k.shape[1]
    g = heads // kv
    dk, dv, tk, tv = (torch.zeros(rows, kv, d, dtype=torch.float64, device="cuda") for _ in range(4))
    at = first
    for n in lengths:
        s_ = slice(at, at + n)
        at += n
        if n == 0:
            continue
        see = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        for h in range(heads):
            Q, K, V = q[s_, h].double(), k[s_, h // g].double(), v[s_, h // g].double()
            s = (Q @ K.t()) * scale
            es = scale * d * 2 * U * (Q.abs() @ K.abs().t()) + 4 * U * s.abs()
            L = torch.logsumexp(s.masked_fill(~see, -math.inf), 1)
            p = torch.where(see, (s - L[:, None]).exp(), torch.zeros_like(s))
            worst = (es * see).amax(1)
            r = es + worst[:, None] + 8 * U
            o = p @ V
            yield "lse", (h, s_), L, worst + (n + 16) * U + 4 * U * L.abs()
            yield "out", (s_, h), o, 1.25 * ((p * (B + 2 * r)) @ V.abs() + n * 2 * U * (p @ V.abs()))
            if do is None:
                continue
            D = do[s_, h].double()
            given = out[s_, h].double()
            delta = (D * o).sum(1, keepdim=True)
            e_delta = (D.abs() * (given - o).abs()).sum(1, keepdim=True) + d * U * (D.abs() * given.abs()).sum(1, keepdim=True)
            dp = D @ V.t()
            e_dp = d * 2 * U * (D.abs() @ V.abs().t())
            r = es + (lse[h, s_].double() - L).abs()[:, None] + 4 * U * L.abs()[:, None] + 8 * U
            ds = p * (dp - delta)
            e_ds = p * (r * (dp - delta).abs() + e_dp + e_delta) + B * ds.abs() + TINY * (1 + (dp - delta).abs()) * see
            yield "dq", (s_, h), scale * ds @ K, 1.25 * scale * (e_ds @ K.abs() + n * 2 * U * (ds.abs() @ K.abs()))
            j = h // g
            dk[s_, j] += scale * ds.t() @ Q
            tk[s_, j] += 1.25 * scale * (e_ds.t() @ Q.abs() + g * n * 2 * U * (ds.abs().t() @ Q.abs()))
            dv[s_, j] += p.t() @ D
            tv[s_, j] += 1.25 * ((p * (B + r) + TINY * see).t() @ D.abs() + g * n * 2 * U * (p.t() @ D.abs()))
    if do is not None:
        for j in range(kv):
            yield "dk", (slice(first, at), j), dk[first:at, j], tk[first:at, j]
            yield "dv", (slice(first, at), j), dv[first:at, j], tv[first:at, j]


def check(q, k, v, do, lengths, first=0, scale=None, cu="given"):
    from memory_lean_optimizer_gb300 import block
    cu = borders(lengths, first) if cu == "given" else cu
    out, lse = block.attention_forward(q, k, v, cu, scale)
    got = dict(out=out, lse=lse)
    if do is not None:
        got["dq"], got["dk"], got["dv"] = block.attention_backward(do, q, k, v, out, lse, cu, scale)
    for what, at, want, tol in reference(q, k, v, do, lengths, first, scale or q.shape[2] ** -0.5, out, lse):
        if what == "lse":
            assert bool(((lse[at].double() - want).abs() <= tol).all()), (what, at)
        else:
            assert within(got[what][at], want, tol), (what, at)
    end = first + sum(lengths)
    for name in ("out", "dq", "dk", "dv"):
        if name in got:
            assert not got[name][:first].any() and not got[name][end:].any(), name
    assert not lse[:, :first].any() and not lse[:, end:].any()
    return got


LENGTHS = [[1], [2], [37], [64], [65], [127], [128], [129], [192], [255], [256], [257], [640], [1000], [64, 1, 0, 130, 3], [1] * 40,
           [0, 0, 300, 0, 513, 0]]


@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda x: "-".join(map(str, x[:6])))
def test_lengths(lengths):
    q, k, v, do = inputs(sum(lengths), 2, 1, 64)
    check(q, k, v, do, lengths)


@pytest.mark.parametrize("dim", [8, 16, 24, 32, 40, 64, 72, 80, 96, 120, 128])
@pytest.mark.parametrize("heads,kv", [(1, 1), (6, 2)])
def test_head_sizes(heads, kv, dim):
    lengths = [130, 1, 200]
    check(*inputs(sum(lengths), heads, kv, dim), lengths)


@pytest.mark.parametrize("heads,kv", [(3, 3), (8, 1), (8, 4)])
def test_groups(heads, kv):
    check(*inputs(330, heads, kv, 128), [330])


@pytest.mark.parametrize("first,tail", [(0, 5), (3, 0), (130, 300), (1, 1)])
def test_rows_of_no_sequence(first, tail):
    from memory_lean_optimizer_gb300 import block
    lengths = [70, 129, 0, 5]
    rows = first + sum(lengths) + tail
    q, k, v, do = inputs(rows, 4, 2, 64)
    clean = check(q, k, v, do, lengths, first)
    for t in (q, k, v, do):                       # whatever they hold
        t[:first] = float("nan")
        t[rows - tail:] = float("inf")
    got = check(q, k, v, do, lengths, first)
    assert all(torch.equal(got[n], clean[n]) for n in clean)
    # no sequence at all
    out, lse = block.attention_forward(q, k, v, torch.tensor([first], dtype=torch.int32, device="cuda"))
    assert not out.any() and not lse.any()
    assert not any(t.any() for t in block.attention_backward(do, q, k, v, out, lse, torch.tensor([first], dtype=torch.int32, device="cuda")))


@pytest.mark.parametrize("size", [0.0, 0.05, 3.0, 8.0])
def test_flat_and_sharp_scores(size):
    """Scores from all equal to one key far above the others, and a reference that moves along the keys."""
    q, k, v, do = inputs(700, 2, 1, 64, size=size)
    check(q, k, v, do, [700])
    k = (k.float() + torch.linspace(0, size, 700, device="cuda")[:, None, None] * q[300, :1].float()).to(BF)
    check(q, k, v, do, [300, 400])


def test_scale():
    check(*inputs(150, 2, 2, 64), [150], scale=0.02)
    check(*inputs(150, 2, 2, 64), [150], scale=1.0)


def test_later_tokens_and_other_sequences_do_not_reach():
    """NaN and infinities in every place that is masked, for every row on both sides of the tiles' borders."""
    from memory_lean_optimizer_gb300 import block
    lengths = [200, 333]
    q, k, v, do = inputs(533, 4, 2, 80)
    cu = borders(lengths)
    out, lse = block.attention_forward(q, k, v, cu)
    grads = block.attention_backward(do, q, k, v, out, lse, cu)
    for at in (0, 1, 63, 64, 127, 128, 190, 199, 200, 263, 264, 328, 456, 520, 532):
        start, end = (0, 200) if at < 200 else (200, 533)
        for bad in (float("nan"), float("inf"), -float("inf")):
            for which in range(3):
                t = [x.clone() for x in (q, k, v)]
                t[which][at] = bad
                o, l = block.attention_forward(*t, cu)
                keep = [i for i in range(533) if not at <= i < end] if which else [i for i in range(533) if i != at]
                assert torch.equal(o[keep], out[keep]) and torch.equal(l[:, keep], lse[:, keep]), (at, bad, which)
                lost = [i for i in range(at, end)] if which else [at]
                assert bool((~o[lost].isfinite()).any(2).all()), (at, bad, which)
                dq, dk, dv = block.attention_backward(do, *t, o, l, cu)
                assert torch.equal(dq[keep], grads[0][keep]), (at, bad, which)
                # a row that is lost takes the keys that it sees with it; those behind it and other sequences are left
                free = [i for i in range(533) if not start <= i < end] + ([i for i in range(at + 1, end)] if which == 0 else [])
                assert torch.equal(dk[free], grads[1][free]) and torch.equal(dv[free], grads[2][free]), (at, bad, which)
            g = do.clone()
            g[at] = bad
            dq, dk, dv = block.attention_backward(g, q, k, v, out, lse, cu)
            keep = [i for i in range(533) if i != at]
            free = [i for i in range(533) if not start <= i <= at]
            assert torch.equal(dq[keep], grads[0][keep]) and not dq[at].isfinite().any()
            assert torch.equal(dk[free], grads[1][free]) and torch.equal(dv[free], grads[2][free])
            assert not dv[start:at + 1].isfinite().any()


def test_one_infinite_value_stays_in_its_column():
    from memory_lean_optimizer_gb300 import block
    q, k, v, do = inputs(300, 2, 1, 64)
    out, _ = block.attention_forward(q, k, v)
    v[100, 0, 7] = float("inf")
    got, _ = block.attention_forward(q, k, v)
    other = [i for i in range(64) if i != 7]
    assert torch.equal(got[..., other], out[..., other]) and torch.equal(got[:100], out[:100])
    assert bool((got[100:, :, 7] == float("inf")).all())


def test_strides_and_layouts():
    """q, k and v as views of one projection, heads outside tokens, off 16 bytes, and one head shown to all."""
    lengths = [100, 57]
    q, k, v, do = inputs(157, 4, 2, 64)
    want = check(q, k, v, do, lengths)

    def same(q, k, v, do):
        got = check(q, k, v, do, lengths)
        assert all(torch.equal(got[n], want[n]) for n in want)
    qkv = torch.cat((q, k, v, do), 1)
    same(qkv[:, :4], qkv[:, 4:6], qkv[:, 6:8], qkv[:, 8:])
    same(*(t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v, do)))
    wide = torch.zeros(157, 12, 67, dtype=BF, device="cuda")
    wide[:, :, 1:65] = qkv
    same(wide[:, :4, 1:65], wide[:, 4:6, 1:65], wide[:, 6:8, 1:65], wide[:, 8:, 1:65])
    same(*(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v, do)))
    one = k[:, :1].expand(157, 2, 64)
    got = check(q, one, v, do, lengths)
    again = check(q, one.contiguous(), v, do, lengths)
    assert all(torch.equal(got[n], again[n]) for n in got)
    check(q, k, v, do[:, :1].expand(157, 4, 64), lengths)


def test_batches_of_one_length():
    from memory_lean_optimizer_gb300 import block
    q, k, v, do = inputs(3 * 140, 4, 2, 64)
    want = check(q, k, v, do, [140] * 3)
    b = lambda t: t.view(3, 140, *t.shape[1:])
    out, lse = block.attention_forward(b(q), b(k), b(v))
    assert out.shape == (3, 140, 4, 64) and torch.equal(out.view(420, 4, 64), want["out"]) and torch.equal(lse, want["lse"])
    for got, name in zip(block.attention_backward(b(do), b(q), b(k), b(v), out, lse), ("dq", "dk", "dv")):
        assert torch.equal(got.flatten(0, 1), want[name])
    # no borders: one sequence
    assert torch.equal(block.attention_forward(q, k, v)[0], block.attention_forward(q, k, v, borders([420]))[0])
    # [batch, heads, length, dim] as many programs keep them
    t = lambda t: b(t).transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(block.attention_forward(t(q), t(k), t(v))[0], out)


def test_empty():
    from memory_lean_optimizer_gb300 import block
    q, k, v, do = inputs(0, 2, 1, 64)
    out, lse = block.attention_forward(q, k, v)
    assert out.shape == (0, 2, 64) and lse.shape == (2, 0)
    assert [t.shape for t in block.attention_backward(do, q, k, v, out, lse)] == [(0, 2, 64), (0, 1, 64), (0, 1, 64)]
    assert block.attention_forward(q.view(2, 0, 2, 64), k.view(2, 0, 1, 64), v.view(2, 0, 1, 64))[0].shape == (2, 0, 2, 64)


def test_runs_agree_bit_for_bit():
    from memory_lean_optimizer_gb300 import block
    lengths = [900, 3, 1500, 64]
    q, k, v, do = inputs(sum(lengths), 8, 2, 128)
    cu = borders(lengths)
    first = None
    for _ in range(5):
        out, lse = block.attention_forward(q, k, v, cu)
        got = (out, lse, *block.attention_backward(do, q, k, v, out, lse, cu))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    # a sequence's results do not depend on its place in the buffer
    alone = block.attention_forward(q[903:2403], k[903:2403], v[903:2403])
    assert torch.equal(alone[0], first[0][903:2403]) and torch.equal(alone[1], first[1][:, 903:2403])


def test_borders_that_make_no_sense_stay_in_the_buffers():
    from memory_lean_optimizer_gb300 import block
    q, k, v, do = inputs(500, 2, 1, 64)
    for cu in ([0, 9999999], [-5, 100, 500], [0, 400, 100, 500], [500, 0], [2 ** 31 - 1] * 3, [-2 ** 31, 2 ** 31 - 1]):
        t = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out, lse = block.attention_forward(q, k, v, t)
        block.attention_backward(do, q, k, v, out, lse, t)
    torch.cuda.synchronize()
    t = torch.tensor([0, 9999999], dtype=torch.int32, device="cuda")
    assert torch.equal(block.attention_forward(q, k, v, t)[0], block.attention_forward(q, k, v)[0])


def test_autograd_and_parts_of_the_gradient():
    from memory_lean_optimizer_gb300 import block
    lengths = [77, 200]
    q, k, v, do = inputs(277, 4, 2, 64)
    cu = borders(lengths)
    out, lse = block.attention_forward(q, k, v, cu)
    want = block.attention_backward(do, q, k, v, out, lse, cu)
    a, b, c = (t.clone().requires_grad_() for t in (q, k, v))
    y = block.attention(a, b, c, cu)
    assert torch.equal(y, out)
    assert all(torch.equal(g, w) for g, w in zip(torch.autograd.grad(y, (a, b, c), do, retain_graph=True), want))
    assert torch.equal(torch.autograd.grad(y, a, do)[0], want[0])
    y = block.attention(q, b, c, cu)
    assert torch.equal(torch.autograd.grad(y, c, do)[0], want[2])
    got = block.attention_backward(do, q, k, v, out, lse, cu, need_kv=False)
    assert torch.equal(got[0], want[0]) and got[1] is None and got[2] is None
    got = block.attention_backward(do, q, k, v, out, lse, cu, need_q=False)
    assert got[0] is None and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_gradients_against_differences():
    """The loss <out, g> in 64 bits at inputs moved along a direction, against the gradients' product with it."""
    from memory_lean_optimizer_gb300 import block
    q, k, v, do = inputs(90, 2, 1, 32)
    out, lse = block.attention_forward(q, k, v)
    grads = block.attention_backward(do, q, k, v, out, lse)

    def loss(q, k, v):
        s = torch.einsum("ihd,jhd->hij", q, k.expand(90, 2, 32)) / math.sqrt(32)
        s = s.masked_fill(torch.ones(90, 90, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        return float((torch.einsum("hij,jhd->ihd", s.softmax(2), v.expand(90, 2, 32)) * do.double()).sum())
    torch.manual_seed(0)
    for which in range(3):
        x = [t.double() for t in (q, k, v)]
        step = torch.randn_like(x[which])
        h = 1e-4
        x[which] = x[which] + h * step
        up = loss(*x)
        x[which] = x[which] - 2 * h * step
        slope = (up - loss(*x)) / (2 * h)
        g = grads[which].double()
        # p, dS and the gradient are rounded to bf16: 3 b of the gradient's size, along a random direction
        assert abs(float((g * step).sum()) - slope) <= 3 * B * float(g.norm()) * 4


def test_other_streams_and_graphs():
    from memory_lean_optimizer_gb300 import block
    lengths = [130, 260]
    q, k, v, do = inputs(390, 4, 2, 64)
    cu = borders(lengths)
    out, lse = block.attention_forward(q, k, v, cu)
    want = block.attention_backward(do, q, k, v, out, lse, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, l = block.attention_forward(q, k, v, cu, stream=s)
    got = block.attention_backward(do, q, k, v, o, l, cu, stream=s)
    s.synchronize()
    assert torch.equal(o, out) and all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = block.attention_forward(q, k, v, cu)
        got = block.attention_backward(do, q, k, v, o, l, cu)
    cu.copy_(borders([200, 190]))                 # other borders, the same graph
    g.replay()
    torch.cuda.synchronize()
    out, lse = block.attention_forward(q, k, v, cu)
    assert torch.equal(o, out) and all(torch.equal(a, b) for a, b in zip(got, block.attention_backward(do, q, k, v, out, lse, cu)))


def test_long():
    """Rows at the end of a long sequence, from the keys of all of it."""
    from memory_lean_optimizer_gb300 import block
    n, d = 20000, 64
    q, k, v, _ = inputs(n, 2, 1, d)
    out, lse = block.attention_forward(q, k, v)
    rows = slice(n - 40, n)
    for h in range(2):
        s = q[rows, h].double() @ k[:, 0].double().t() * d ** -0.5
        s = s.masked_fill(torch.arange(n, device="cuda")[None] > torch.arange(n - 40, n, device="cuda")[:, None], -math.inf)
        p = s.softmax(1)
        es = d ** -0.5 * d * 2 * U * (q[rows, h].double().abs() @ k[:, 0].double().abs().t()) + 4 * U * s.abs().nan_to_num(posinf=0.0)
        r = es + es.amax(1, keepdim=True) + 8 * U
        mag = p @ v[:, 0].double().abs()
        assert within(out[rows, h], p @ v[:, 0].double(), 1.25 * ((p * (B + 2 * r)) @ v[:, 0].double().abs() + n * 2 * U * mag))


@pytest.mark.parametrize("count", [300, 700, 3000])
def test_more_sequences_than_threads(count):
    """Tiles are looked up in one round of borders for as many sequences as a CTA has threads (256 and 384), in several for more."""
    from memory_lean_optimizer_gb300 import block
    g = torch.Generator().manual_seed(count)
    lengths = torch.randint(0, 6, (count,), generator=g)
    lengths[count // 3], lengths[-2] = 200, 130
    n = int(lengths.sum())
    q, k, v, do = inputs(n + 9, 2, 1, 32)
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), lengths.cumsum(0))).to(torch.int32).cuda()
    out, lse = block.attention_forward(q, k, v, cu)
    got = (out, lse.t()[..., None], *block.attention_backward(do, q, k, v, out, lse, cu))
    # the same sequences one by one, in a few places
    at = cu.tolist()
    for i in (0, 1, count // 3, count // 2, count - 2, count - 1):
        s = slice(at[i], at[i + 1])
        if at[i] == at[i + 1]:
            continue
        o, l = block.attention_forward(q[s], k[s], v[s])
        alone = (o, l.t()[..., None], *block.attention_backward(do[s], q[s], k[s], v[s], o, l))
        assert all(torch.equal(a[s], b) for a, b in zip(got, alone)), i
    assert not any(t[n:].any() for t in got)
    # and all of them against one batch of sequences of three
    if count == 700:
        three = torch.arange(0, n // 3 * 3 + 1, 3, dtype=torch.int32, device="cuda")
        m = n // 3 * 3
        a = block.attention_forward(q[:m], k[:m], v[:m], three)[0]
        b = block.attention_forward(*(t[:m].view(m // 3, 3, -1, 32) for t in (q, k, v)))[0]
        assert torch.equal(a, b.flatten(0, 1))


def test_two_streams_at_once():
    """Calls on two streams, among them the cross entropy's products, which use tensor memory too: each as by itself."""
    from memory_lean_optimizer_gb300 import block, head
    sets = [inputs(600 + 100 * i, 8, 2, 64, seed=i) for i in range(2)]
    h, w = torch.randn(300, 256, device="cuda").to(BF), torch.randn(5000, 256, device="cuda").to(BF)
    t = torch.randint(5000, (300,), device="cuda")

    def work(i):
        q, k, v, do = sets[i]
        out, lse = block.attention_forward(q, k, v)
        return (out, lse, *block.attention_backward(do, q, k, v, out, lse), *head.xent_forward(h, w, t))
    want = [work(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(work(i))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, want[i]))


def test_first_calls_of_a_thread():
    """In a thread that has made no CUDA call yet (nothing to allocate either: the allocator has the memory)."""
    import threading
    from memory_lean_optimizer_gb300 import block, head
    q, k, v, do = inputs(200, 4, 2, 64)
    h, w, t = q.flatten(1), torch.randn(3000, 256, device="cuda").to(BF), torch.randint(3000, (200,), device="cuda")
    want = block.attention_forward(q, k, v)
    grads = block.attention_backward(do, q, k, v, *want)
    loss = head.xent_forward(h, w, t)
    x = head.xent_backward(h, w, t, loss[1], torch.ones_like(loss[0]))
    del grads
    grads = block.attention_backward(do, q, k, v, *want)
    torch.cuda.synchronize()
    for call, ref in ((lambda: block.attention_forward(q, k, v), want), (lambda: block.attention_backward(do, q, k, v, *want), grads),
                      (lambda: head.xent_forward(h, w, t), loss), (lambda: head.xent_backward(h, w, t, loss[1], torch.ones_like(loss[0])), x),
                      (lambda: (block.unpack_activation(block.pack_activation(q)),), (block.unpack_activation(block.pack_activation(q)),))):
        got, error = [], []

        def run():
            try:
                got.extend(call())
            except Exception as e:      # a thread's exceptions stay in it
                error.append(e)
        thread = threading.Thread(target=run)
        thread.start()
        thread.join()
        torch.cuda.synchronize()
        assert not error and all(torch.equal(a, b) for a, b in zip(got, ref)), error


def test_gradients_of_broadcast_inputs_and_of_one_sequence():
    """A key head shown to several, a gradient that is one number everywhere, no borders: autograd sums what was shared."""
    from memory_lean_optimizer_gb300 import block
    q, k, v, _ = inputs(190, 4, 1, 64)
    a, b, c = (t.clone().requires_grad_() for t in (q, k, v))
    y = block.attention(a, b.expand(190, 2, 64), c.expand(190, 2, 64))
    y.sum().backward()                                  # the gradient of y is one expanded element
    out, lse = block.attention_forward(q, k.expand(190, 2, 64), v.expand(190, 2, 64))
    dq, dk, dv = block.attention_backward(torch.ones_like(q), q, k.expand(190, 2, 64), v.expand(190, 2, 64), out, lse)
    assert torch.equal(a.grad, dq) and torch.equal(b.grad, dk.sum(1, keepdim=True)) and torch.equal(c.grad, dv.sum(1, keepdim=True))
    # two heads that share a key head outright: the same sums, one rounding less
    y = block.attention(a, b, c)
    got = torch.autograd.grad(y, (b, c), torch.ones_like(y))
    for one, two in zip(got, (dk, dv)):
        # each of the two was rounded, and their sum, and this one
        assert bool(((one.double() - two.double().sum(1, keepdim=True)).abs() <= 2 * B * two.double().abs().sum(1, keepdim=True) + 2 ** -20).all())
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(block.attention(a, b, c).float().pow(2).sum(), a, create_graph=True)
        g.sum().backward()


def test_nothing_finite():
    """A training run that has blown up: every call still returns, and says so."""
    from memory_lean_optimizer_gb300 import block
    for bad in (float("nan"), float("inf")):
        q, k, v, do = (torch.full_like(t, bad) for t in inputs(3000, 4, 2, 128))
        out, lse = block.attention_forward(q, k, v)
        got = block.attention_backward(do, q, k, v, out, lse)
        torch.cuda.synchronize()
        assert not out.isfinite().any() and not any(t.isfinite().any() for t in got[:1])


@pytest.mark.parametrize("lengths", [[2] * 20, [9], [6, 3, 8, 13, 2, 11] * 4, [64] * 4, [65, 100]], ids=["two", "nine", "few", "block", "tile"])
def test_gradients_of_queries_that_see_few_keys(lengths):
    """out's rounding, 2^-8 of a mean that is not small beside its values here, must not reach dq: in the 2-norm dq is off by its own rounding
    (as the formula's, rounded) and by no more than 2^-11 beside it.  What is left: dS in two parts (2^-17), and the correction's
    own rounding, 2^-8 of a correction of 2^-8 delta |sum p k|, which stays below 2^5 |dq| for these inputs."""
    from memory_lean_optimizer_gb300 import block
    rows = sum(lengths)
    q, k, v, do = inputs(rows, 8, 2, 64)
    cu = borders(lengths)
    out, lse = block.attention_forward(q, k, v, cu)
    dq = block.attention_backward(do, q, k, v, out, lse, cu)[0]
    qd, kd, vd = (t.double().requires_grad_() for t in (q, k, v))
    outs, at = [], 0
    for n in lengths:
        s = torch.einsum("ihd,jhd->hij", qd[at:at + n], kd[at:at + n].repeat_interleave(4, 1)) * 64 ** -0.5
        s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -math.inf)
        outs.append(torch.einsum("hij,jhd->ihd", s.softmax(2), vd[at:at + n].repeat_interleave(4, 1)))
        at += n
    want = torch.autograd.grad(torch.cat(outs), qd, do.double())[0]
    rounded = float((want.to(BF).double() - want).norm())
    assert float((dq.double() - want).norm()) <= 1.02 * rounded + 2.0 ** -11 * float(want.norm())
