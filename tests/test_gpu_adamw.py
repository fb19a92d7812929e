"""AdamW groups against a plain implementation of the formulas: every product, sum, root and quotient
rounded once to fp32 with numpy (bit for bit), the same update in 64 bits (within rounding), and the
8-bit storage's own definition.

Tolerances of the 64-bit comparison: the fp32 sequence of the update makes at most 12 roundings of
relative size 2^-24 on quantities no larger than |w|, |update|, m or v, so m and v are held to
4 * 2^-24 of their terms' magnitudes and the master weight to 2 * 2^-24 |w| + 12 * 2^-24 |update|
(written 2^-20 |update|)."""
import numpy as np
import pytest
import torch

from helpers import alloc_offset
from memory_lean_optimizer_gb300 import lmopt

pytestmark = pytest.mark.gpu

HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
SIZES = [1, 7, 255, 256, 257, 4095, 4096, 4097, 4352, 4353, 5000, 16383, 16384, 16385, 32768, 40001, 100003]
f32 = np.float32


def scalars(hp, t):
    b1, b2, lr, wd = (float(f32(hp[k])) for k in ("beta1", "beta2", "lr", "weight_decay"))
    return dict(b1=f32(b1), omb1=f32(1 - b1), b2=f32(b2), omb2=f32(1 - b2), eps=f32(hp["eps"]), lr_wd=f32(lr * wd),
                k1=f32(lr / (1 - b1 ** t)), k2=f32(1 / np.sqrt(1 - b2 ** t)))


def blocks(x):
    n = x.size
    pad = np.zeros(-(-n // 256) * 256, x.dtype)
    pad[:n] = x
    return pad.reshape(-1, 256)


def encode(x, signed):
    b = blocks(x)
    top = np.where(np.isfinite(b), np.abs(b), 0).max(1).astype(f32)
    one = f32(1)
    q = np.sqrt(top) * (one / f32(127)) if signed else np.sqrt(np.sqrt(top)) * (one / f32(255))
    with np.errstate(all="ignore"):
        r = np.where(q > 0, np.minimum(one / (q * q), np.finfo(f32).max), f32(0)).astype(f32)[:, None]
        y = np.sqrt(np.abs(b) * r) if signed else np.sqrt(np.sqrt(b) * r)
    y = np.rint(np.fmin(y, f32(127 if signed else 255)))
    if signed:
        code = 128 + np.where(np.signbit(b), -y, y)
    else:
        code = np.where(b != 0, np.fmax(y, f32(1)), f32(0))
    return code.astype(np.uint8).reshape(-1)[:x.size], q


def decode(code, q, signed):
    n = code.size
    c = blocks(code).astype(f32)
    with np.errstate(invalid="ignore"):
        if signed:
            t = (c - f32(128)) * q[:, None]
            x = t * np.abs(t)
        else:
            z = c * q[:, None]
            x = (z * z) * (z * z)
    return x.reshape(-1)[:n]


class Plain:
    """fp32 AdamW state of one tensor, one rounding per operation."""

    def __init__(self, master, packed, kahan=True):
        self.hi_lo = master.view(np.uint32).copy()
        if not kahan:
            self.hi_lo = rne(master) << 16
        self.packed, self.kahan = packed, kahan
        n = master.size
        zero = np.zeros(n, f32)
        nb = -(-n // 256)
        self.m = (np.zeros(n, np.uint8), np.zeros(nb, f32)) if packed else zero
        self.v = (np.zeros(n, np.uint8), np.zeros(nb, f32)) if packed else zero.copy()

    def step(self, g, t, hp, gs=1.0):
        k = scalars(hp, t)
        with np.errstate(all="ignore"):
            g = g.astype(f32) * f32(gs)
            m = decode(*self.m, True) if self.packed else self.m
            v = decode(*self.v, False) if self.packed else self.v
            m = k["b1"] * m + k["omb1"] * g
            v = k["b2"] * v + k["omb2"] * (g * g)
            w = self.hi_lo.view(f32)
            w = w - k["lr_wd"] * w
            w = w - (k["k1"] * m) / (np.sqrt(v) * k["k2"] + k["eps"])
        self.fm, self.fv = m, v
        self.m = encode(m, True) if self.packed else m
        self.v = encode(v, False) if self.packed else v
        self.hi_lo = w.astype(f32).view(np.uint32).copy() if self.kahan else rne(w) << 16


def rne(x):
    return torch.from_numpy(np.ascontiguousarray(x, f32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16).astype(np.uint32)


def make(n, rng, std=0.02):
    return (rng.standard_normal(n) * std).astype(f32)


def grad(n, rng, std=1e-3):
    return torch.from_numpy((rng.standard_normal(n) * std).astype(f32)).to(torch.bfloat16)


def group_for(masters, states, kahan=True, align=0):
    from memory_lean_optimizer_gb300 import engine
    ws, rs = [], []
    for x in masters:
        _, w = alloc_offset(x.size, torch.bfloat16, align)
        _, r = alloc_offset(x.size, torch.int16, align)
        if kahan:
            hi, lo = engine.kahan_split(torch.from_numpy(x).cuda())
            w.copy_(hi)
            r.copy_(lo)
        else:
            w.copy_(torch.from_numpy(x).cuda().to(torch.bfloat16))
        ws.append(w)
        rs.append(r if kahan else None)
    return engine.AdamWGroup(ws, rs if kahan else None, kahan=kahan, states=states)


def check(plain, group, states):
    from memory_lean_optimizer_gb300 import engine
    for i, p in enumerate(plain):
        n = group.weights[i].numel()
        hi = group.weights[i].view(torch.int16).cpu().numpy().view(np.uint16)
        assert np.array_equal(hi, (p.hi_lo >> 16).astype(np.uint16)), f"tensor {i} (n={n}): weights"
        if p.kahan:
            lo = group.res[i].cpu().numpy().view(np.uint16)
            assert np.array_equal(lo, (p.hi_lo & 0xFFFF).astype(np.uint16)), f"tensor {i} (n={n}): residuals"
        for buf, x, name in ((group.m[i], p.m, "m"), (group.v[i], p.v, "v")):
            if p.packed:
                codes, q = engine.u8_state_views(buf, n)
                assert np.array_equal(codes.cpu().numpy(), x[0]), f"tensor {i} (n={n}): {name} codes"
                assert np.array_equal(q.cpu().numpy().view(np.uint32), x[1].astype(f32).view(np.uint32)), f"tensor {i}: {name} scales"
            else:
                # -0.0 and 0.0 both stand for an untouched moment
                assert np.array_equal(buf.cpu().numpy(), x, equal_nan=True), f"tensor {i} (n={n}): {name}"


@pytest.mark.parametrize("states", ["u8", "fp32"])
@pytest.mark.parametrize("align", [0, 1])
def test_bit_exact_over_sizes(states, align):
    rng = np.random.default_rng(0)
    masters = [make(n, rng) for n in SIZES]
    plain = [Plain(x, states == "u8" and x.size > 4096) for x in masters]
    group = group_for(masters, states, align=align)
    gs = torch.tensor([0.75], device="cuda")
    for t in range(1, 4):
        grads = [grad(n, rng) for n in SIZES]
        for p, g in zip(plain, grads):
            p.step(g.float().numpy(), t, HP, 0.75)
        dev = [alloc_offset(n, torch.bfloat16, align)[1].copy_(g) for n, g in zip(SIZES, grads)]
        group.step(dev, HP, grad_scale=gs)
        check(plain, group, states)
    group.close()


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_no_residual_rounds_to_nearest(states):
    rng = np.random.default_rng(1)
    sizes = [300, 5001]
    masters = [make(n, rng) for n in sizes]
    plain = [Plain(x, states == "u8" and x.size > 4096, kahan=False) for x in masters]
    group = group_for(masters, states, kahan=False)
    for t in (1, 2):
        grads = [grad(n, rng) for n in sizes]
        for p, g in zip(plain, grads):
            p.step(g.float().numpy(), t, HP)
        group.step([g.cuda() for g in grads], HP)
        check(plain, group, states)


def degenerate(kind, n, rng, t):
    g = (rng.standard_normal(n) * 1e-3).astype(f32)
    if kind == "zero" or (kind == "zero_then" and t < 3):
        g[:] = 0
    if kind == "subnormal":
        g *= f32(1e-36)
    if kind == "large":
        g *= f32(1e21)
    if kind == "two_scales":
        g[: n // 2] *= f32(1e-20)
        g[n // 2:] *= f32(1e6)
    if kind == "sparse_blocks":
        g[np.arange(n) % 512 >= 256] = 0
        g[0] = 1.0
    return torch.from_numpy(g).to(torch.bfloat16)


@pytest.mark.parametrize("states", ["u8", "fp32"])
@pytest.mark.parametrize("kind", ["zero", "zero_then", "subnormal", "large", "two_scales", "sparse_blocks"])
def test_degenerate_gradients_bit_exact(states, kind):
    rng = np.random.default_rng(2)
    sizes = [100, 4100, 9000]
    masters = [make(n, rng) for n in sizes]
    plain = [Plain(x, states == "u8" and x.size > 4096) for x in masters]
    group = group_for(masters, states)
    hp = dict(HP, beta1=0.0) if kind == "two_scales" else HP
    for t in range(1, 5):
        grads = [degenerate(kind, n, rng, t) for n in sizes]
        for p, g in zip(plain, grads):
            p.step(g.float().numpy(), t, hp)
        group.step([g.cuda() for g in grads], hp)
        check(plain, group, states)
    assert lmopt.optim_query_nonfinite(group.handle) == 0


def test_non_finite_gradient_stays_in_its_elements():
    """An infinity or a NaN spoils its own weight only: its block's scale, and so its neighbours' states, are
    those of the finite values."""
    rng = np.random.default_rng(3)
    n = 8192
    master = make(n, rng)
    plain = [Plain(master, True)]
    group = group_for([master], "u8")
    g = grad(n, rng)
    g[300], g[5000] = float("nan"), float("inf")
    plain[0].step(g.float().numpy(), 1, HP)
    group.step([g.cuda()], HP)
    from memory_lean_optimizer_gb300 import engine
    good = np.ones(n, bool)
    good[[300, 5000]] = False
    for buf, x in ((group.m[0], plain[0].m), (group.v[0], plain[0].v)):
        codes, q = engine.u8_state_views(buf, n)
        assert np.array_equal(codes.cpu().numpy()[good], x[0][good])
        assert np.array_equal(q.cpu().numpy(), x[1])
    w = torch.cat([x.view(-1) for x in group.masters()]).cpu().numpy()
    assert np.array_equal(w[good], plain[0].hi_lo.view(f32)[good]) and not np.isfinite(w[~good]).any()
    assert lmopt.optim_query_nonfinite(group.handle) in (1, 2)


def test_against_64_bits():
    rng = np.random.default_rng(4)
    n = 50000
    master = make(n, rng)
    group = group_for([master], "fp32")
    w, m, v = master.astype(np.float64), np.zeros(n), np.zeros(n)
    lr, b1, b2, eps, wd = (float(f32(HP[k])) for k in ("lr", "beta1", "beta2", "eps", "weight_decay"))
    for t in range(1, 6):
        g = grad(n, rng)
        g64 = g.double().numpy()
        m = b1 * m + (1 - b1) * g64
        v = b2 * v + (1 - b2) * g64 ** 2
        upd = lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
        w = w * (1 - lr * wd) - upd
        group.step([g.cuda()], HP)
    got = group.masters()[0].cpu().numpy().astype(np.float64)
    u = 2.0 ** -24
    assert np.all(np.abs(group.m[0].cpu().numpy() - m) <= 5 * 4 * u * (np.abs(m) + 1e-3))
    assert np.all(np.abs(group.v[0].cpu().numpy() - v) <= 5 * 4 * u * (v + 1e-6))
    # 5 steps; m near zero keeps an absolute error of its terms, which the update divides by sqrt(v)
    slack = 5 * 20 * u * lr * 10
    assert np.all(np.abs(got - w) <= 5 * (2 * u * np.abs(w) + 2.0 ** -20 * lr) + slack)


def test_codes_hold_values_within_half_a_step():
    """The stored moment differs from the computed one by at most half a code step on the companded scale:
    |sqrt(m) - sqrt(stored)| <= q / 2, |v^(1/4) - stored^(1/4)| <= q / 2 (one step up for values kept from
    zero), plus the codec's own fp32 roundings (4 * 2^-24 of the block's largest root)."""
    rng = np.random.default_rng(5)
    n = 20000
    master = make(n, rng)
    plain, group = Plain(master, True), group_for([master], "u8")
    g = grad(n, rng)
    plain.step(g.float().numpy(), 1, HP)
    group.step([g.cuda()], HP)
    m, v = (x.cpu().numpy().astype(np.float64) for x in group.unpack_states())
    qm, qv = np.repeat(plain.m[1], 256)[:n].astype(np.float64), np.repeat(plain.v[1], 256)[:n].astype(np.float64)
    sm = np.sign(plain.fm) * np.sqrt(np.abs(plain.fm.astype(np.float64)))
    assert np.all(np.abs(np.sign(m[:n]) * np.sqrt(np.abs(m[:n])) - sm) <= qm * (0.5 + 127 * 4 * 2.0 ** -24))
    sv, dv = plain.fv.astype(np.float64) ** 0.25, v[:n] ** 0.25
    assert np.all(np.abs(dv - sv) <= qv * np.where(dv < 1.5 * qv, 1.0, 0.5 + 255 * 4 * 2.0 ** -24) + 1e-300)


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_unpack_states_layout(states):
    from memory_lean_optimizer_gb300 import engine
    rng = np.random.default_rng(6)
    sizes = [5, 0, 4097, 64, 9001]
    group = group_for([make(n, rng) for n in sizes], states)
    group.step([grad(n, rng).cuda() for n in sizes], HP)
    flats = [torch.full((group.unpacked_numel() + 1,), 7.0, device="cuda")[1:] for _ in range(2)]   # 4-byte aligned
    group.unpack_states(*flats)
    at = 0
    for i, n in enumerate(sizes):
        for buf, flat, signed in ((group.m[i], flats[0], True), (group.v[i], flats[1], False)):
            want = buf.cpu().numpy()
            if states == "u8" and n > 4096:
                codes, q = engine.u8_state_views(buf, n)
                want = decode(codes.cpu().numpy(), q.cpu().numpy(), signed)
            assert np.array_equal(flat[at:at + n].cpu().numpy(), want)
            assert bool((flat[at + n:at + (n + 63) // 64 * 64] == 7.0).all())
        at += (n + 63) // 64 * 64


@pytest.mark.parametrize("states", ["u8", "fp32"])
@pytest.mark.parametrize("form", ["host", "engine"])
def test_offloaded_equals_resident(states, form):
    from memory_lean_optimizer_gb300 import engine
    rng = np.random.default_rng(7)
    sizes = [100, 4097, 70001]
    masters = [torch.from_numpy(make(n, rng)).cuda() for n in sizes]
    a = engine.AdamWGroup.from_masters(masters, states=states)
    eng = None
    if form == "engine":
        kind = lmopt.OPTIM_KIND_ADAMW_U8 if states == "u8" else lmopt.OPTIM_KIND_ADAMW
        eng = engine.OffloadEngine(engine.offload_slot_bytes(sizes, kind=kind))
        b = engine.AdamWGroup.from_masters(masters, states=states, offload=eng)
    else:
        b = engine.AdamWGroup.from_masters(masters, states=states)
        b.attach_host()
    for t in range(3):
        grads = [grad(n, rng).cuda() for n in sizes]
        a.step(grads, HP)
        if form == "host":
            b.prefetch()
        b.step(grads, HP)
        if form == "host":
            b.writeback()
    torch.cuda.synchronize()
    (eng.sync if eng else engine.OffloadEngine.sync_library_ring)()
    for i in range(len(sizes)):
        assert torch.equal(a.weights[i], b.weights[i])
        for x, y in ((a.res[i], b.res[i]), (a.m[i], b.m[i]), (a.v[i], b.v[i])):
            assert torch.equal(x.cpu(), y.cpu())
    with pytest.raises(lmopt.LmoptError) as e:
        b.unpack_states()
    assert e.value.code == lmopt.OPTIM_ESTATE
    b.close()
    if eng:
        eng.close()


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_resume_and_second_stream_bit_identical(states):
    """A run cut after two steps and resumed from its buffers on another stream equals the uninterrupted one."""
    from memory_lean_optimizer_gb300 import engine
    rng = np.random.default_rng(8)
    sizes = [33, 12345]
    masters = [torch.from_numpy(make(n, rng)).cuda() for n in sizes]
    grads = [[grad(n, rng).cuda() for n in sizes] for _ in range(4)]
    a = engine.AdamWGroup.from_masters(masters, states=states)
    b = engine.AdamWGroup.from_masters(masters, states=states)
    for t in range(4):
        a.step(grads[t], HP)
    for t in range(2):
        b.step(grads[t], HP)
    c = engine.AdamWGroup([w.clone() for w in b.weights], [r.clone() for r in b.res], states=states)
    for i in range(len(sizes)):
        c.m[i].copy_(b.m[i])
        c.v[i].copy_(b.v[i])
    c.set_step(2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (2, 3):
        c.step(grads[t], HP, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(a.weights + a.res + a.m + a.v, c.weights + c.res + c.m + c.v):
        assert torch.equal(x, y)


def test_stochastic_rounding_reproducible_and_unbiased():
    """Without a residual: two runs agree, the stored weight is one of the two neighbours of the fp32
    update, and rounds up as often as the dropped part says (binomial bound, 5 sigma)."""
    n = 40000
    master = np.full(n, 1.0, f32)
    hp = dict(HP, lr=2.0 ** -9 * 0.3, weight_decay=0.0, stochastic_rounding=1, seed=11, eps=0.0)
    out = []
    for _ in range(2):
        group = group_for([master], "u8", kahan=False)
        group.step([torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")], hp)
        out.append(group.weights[0].float().cpu().numpy())
    assert np.array_equal(out[0], out[1])
    lo, hi = 1.0 - 2.0 ** -8, 1.0                 # step 1 moves every weight by lr; bf16 step below 1 is 2^-8
    assert set(np.unique(out[0])) <= {lo, hi}
    p = 1 - 2.0 ** -9 * 0.3 / 2.0 ** -8
    assert abs((out[0] == hi).mean() - p) < 5 * np.sqrt(p * (1 - p) / n) + 2.0 ** -14


def test_refusals():
    from memory_lean_optimizer_gb300 import engine
    w = torch.zeros(5000, dtype=torch.bfloat16, device="cuda")
    group = engine.AdamWGroup([w])
    g = torch.zeros_like(w)

    def code(fn):
        with pytest.raises(lmopt.LmoptError) as e:
            fn()
        return e.value.code
    for bad in (dict(lr=-1.0), dict(beta1=1.0), dict(beta2=float("nan")), dict(eps=-1e-8),
                dict(weight_decay=float("inf")), dict(stochastic_rounding=2)):
        assert code(lambda: group.step([g], dict(HP, **bad))) == lmopt.OPTIM_EINVAL
    hp = lmopt.AdamWHparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
    assert code(lambda: lmopt.optim_step_adamw(group.handle, [g.data_ptr()], 2, hp)) == lmopt.OPTIM_EINVAL
    assert code(lambda: lmopt.optim_step_adamw(group.handle, [None], 1, hp)) == lmopt.OPTIM_EINVAL
    assert code(lambda: lmopt.optim_step_adamw(group.handle, [g.data_ptr() + 1], 1, hp)) == lmopt.OPTIM_EALIGN
    assert code(lambda: lmopt.optim_step_adamw(group.handle, [g.data_ptr()], 1, hp, g.data_ptr() + 2)) == lmopt.OPTIM_EALIGN
    nadam = engine.NadamGroup([w])
    assert code(lambda: lmopt.optim_step_adamw(nadam.handle, [g.data_ptr()], 1, hp)) == lmopt.OPTIM_EINVAL
    assert code(lambda: lmopt.optim_group_unpack_state(nadam.handle, w.data_ptr(), w.data_ptr())) == lmopt.OPTIM_EINVAL
    assert code(lambda: lmopt.optim_group_unpack_state(group.handle, None, w.data_ptr())) == lmopt.OPTIM_EINVAL
    assert code(lambda: lmopt.optim_group_unpack_state(group.handle, w.data_ptr() + 2, w.data_ptr())) == lmopt.OPTIM_EALIGN
    group.step([g], HP)                             # the refused calls changed nothing
    assert group.step_count == 1
    assert lmopt.optim_query_launches(group.handle) == 1


@pytest.mark.parametrize("states", ["u8", "fp32"])
def test_hooks_step_adamw_groups(states):
    from memory_lean_optimizer_gb300.hooks import attach_fused_adamw
    torch.manual_seed(0)
    model = torch.nn.Sequential(torch.nn.Linear(128, 256), torch.nn.GELU(), torch.nn.Linear(256, 64)).cuda().to(torch.bfloat16)
    params = list(model.parameters())
    plain = [Plain(p.detach().float().cpu().numpy().reshape(-1), states == "u8" and p.numel() > 4096) for p in params]
    seen = {}
    stepper = attach_fused_adamw(params, 2, HP, states=states,
                                 on_step=lambda gi, gr: seen.setdefault(gi, []).append([g.float().cpu().numpy().reshape(-1) for g in gr]))
    x = torch.randn(16, 128, device="cuda", dtype=torch.bfloat16)
    for _ in range(2):
        model(x).float().pow(2).mean().backward()
    for gi, idx in enumerate(stepper.index):
        for t in (1, 2):
            for i, g in zip(idx, seen[gi][t - 1]):
                plain[i].step(g, t, HP)
        for i, p in zip(idx, stepper.groups[gi].weights):
            assert np.array_equal(p.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1), (plain[i].hi_lo >> 16).astype(np.uint16))
    stepper.remove()
