"""The operators inside a transformer block's training step, each in a plain form and as the framework's own
calls: causal attention over packed sequences with grouped heads, forward and backward; rotary positions
of queries and keys, forward and backward; activation checkpoints in 8 bits, alone and in the gated
activation whose backward pass reads them.

``own`` chooses the side: False computes every operator with elementary torch operations in 32 bits
(angles in 64), True makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32            # elements of a row that share an exponent in the 8-bit checkpoints
_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------- cases
def _lengths(case):
    """Lengths of the packed sequences; they may leave rows of the buffers behind the last one."""
    if case["layout"] == "equal":
        return [case["length"]] * case["count"]
    rng = np.random.default_rng(case["layout_seed"])      # ragged: 2^U(0, log2 length), one of them empty
    n = [int(2.0 ** e) for e in rng.uniform(0.0, math.log2(case["length"]), case["count"])]
    if case["count"] > 2:
        n[case["count"] // 2] = 0
    return n


def listed():
    return [
        # a prompt of 37 tokens in a small model: latency counts
        dict(name="attn_fwd_prompt", op="attn", layout="equal", length=37, count=1, tail=0, heads=8, kv_heads=2, dim=64,
             grad=False),
        # the training batch of the small language model: 16 sequences of 512 tokens
        dict(name="attn_grad_batch", op="attn", layout="equal", length=512, count=16, tail=0, heads=4, kv_heads=2, dim=64,
             grad=True),
        # fine-tuning texts of 1 to 2048 tokens packed into one buffer with padding behind them; heads of 80
        dict(name="attn_grad_ragged", op="attn", layout="ragged", length=2048, count=40, layout_seed=5, tail=101, heads=12,
             kv_heads=3, dim=80, grad=True),
        # one long text, trained on
        dict(name="attn_grad_long", op="attn", layout="equal", length=16384, count=1, tail=0, heads=16, kv_heads=4, dim=128,
             grad=True),
        # a whole long prompt, read without a gradient
        dict(name="attn_fwd_long", op="attn", layout="equal", length=32768, count=1, tail=0, heads=16, kv_heads=4, dim=128,
             grad=False),
        # the next tokens of 16 texts, far into them: latency
        dict(name="rope_tokens", op="rope", rows=16, heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False,
             scaling="none", span=131072, x="bf16", pad=0, grad=False),
        # a training batch with positions scaled for four times the length, forward and backward
        dict(name="rope_grad_batch", op="rope", rows=16384, heads=32, kv_heads=8, dim=128, rotary=128, interleaved=False,
             scaling="yarn", span=16384, x="bf16", pad=0, grad=True),
        # fp32 heads of 80, half of each rotated in neighbouring pairs, rows cut from a wider projection
        dict(name="rope_grad_partial", op="rope", rows=5003, heads=12, kv_heads=3, dim=80, rotary=40, interleaved=True,
             scaling="linear", span=100000, x="f32", pad=80, grad=True),
        # the checkpoint of one short sequence's hidden states, written and read back
        dict(name="pack_small", op="pack", rows=64, cols=512, x="bf16"),
        # fp32 activations of an odd width
        dict(name="pack_odd_f32", op="pack", rows=5003, cols=2047, x="f32"),
        # the gated activation of a training batch, forward and backward
        dict(name="swiglu_grad_batch", op="swiglu", rows=16384, cols=8192, x="bf16"),
        # odd sizes: blocks that end with the row, rows that start off every vector
        dict(name="swiglu_grad_odd", op="swiglu", rows=1500, cols=1291, x="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "rope", "pack", "swiglu"])
    if op == "attn":
        kv = rng.choice([1, 2, 3, 4, 8])
        case = dict(op="attn", kv_heads=kv, heads=kv * rng.choice([1, 1, 2, 3, 4, 8]), dim=rng.choice([32, 64, 80, 96, 128, 128]),
                    tail=rng.choice([0, 0, 7, 300]), grad=rng.random() < 0.7)
        if rng.random() < 0.5:
            case.update(layout="equal", length=_log_int(rng, 1, 8192), count=_log_int(rng, 1, 16))
        else:
            case.update(layout="ragged", length=_log_int(rng, 2, 8192), count=_log_int(rng, 1, 64),
                        layout_seed=rng.randrange(1 << 20))
        while sum(n * n for n in _lengths(case)) * case["heads"] * case["dim"] > 1 << 38:
            case["count"] = (case["count"] + 1) // 2
            if case["count"] == 1:
                case["length"] = (case["length"] + 1) // 2
        return case
    if op == "rope":
        kv = rng.choice([1, 2, 3, 4, 8])
        dim = rng.choice([64, 80, 96, 128, 256])
        return _within(dict(op="rope", rows=_log_int(rng, 1, 16384), heads=kv * rng.choice([1, 2, 3, 4]), kv_heads=kv, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2, 2 * (dim // 5)]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "yarn"]), span=_log_int(rng, 16, 1 << 20),
                    x=rng.choice(["bf16", "bf16", "f32"]), pad=rng.choice([0, 0, 8, dim]), grad=rng.random() < 0.7))
    return _within(dict(op=op, rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 2, 8192) | rng.choice([0, 0, 1]),
                        x=rng.choice(["bf16", "bf16", "f32"])))


def _within(case):
    """The case with no more bytes than the largest listed one."""
    while work(case)["bytes"] > 2.4e9:
        case["rows"] = (case["rows"] + 1) // 2
    return case


def _tokens(case):
    return sum(_lengths(case)) + case["tail"]


def work(case):
    if case["op"] == "attn":
        t, h, kv, d = sum(_lengths(case)), case["heads"], case["kv_heads"], case["dim"]
        rows = _tokens(case)
        pairs = sum(n * (n + 1) // 2 for n in _lengths(case)) * h
        nbytes = 2 * d * t * (h + 2 * kv) + 2 * d * rows * h + 4 * rows * h
        flops = 4 * d * pairs
        if case["grad"]:          # d_out comes in, three gradients go out; five products beside the forward pass's two
            nbytes += 2 * d * t * h + 2 * d * rows * (h + 2 * kv)
            flops += 10 * d * pairs
        return {"bytes": nbytes, "flops": flops}
    e = 2 if case["x"] == "bf16" else 4
    if case["op"] == "rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"])
        passes = 2 if case["grad"] else 1
        return {"bytes": passes * (2 * e * n * case["dim"] + 8 * case["rows"]), "flops": passes * 3 * n * case["rotary"]}
    n = case["rows"] * case["cols"]
    blocks = case["rows"] * -(-case["cols"] // BLOCK)
    if case["op"] == "pack":      # in, codes out; codes in, out
        return {"bytes": 2 * (e * n + n + blocks), "flops": 6 * n}
    # gate and up in, h and both codes out; the h's gradient and both codes in, both gradients and h again out
    return {"bytes": 2 * e * n + e * n + 2 * (n + blocks) + e * n + 2 * (n + blocks) + 2 * e * n + e * n, "flops": 50 * n}


# ------------------------------------------------------------------------------------ inputs, states
def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1_000_003 + stream * 15_485_863 + 29) % (2 ** 62))
    return g


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _attn_inputs(case, seed):
    """q, k, v as views of one projection's output, the sequences' borders and the gradient of the output."""
    gen = _gen(seed, 1)
    t, h, kv, d = _tokens(case), case["heads"], case["kv_heads"], case["dim"]
    qkv = _randn(gen, t, h + 2 * kv, d)
    qkv[:, :h] *= 0.5 + 1.5 * torch.rand(h, 1, generator=gen, device="cuda")     # flat heads and sharp ones
    qkv = qkv.to(torch.bfloat16)
    q, k, v = qkv[:, :h], qkv[:, h:h + kv], qkv[:, h + kv:]
    cu = torch.tensor(np.concatenate(([0], np.cumsum(_lengths(case)))), dtype=torch.int32, device="cuda")
    d_out = (_randn(gen, t, h, d) * 1e-2).to(torch.bfloat16) if case["grad"] else None
    return q, k, v, cu, d_out


def _rope_inputs(case, seed):
    gen = _gen(seed, 2)
    n, h, kv, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
    wide = (h + kv) * d + case["pad"]

    def heads():
        x = _randn(gen, n, wide).to(_DTYPES[case["x"]])
        return x[:, :h * d].view(n, h, d), x[:, h * d:(h + kv) * d].view(n, kv, d)
    q, k = heads()
    positions = torch.randint(case["span"], (n,), generator=gen, device="cuda")
    dq, dk = heads() if case["grad"] else (None, None)
    return q, k, positions, dq, dk


FACTOR, ORIGINAL = 4.0, 4096      # lengths scaled by 4, from 4096 positions


def _rope_table(case):
    """Radians a position of each pair, and the factor on what is rotated."""
    r, base, s = case["rotary"], 10000.0, FACTOR
    if case["scaling"] == "ntk" and r > 2:
        base *= s ** (r / (r - 2))
    freq = [base ** (-2.0 * j / r) for j in range(r // 2)]
    if case["scaling"] == "linear":
        freq = [f / s for f in freq]
    if case["scaling"] == "yarn":
        keep = [min(max((ORIGINAL * f / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0) for f in freq]
        return [f * g + f / s * (1 - g) for f, g in zip(freq, keep)], 1.0 + 0.1 * math.log(s)
    return freq, 1.0


def _matrix_inputs(case, seed):
    """Hidden states (pack), or gate and up side by side with the gradient of the product (swiglu)."""
    gen = _gen(seed, 3)
    n, c, t = case["rows"], case["cols"], _DTYPES[case["x"]]
    if case["op"] == "pack":
        size = torch.rand(n, 1, generator=gen, device="cuda") * 3 + 0.05
        x = _randn(gen, n, c) * size
        x[:, :: 97] *= 20.0               # outlying channels
        return x.to(t), None
    gate_up = _randn(gen, n, 2 * c) * (torch.rand(n, 1, generator=gen, device="cuda") * 2 + 0.2)
    return gate_up.to(t), (_randn(gen, n, c) * 1e-2).to(t)


def prepare(case, seed):
    st = dict(case=case)
    if case["op"] == "attn":
        st["q"], st["k"], st["v"], st["cu"], st["d_out"] = _attn_inputs(case, seed)
        return st
    if case["op"] == "rope":
        st["q"], st["k"], st["positions"], st["dq"], st["dk"] = _rope_inputs(case, seed)
        if own:
            from memory_lean_optimizer_gb300 import block
            scaling = None if case["scaling"] == "none" else case["scaling"]
            st["plan"] = block.RotaryPlan(case["rotary"], interleaved=case["interleaved"], scaling=scaling, factor=FACTOR,
                                          original_length=ORIGINAL)
        else:
            freq, st["factor"] = _rope_table(case)
            st["freq"] = torch.tensor(freq, dtype=torch.float64, device="cuda")
        return st
    st["x"], st["dh"] = _matrix_inputs(case, seed)
    return st


# --------------------------------------------------------------------------------------- the passes
def _attn_plain(st):
    case = st["case"]
    h, kv, d = case["heads"], case["kv_heads"], case["dim"]
    g, scale = h // kv, d ** -0.5
    t = _tokens(case)
    out = dict(out=torch.zeros(t, h, d, dtype=torch.bfloat16, device="cuda"), lse=torch.zeros(h, t, device="cuda"))
    if case["grad"]:
        out.update(dq=torch.zeros(t, h, d, dtype=torch.bfloat16, device="cuda"),
                   dk=torch.zeros(t, kv, d, dtype=torch.bfloat16, device="cuda"),
                   dv=torch.zeros(t, kv, d, dtype=torch.bfloat16, device="cuda"))
    end = 0
    for n in _lengths(case):
        rows = slice(end, end + n)
        end += n
        if n == 0:
            continue
        later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
        for j in range(kv):               # one key head and the queries that share it: [g, n, d]
            q = st["q"][rows, j * g:(j + 1) * g].float().transpose(0, 1)
            k, v = st["k"][rows, j].float(), st["v"][rows, j].float()
            s = (q @ k.t()) * scale
            s = s.masked_fill(later, -math.inf)
            top = s.amax(2, keepdim=True)
            p = (s - top).exp()
            total = p.sum(2, keepdim=True)
            p = p / total
            o = p @ v
            out["out"][rows, j * g:(j + 1) * g] = o.transpose(0, 1).to(torch.bfloat16)
            out["lse"][j * g:(j + 1) * g, rows] = (top + total.log())[:, :, 0]
            if case["grad"]:
                do = st["d_out"][rows, j * g:(j + 1) * g].float().transpose(0, 1)
                dp = do @ v.t()
                ds = p * (dp - (do * o).sum(2, keepdim=True)) * scale
                out["dv"][rows, j] = (p.transpose(1, 2) @ do).sum(0).to(torch.bfloat16)
                out["dk"][rows, j] = (ds.transpose(1, 2) @ q).sum(0).to(torch.bfloat16)
                out["dq"][rows, j * g:(j + 1) * g] = (ds @ k).transpose(0, 1).to(torch.bfloat16)
    return out


def _attn_own(st):
    from memory_lean_optimizer_gb300 import block
    out, lse = block.attention_forward(st["q"], st["k"], st["v"], st["cu"])
    res = dict(out=out, lse=lse)
    if st["d_out"] is not None:
        res["dq"], res["dk"], res["dv"] = block.attention_backward(st["d_out"], st["q"], st["k"], st["v"], out, lse, st["cu"])
    return res


def _rotate_plain(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    f = x.float()
    if interleaved:
        a, b = f[..., 0:r:2], f[..., 1:r:2]
    else:
        a, b = f[..., :r // 2], f[..., r // 2:r]
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y, z), -1).flatten(-2) if interleaved else torch.cat((y, z), -1)
    return torch.cat((y, f[..., r:]), -1).to(x.dtype)


def _rope_plain(st):
    case = st["case"]
    angle = st["positions"].double()[:, None, None] * st["freq"]
    cos, sin = (angle.cos() * st["factor"]).float(), (angle.sin() * st["factor"]).float()
    out = dict(q=_rotate_plain(st["q"], cos, sin, case["interleaved"]), k=_rotate_plain(st["k"], cos, sin, case["interleaved"]))
    if case["grad"]:
        out["dq"] = _rotate_plain(st["dq"], cos, -sin, case["interleaved"])
        out["dk"] = _rotate_plain(st["dk"], cos, -sin, case["interleaved"])
    return out


def _rope_own(st):
    from memory_lean_optimizer_gb300 import block
    q, k = block.rotary_forward(st["q"], st["k"], st["positions"], st["plan"])
    out = dict(q=q, k=k)
    if st["case"]["grad"]:
        out["dq"], out["dk"] = block.rotary_backward(st["dq"], st["dk"], st["positions"], st["plan"])
    return out


def _pack_plain(x):
    """8-bit codes of a matrix, an exponent per 32 elements of a row: x = code 2^exponent."""
    n, c = x.shape
    blk = torch.nn.functional.pad(x.float(), (0, -c % BLOCK)).view(n, -1, BLOCK)
    top = blk.abs().amax(2)
    mant, exp = torch.frexp(top)                           # top = mant 2^exp, mant in [0.5, 1)
    exp = torch.where(mant >= 127.5 / 128.0, exp + 1, exp)
    exp = torch.where(top > 0, exp, torch.full_like(exp, -126)).clamp(min=-126) - 7
    code = torch.ldexp(blk, -exp[:, :, None]).round()
    return code.to(torch.int8), exp


def _unpack_plain(code, exp, cols):
    return torch.ldexp(code.float(), exp[:, :, None]).flatten(1)[:, :cols]


def _pack_roundtrip_plain(st):
    x = st["x"]
    return dict(x=_unpack_plain(*_pack_plain(x), x.shape[1]).to(x.dtype))


def _pack_own(st):
    from memory_lean_optimizer_gb300 import block
    return dict(x=block.unpack_activation(block.pack_activation(st["x"])))


def _swiglu_plain(st):
    x, dh = st["x"], st["dh"].float()
    c = dh.shape[1]
    gate, up = x[:, :c].float(), x[:, c:].float()
    h = gate / (1.0 + (-gate).exp()) * up
    gate_kept, up_kept = _pack_plain(x[:, :c]), _pack_plain(x[:, c:])
    # the backward pass starts from what was kept
    gate, up = _unpack_plain(*gate_kept, c), _unpack_plain(*up_kept, c)
    sig = 1.0 / (1.0 + (-gate).exp())
    act = gate * sig
    d_gate = dh * up * (sig + act * (1.0 - sig))
    return dict(h=h.to(x.dtype), d_gate_up=torch.cat((d_gate, dh * act), 1).to(x.dtype), h_again=(act * up).to(x.dtype))


def _swiglu_own(st):
    from memory_lean_optimizer_gb300 import block
    h, packed = block.swiglu_forward(st["x"])
    d_gate_up, h_again = block.swiglu_backward(st["dh"], packed, need_h=True)
    return dict(h=h, d_gate_up=d_gate_up, h_again=h_again)


def run(state):
    forms = dict(attn=(_attn_plain, _attn_own), rope=(_rope_plain, _rope_own), pack=(_pack_roundtrip_plain, _pack_own),
                 swiglu=(_swiglu_plain, _swiglu_own))
    return forms[state["case"]["op"]][1 if own else 0](state)


# ------------------------------------------------------------------------------------ in 64 bits
def _attn_exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    q, k, v, cu, d_out = _attn_inputs(case, seed)
    t, h, d = q.shape
    kv = k.shape[1]
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    res = dict(out=zeros(t, h, d), lse=zeros(h, t))
    if d_out is not None:
        res.update(dq=zeros(t, h, d), dk=zeros(t, kv, d), dv=zeros(t, kv, d))
    borders = cu.tolist()
    for a, b in zip(borders, borders[1:]):
        for head in range(h):
            j = head * kv // h
            K, V = k[a:b, j].double(), v[a:b, j].double()
            for lo in range(a, b, 2048):                     # rows lo..hi see the keys a..hi
                hi = min(lo + 2048, b)
                Q = q[lo:hi, head].double()
                s = torch.einsum("id,jd->ij", Q, K[:hi - a]) / math.sqrt(d)
                row = torch.arange(lo, hi, device="cuda")[:, None]
                s[torch.arange(a, hi, device="cuda")[None, :] > row] = -math.inf
                lse = torch.logsumexp(s, 1)
                p = torch.exp(s - lse[:, None])
                o = torch.einsum("ij,jd->id", p, V[:hi - a])
                res["out"][lo:hi, head], res["lse"][head, lo:hi] = o, lse
                if d_out is None:
                    continue
                dO = d_out[lo:hi, head].double()
                ds = torch.einsum("id,jd->ij", dO, V[:hi - a])
                ds = p * (ds - torch.einsum("id,id->i", dO, o)[:, None]) / math.sqrt(d)
                res["dv"][a:hi, j] += torch.einsum("ij,id->jd", p, dO)
                res["dk"][a:hi, j] += torch.einsum("ij,id->jd", ds, Q)
                res["dq"][lo:hi, head] = torch.einsum("ij,jd->id", ds, K[:hi - a])
    return res


def _turn64(x, positions, case, sign):
    """Each pair as a complex number, times exp(i sign angle)."""
    r, s = case["rotary"], FACTOR
    j = torch.arange(0, r, 2, dtype=torch.float64, device="cuda")
    base = 10000.0 * (s ** (r / (r - 2.0)) if case["scaling"] == "ntk" and r > 2 else 1.0)
    freq, size = torch.exp(-math.log(base) * j / r), 1.0
    if case["scaling"] == "linear":
        freq = freq / s
    elif case["scaling"] == "yarn":
        kept = ((ORIGINAL / (2 * math.pi) * freq - 1) / 31).clamp(0, 1)
        freq, size = torch.lerp(freq / s, freq, kept), 1 + math.log(s) / 10
    turn = torch.polar(torch.full((len(positions), 1, r // 2), size, dtype=torch.float64, device="cuda"),
                       sign * torch.einsum("n,j->nj", positions.double(), freq)[:, None])
    y = x.double().clone()
    first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _rope_exact(case, seed):
    q, k, positions, dq, dk = _rope_inputs(case, seed)
    res = dict(q=_turn64(q, positions, case, 1.0), k=_turn64(k, positions, case, 1.0))
    if dq is not None:
        res.update(dq=_turn64(dq, positions, case, -1.0), dk=_turn64(dk, positions, case, -1.0))
    return res


def _kept64(x):
    """What 8 bits keep of each block of a row: multiples of a power of two, the smallest power with which no
    value of the block rounds past 127 of them."""
    y = x.double()
    for part in y.split(BLOCK, dim=1):
        top = part.abs().max(1, keepdim=True).values
        step = torch.exp2((torch.log2(top.clamp(min=2.0 ** -126)).floor() - 7).clamp(min=-133))
        while bool((torch.round(top / step) > 127).any()):
            step = torch.where(torch.round(top / step) > 127, 2 * step, step)
        part.copy_(torch.round(part / step) * step)
    return y


def _swiglu_exact(case, seed):
    x, dh = _matrix_inputs(case, seed)
    c = case["cols"]
    h = torch.nn.functional.silu(x[:, :c].double()) * x[:, c:].double()
    gate, up = _kept64(x[:, :c]), _kept64(x[:, c:])
    sig = torch.sigmoid(gate)
    slope = sig * (1 + gate * torch.sigmoid(-gate))
    dh = dh.double()
    return dict(h=h, d_gate_up=torch.cat((dh * up * slope, dh * gate * sig), 1), h_again=gate * sig * up)


def exact(case, seed):
    if case["op"] == "pack":
        return dict(x=_kept64(_matrix_inputs(case, seed)[0]))
    return dict(attn=_attn_exact, rope=_rope_exact, swiglu=_swiglu_exact)[case["op"]](case, seed)
