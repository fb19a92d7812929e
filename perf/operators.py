"""The operators at the end of a language model's training step, each in a plain form and as the
framework's own calls: layer norm with its gradient, softmax cross entropy over a vocabulary straight
from the hidden states with its gradients, and the AdamW step over many tensors with states in 8 bits
or 32.

``own`` chooses the side: False computes every operator with elementary torch operations in 32 bits
(each rounded once, one operation at a time), True makes the framework's calls.
"""
import math

import numpy as np
import torch

own = False

U8_BLOCK = 256        # elements that share one scale in the 8-bit states
SMALL = 4096          # tensors of this many elements or fewer keep fp32 states
FLT_MAX = float(np.finfo(np.float32).max)
IGNORE = -100
LN_EPS = 1e-5


# ------------------------------------------------------------------------------------------- cases
def _block(c):
    """The matrices and vectors of one transformer block of width c (the diffusion workload's linears)."""
    return [(c, c)] * 6 + [(c, 2048)] * 2 + [(8 * c, c), (c, 4 * c)] + [(c,)] * 6


def _shapes(case):
    if case["layout"] == "square":
        return [(case["width"], case["width"])]
    if case["layout"] == "blocks":
        return [s for _ in range(case["count"]) for s in _block(case["width"])]
    rng = np.random.default_rng(case["layout_seed"])      # ragged: sizes 2^U(6, 22)
    return [(int(round(2.0 ** e)),) for e in rng.uniform(6.0, 22.0, case["count"])]


def listed():
    return [
        # one 1024 x 1024 weight: an optimizer group of one matrix, where the call's latency counts
        dict(name="adamw_u8_1m", op="adamw", states="u8", layout="square", width=1024, wd=0.01, step=7, zeros=0.0),
        # one optimizer group of a 2.6e9-parameter model cut into ten: large linears and their vectors
        dict(name="adamw_u8_blocks", op="adamw", states="u8", layout="blocks", width=1280, count=8, wd=0.01,
             step=1000, zeros=0.0),
        # tensors of every size from 64 to 4 M elements, unaligned tails, 1 % exact-zero gradients
        dict(name="adamw_u8_ragged", op="adamw", states="u8", layout="ragged", count=256, layout_seed=3, wd=0.0,
             step=2, zeros=0.01),
        # the same blocks with fp32 states, for models whose states fit
        dict(name="adamw_f32_blocks", op="adamw", states="fp32", layout="blocks", width=640, count=12, wd=0.1,
             step=100, zeros=0.0),
        # scoring a few tokens: the norm before the head on 16 rows
        dict(name="norm_fwd_tokens", op="norm", rows=16, dim=4096, pad=0, x="bf16", w="bf16", grad=False),
        # a training batch of 16384 tokens, forward and backward
        dict(name="norm_grad_batch", op="norm", rows=16384, dim=4096, pad=0, x="bf16", w="bf16", grad=True),
        # fp32 residual stream of an odd width, rows cut from a wider buffer, fp32 weights
        dict(name="norm_grad_odd_f32", op="norm", rows=5003, dim=2047, pad=14, x="f32", w="f32", grad=True),
        # a short sequence and a small vocabulary: latency
        dict(name="xent_grad_small", op="xent", rows=64, dim=512, vocab=2048, ignored=0.0, grad=True),
        # a training batch on a middle-sized vocabulary
        dict(name="xent_grad_batch", op="xent", rows=4096, dim=2048, vocab=32768, ignored=0.0, grad=True),
        # odd sizes; a third of the tokens (the prompts) carry no loss
        dict(name="xent_grad_odd", op="xent", rows=1500, dim=1290, vocab=50021, ignored=0.35, grad=True),
        # a long batch on a large vocabulary: the largest
        dict(name="xent_grad_large", op="xent", rows=8192, dim=4096, vocab=131072, ignored=0.0, grad=True),
        # scoring the next token of 16 sequences: no gradient, the weight is read once
        dict(name="xent_fwd_tokens", op="xent", rows=16, dim=4096, vocab=131072, ignored=0.0, grad=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "norm", "xent"])
    if op == "adamw":
        case = dict(op="adamw", states=rng.choice(["u8", "u8", "fp32"]), wd=rng.choice([0.0, 0.01, 0.1]),
                    step=_log_int(rng, 1, 20000), zeros=rng.choice([0.0, 0.01]))
        layout = rng.choice(["square", "blocks", "ragged"])
        if layout == "square":
            return dict(case, layout=layout, width=_log_int(rng, 65, 8192))
        if layout == "blocks":
            return dict(case, layout=layout, width=rng.choice([320, 640, 1280]), count=rng.randint(1, 8))
        return dict(case, layout=layout, count=_log_int(rng, 2, 256), layout_seed=rng.randrange(1 << 20))
    if op == "norm":
        x = rng.choice(["bf16", "bf16", "f32"])
        return dict(op="norm", rows=_log_int(rng, 1, 16384), dim=_log_int(rng, 33, 8192) | rng.choice([0, 0, 1]),
                    pad=rng.choice([0, 0, 8, 14]), x=x, w=rng.choice(["bf16", x]), grad=rng.random() < 0.7)
    dim = _log_int(rng, 64, 4096)
    if rng.random() < 0.7:
        dim = (dim + 7) // 8 * 8
    return dict(op="xent", rows=_log_int(rng, 1, 8192), dim=dim, vocab=_log_int(rng, 1000, 131072),
                ignored=rng.choice([0.0, 0.0, 0.35, 0.9]), grad=rng.random() < 0.7)


def _n_ignored(case):
    return min(case["rows"] - 1, int(round(case["ignored"] * case["rows"])))


def work(case):
    if case["op"] == "adamw":
        n_small = n_large = blocks = 0
        for s in _shapes(case):
            n = math.prod(s)
            if case["states"] == "u8" and n > SMALL:
                n_large += n
                blocks += -(-n // U8_BLOCK)
            else:
                n_small += n
        # weight, residual and gradient; states read and written; 8-bit states also given out as fp32
        nbytes = 10 * (n_small + n_large) + 16 * n_small + (4 + 8) * n_large + 16 * blocks
        return {"bytes": nbytes, "flops": 16 * (n_small + n_large)}
    if case["op"] == "norm":
        e, we = (2 if case["x"] == "bf16" else 4), (2 if case["w"] == "bf16" else 4)
        n = case["rows"] * case["dim"]
        nbytes = 2 * e * n + 2 * we * case["dim"] + 8 * case["rows"]
        if case["grad"]:       # the gradient comes in, goes out; the weight's and bias's gradients go out
            nbytes += 2 * e * n + 2 * we * case["dim"]
        return {"bytes": nbytes, "flops": (20 if case["grad"] else 7) * n}
    used = case["rows"] - _n_ignored(case)
    n, v, d = case["rows"], case["vocab"], case["dim"]
    nbytes = 2 * used * d + 2 * v * d + 16 * n
    if case["grad"]:
        nbytes += 4 * n + 2 * n * d + 2 * v * d
    return {"bytes": nbytes, "flops": (6 if case["grad"] else 2) * used * v * d}


# ------------------------------------------------------------------------------------ inputs, states
def _gen(seed, stream):
    g = torch.Generator(device="cuda")
    g.manual_seed((seed * 1_000_003 + stream * 15_485_863 + 17) % (2 ** 62))
    return g


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _adamw_inputs(case, seed):
    gen = _gen(seed, 1)
    tensors = []
    for s in _shapes(case):
        n = math.prod(s)
        master = _randn(gen, n).mul_(0.02)
        grad = _randn(gen, n).mul_(1e-3)
        if case["zeros"]:
            grad.masked_fill_(torch.rand(n, generator=gen, device="cuda") < case["zeros"], 0.0)
        std = torch.rand(n, generator=gen, device="cuda").mul_(2e-3).add_(1e-5)    # the gradients' size so far
        m = _randn(gen, n).mul_(0.3).mul_(std)
        if case["step"] == 1:
            m.zero_()
            std.zero_()
        tensors.append(dict(shape=s, master=master, grad=grad.to(torch.bfloat16), m=m, v=std.mul_(std)))
    return tensors


def _adamw_scalars(case, t):
    """The step's scalars, computed in 64 bits from the fp32 hyper-parameters, each rounded once."""
    lr, b1, b2, eps, wd = (float(np.float32(x)) for x in (3e-4, 0.9, 0.999, 1e-8, case["wd"]))
    f = lambda x: float(np.float32(x))
    return dict(b1=b1, omb1=f(1.0 - b1), b2=b2, omb2=f(1.0 - b2), eps=eps, lr_wd=f(lr * wd),
                k2=f(1.0 / math.sqrt(1.0 - b2 ** t)), k1=f(lr / (1.0 - b1 ** t)))


def _split(x):
    """fp32 master -> (bf16 upper half, int16 lower half)."""
    h = x.view(torch.int16).view(-1, 2)
    return h[:, 1].contiguous().view(torch.bfloat16), h[:, 0].contiguous()


def _merge(hi, lo):
    return torch.stack((lo, hi.view(torch.int16)), 1).view(-1).view(torch.float32)


def _quantise(x, signed):
    """8-bit codes and block scales of a moment (signed: the first moment)."""
    n = x.numel()
    blk = torch.nn.functional.pad(x, (0, -n % U8_BLOCK)).view(-1, U8_BLOCK)
    if signed:
        q = blk.abs().amax(1).sqrt() * float(np.float32(1.0) / np.float32(127.0))
    else:
        q = blk.amax(1).sqrt().sqrt() * float(np.float32(1.0) / np.float32(255.0))
    r = torch.where(q > 0, (torch.ones_like(q) / (q * q)).clamp(max=FLT_MAX), torch.zeros_like(q))
    if signed:
        y = (blk.abs() * r[:, None]).sqrt().clamp(max=127.0).round()
        code = 128 + torch.where(blk < 0, -y, y)
    else:
        y = (blk.sqrt() * r[:, None]).sqrt().clamp(max=255.0).round()
        code = torch.where(blk > 0, y.clamp(min=1.0), torch.zeros_like(y))
    return code.to(torch.uint8).view(-1)[:n].contiguous(), q


def _offsets(case):
    """Where each tensor starts in the flat buffers (a multiple of 64 elements), and their length."""
    starts, end = [], 0
    for s in _shapes(case):
        starts.append(end)
        end += (math.prod(s) + 63) // 64 * 64
    return starts, end


def _dequantise(code, q, signed):
    n = code.numel()
    c = torch.nn.functional.pad(code, (0, -n % U8_BLOCK)).view(-1, U8_BLOCK).to(torch.float32)
    if signed:
        t = (c - 128.0) * q[:, None]
        x = t * t.abs()
    else:
        z = c * q[:, None]
        z = z * z
        x = z * z
    return x.view(-1)[:n].contiguous()


def _xent_inputs(case, seed):
    n, v, d = case["rows"], case["vocab"], case["dim"]
    gen = _gen(seed, 2)
    weight = (_randn(gen, v, d).mul_(0.02)).to(torch.bfloat16)
    target = torch.randint(v, (n,), generator=gen, device="cuda")
    hidden = _randn(gen, n, d)
    gain = torch.rand(n, 1, generator=gen, device="cuda") * (250.0 / d)        # from a guess to near certain
    hidden += 150.0 * gain * weight[target].float()
    order = torch.randperm(n, generator=gen, device="cuda")
    k = _n_ignored(case)
    target[order[:k]] = IGNORE
    scale = torch.full((n,), 1.0 / max(n - k, 1), device="cuda")
    return hidden.to(torch.bfloat16), weight, target, scale


def _norm_inputs(case, seed):
    n, d = case["rows"], case["dim"]
    gen = _gen(seed, 3)
    xt = torch.bfloat16 if case["x"] == "bf16" else torch.float32
    wt = torch.bfloat16 if case["w"] == "bf16" else torch.float32
    wide = d + case["pad"]
    x = _randn(gen, n, wide)
    x = (x * (torch.rand(n, 1, generator=gen, device="cuda") * 3 + 0.1) + _randn(gen, n, 1)).to(xt)[:, :d]
    dy = (_randn(gen, n, wide) * 1e-2).to(xt)[:, :d] if case["grad"] else None
    weight = (1.0 + 0.1 * _randn(gen, d)).to(wt)
    bias = (0.1 * _randn(gen, d)).to(wt)
    return x, weight, bias, dy


def prepare(case, seed):
    st = dict(case=case)
    if case["op"] == "xent":
        st["hidden"], st["weight"], st["target"], st["scale"] = _xent_inputs(case, seed)
        return st
    if case["op"] == "norm":
        st["x"], st["w"], st["b"], st["dy"] = _norm_inputs(case, seed)
        return st
    tensors = _adamw_inputs(case, seed)
    st["gscale"] = torch.full((1,), 0.5 + (seed % 7) / 8, device="cuda")       # a clip factor
    st["grads"] = [t["grad"].view(t["shape"]) for t in tensors]
    st["step"] = case["step"]
    # one flat buffer of each kind, as training programs keep them; the tensors are views of it
    starts, end = _offsets(case)
    flat = dict(w=torch.zeros(end, dtype=torch.bfloat16, device="cuda"),
                res=torch.zeros(end, dtype=torch.int16, device="cuda"))
    if not own or case["states"] == "u8":      # fp32 states as the group itself keeps them
        flat.update(m=torch.zeros(end, device="cuda"), v=torch.zeros(end, device="cuda"))
    views = {k: [x[o:o + t["master"].numel()] for o, t in zip(starts, tensors)] for k, x in flat.items()}
    for i, t in enumerate(tensors):
        hi, lo = _split(t["master"])
        views["w"][i].copy_(hi)
        views["res"][i].copy_(lo)
    st["flat"], st["views"] = flat, views
    packed = [case["states"] == "u8" and t["master"].numel() > SMALL for t in tensors]
    if not own:
        for name, signed in (("m", True), ("v", False)):
            st[name] = [_quantise(t[name], signed) if p else t[name] for t, p in zip(tensors, packed)]
        return st
    from memory_lean_optimizer_gb300 import engine
    group = engine.AdamWGroup([w.view(t["shape"]) for w, t in zip(views["w"], tensors)], views["res"],
                              states=case["states"])
    for i, t in enumerate(tensors):
        for buf, x, signed in ((group.m[i], t["m"], True), (group.v[i], t["v"], False)):
            if packed[i]:
                code, q = _quantise(x, signed)
                codes, scales = engine.u8_state_views(buf, x.numel())
                codes.copy_(code)
                scales.copy_(q)
            else:
                buf.copy_(x)
    group.set_step(case["step"] - 1)
    if case["states"] == "fp32":
        flat.update(m=group.flat_m, v=group.flat_v)
    st["group"] = group
    st["hp"] = dict(lr=3e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=case["wd"])
    return st


# --------------------------------------------------------------------------------------- the passes
def _adamw_plain(st):
    k = _adamw_scalars(st["case"], st["step"])
    views = st["views"]
    for i, grad in enumerate(st["grads"]):
        ms, vs = st["m"][i], st["v"][i]
        packed = isinstance(ms, tuple)
        g = grad.reshape(-1).to(torch.float32) * st["gscale"]
        m = (_dequantise(*ms, True) if packed else ms) * k["b1"]
        m = m + g * k["omb1"]
        v = (_dequantise(*vs, False) if packed else vs) * k["b2"]
        v = v + (g * g) * k["omb2"]
        w = _merge(views["w"][i], views["res"][i])
        w = w - w * k["lr_wd"]
        den = v.sqrt() * k["k2"]
        den = den + k["eps"]
        w = w - (m * k["k1"]) / den
        if packed:
            st["m"][i], st["v"][i] = mq, vq = _quantise(m, True), _quantise(v, False)
            m, v = _dequantise(*mq, True), _dequantise(*vq, False)
        else:
            st["m"][i], st["v"][i] = m, v
        for name, x in zip(("w", "res", "m", "v"), (*_split(w), m, v)):
            views[name][i].copy_(x)
    st["step"] += 1
    return dict(st["flat"])


def _adamw_own(st):
    group = st["group"]
    group.step(st["grads"], st["hp"], grad_scale=st["gscale"])
    if st["case"]["states"] == "u8":
        group.unpack_states(st["flat"]["m"], st["flat"]["v"])
    return dict(st["flat"])


def _norm_plain(st):
    x, w, b = st["x"].float(), st["w"].float(), st["b"].float()
    xt, wt = st["x"].dtype, st["w"].dtype
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((xc * xc).mean(1) + LN_EPS)
    xh = xc * rstd[:, None]
    out = dict(y=(xh * w + b).to(xt), mean=mean, rstd=rstd)
    if st["dy"] is not None:
        dy = st["dy"].float()
        a = dy * w
        dx = (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True)) * rstd[:, None]
        out.update(dx=dx.to(xt), dw=(dy * xh).sum(0).to(wt), db=dy.sum(0).to(wt))
    return out


def _norm_own(st):
    from memory_lean_optimizer_gb300 import head
    y, mean, rstd = head.layer_norm_forward(st["x"], st["w"], st["b"], LN_EPS)
    out = dict(y=y, mean=mean, rstd=rstd)
    if st["dy"] is not None:
        out["dx"], out["dw"], out["db"] = head.layer_norm_backward(st["dy"], st["x"], st["w"], mean, rstd)
    return out


def _xent_plain(st):
    hidden, weight, target = st["hidden"].float(), st["weight"].float(), st["target"]
    valid = target >= 0
    t = target.clamp(min=0)[:, None]
    logits = hidden @ weight.t()
    top = logits.amax(1, keepdim=True)
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    zero = torch.zeros_like(lse)
    out = dict(loss=torch.where(valid, lse - logits.gather(1, t)[:, 0], zero), lse=torch.where(valid, lse, zero))
    if st["case"]["grad"]:
        e = (logits - lse[:, None]).exp()
        e.scatter_add_(1, t, torch.full_like(t, -1, dtype=e.dtype))
        e *= torch.where(valid, st["scale"], zero)[:, None]
        out.update(dh=(e @ weight).to(torch.bfloat16), dw=(e.t() @ hidden).to(torch.bfloat16))
    return out


def _xent_own(st):
    from memory_lean_optimizer_gb300 import head
    loss, lse = head.xent_forward(st["hidden"], st["weight"], st["target"], ignore_index=IGNORE)
    out = dict(loss=loss, lse=lse)
    if st["case"]["grad"]:
        out["dh"], out["dw"] = head.xent_backward(st["hidden"], st["weight"], st["target"], lse, st["scale"],
                                                  ignore_index=IGNORE)
    return out


def run(state):
    forms = dict(adamw=(_adamw_plain, _adamw_own), norm=(_norm_plain, _norm_own), xent=(_xent_plain, _xent_own))
    return forms[state["case"]["op"]][1 if own else 0](state)


# ------------------------------------------------------------------------------------ in 64 bits
def _code64(x, signed):
    """Values that the 8-bit storage keeps for a 64-bit moment: the nearest code on the companded scale
    of the block's largest magnitude."""
    n = x.numel()
    blk = torch.zeros(-(-n // U8_BLOCK) * U8_BLOCK, dtype=torch.float64, device=x.device)
    blk[:n] = x
    blk = blk.view(-1, U8_BLOCK)
    top = blk.abs().max(1).values[:, None]
    safe = torch.where(top > 0, top, torch.ones_like(top))
    if signed:
        c = torch.round(127.0 * (blk.abs() / safe) ** 0.5)
        val = torch.sign(blk) * (c / 127.0) ** 2 * top
    else:
        c = torch.round(255.0 * (blk / safe) ** 0.25)
        c = torch.where((blk > 0) & (c < 1), torch.ones_like(c), c)
        val = (c / 255.0) ** 4 * top
    return val.view(-1)[:n]


def _adamw_exact(case, seed):
    gs = 0.5 + (seed % 7) / 8
    t = case["step"]
    lr, b1, b2, eps, wd = (float(np.float32(x)) for x in (3e-4, 0.9, 0.999, 1e-8, case["wd"]))
    starts, end = _offsets(case)
    out = {name: torch.zeros(end, dtype=torch.float64, device="cuda") for name in ("w", "m", "v")}
    for start, x in zip(starts, _adamw_inputs(case, seed)):
        packed = case["states"] == "u8" and x["master"].numel() > SMALL
        m, v = x["m"], x["v"]
        if packed:                                   # the pass starts from the stored codes
            m, v = _dequantise(*_quantise(m, True), True), _dequantise(*_quantise(v, False), False)
        g = x["grad"].double() * gs
        m = b1 * m.double() + (1 - b1) * g
        v = b2 * v.double() + (1 - b2) * g ** 2
        w = x["master"].double()
        w = w * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
        bits = w.float().view(torch.int32) & -65536  # the weight is the upper half of the fp32 value
        part = slice(start, start + w.numel())
        out["w"][part] = bits.view(torch.float32).double()
        out["m"][part] = _code64(m, True) if packed else m
        out["v"][part] = _code64(v, False) if packed else v
    return dict(w=out["w"], res=None, m=out["m"], v=out["v"])


def _norm_exact(case, seed):
    x, w, b, dy = (None if t is None else t.double() for t in _norm_inputs(case, seed))
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    rstd = (var + LN_EPS) ** -0.5
    xh = (x - mean) * rstd
    out = dict(y=torch.addcmul(b, xh, w), mean=mean[:, 0], rstd=rstd[:, 0])
    if dy is not None:
        d = case["dim"]
        g = dy * w
        out["dx"] = rstd / d * (d * g - g.sum(1, keepdim=True) - xh * torch.einsum("nd,nd->n", g, xh)[:, None])
        out["dw"] = torch.einsum("nd,nd->d", dy, xh)
        out["db"] = torch.einsum("nd->d", dy)
    return out


def _xent_exact(case, seed):
    n, v, d = case["rows"], case["vocab"], case["dim"]
    if 2 * n * v * d > 1e13:
        return None
    grad = case["grad"] and 6 * n * v * d <= 1e13      # the large gradients would take too long in 64 bits
    hidden, weight, target, scale = _xent_inputs(case, seed)
    weight = weight.double()
    out = dict(loss=torch.zeros(n, dtype=torch.float64, device="cuda"),
               lse=torch.zeros(n, dtype=torch.float64, device="cuda"))
    if case["grad"]:
        out.update(dh=None, dw=None)
    if grad:
        out["dh"] = torch.zeros(n, d, dtype=torch.float64, device="cuda")
        out["dw"] = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    rows = torch.nonzero(target != IGNORE)[:, 0]
    for part in rows.split(1024):
        h, t = hidden[part].double(), target[part]
        logits = torch.einsum("nd,vd->nv", h, weight)
        lse = torch.logsumexp(logits, 1)
        out["lse"][part] = lse
        out["loss"][part] = lse - logits[torch.arange(len(part), device="cuda"), t]
        if grad:
            e = torch.exp(logits - lse[:, None])
            e[torch.arange(len(part), device="cuda"), t] -= 1.0
            e *= scale[part].double()[:, None]
            out["dh"][part] = torch.einsum("nv,vd->nd", e, weight)
            out["dw"] += torch.einsum("nv,nd->vd", e, h)
    return out


def exact(case, seed):
    return dict(adamw=_adamw_exact, norm=_norm_exact, xent=_xent_exact)[case["op"]](case, seed)
