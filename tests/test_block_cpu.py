"""Argument checks of the attention, rotary and 8-bit activation calls: they come before any CUDA call, so they are
testable on a host without a GPU.  Pointers are made-up addresses that no accepted call is made with.  And what is
computed on the host: rotary frequencies and their fixed-point turns."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from test_head_cpu import lib, refused  # noqa: F401

P, U = 0x10000, 0x10001


def test_rope(lib):  # noqa: F811
    ok = dict(q=(P, 128, 64, P, 128, 64, 2), k=(P, 64, 64, P, 64, 64, 1), positions=P, turns=P, rows=4, dim=64, rotary=64, factor=1.0,
              interleaved=0, inverse=0, dtype=0)
    call = lambda **kw: (lib.rope_apply, kw.pop("code", lib.OPTIM_EINVAL), *{**ok, **kw}.values())
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=1025), dict(rotary=63), dict(rotary=66), dict(rotary=-2),
               dict(factor=float("nan")), dict(factor=float("inf")), dict(dtype=2), dict(positions=None), dict(turns=None),
               dict(q=(None, 128, 64, P, 128, 64, 2)), dict(q=(P, 128, 64, None, 128, 64, 2)), dict(k=(P, 64, 64, P, 64, 64, -1)),
               dict(q=(P, 128, 64, P, 128, 63, 2)), dict(q=(P, 128, 64, P, 64, 64, 2)), dict(q=(P, -128, 64, P, 128, 64, 2)),
               dict(q=(U, 128, 64, P, 128, 64, 2), code=lib.OPTIM_EALIGN), dict(k=(P, 64, 64, P + 2, 64, 64, 1), dtype=1, code=lib.OPTIM_EALIGN),
               dict(positions=P + 4, code=lib.OPTIM_EALIGN), dict(turns=P + 4, code=lib.OPTIM_EALIGN)):
        refused(lib, *call(**kw))


def test_pack_and_unpack(lib):  # noqa: F811
    ok = dict(x=P, ldx=70, codes=P, ldc=96, exponents=P, lde=3, rows=4, cols=70, dtype=0)
    for kw in (dict(rows=-1), dict(cols=0), dict(rows=1 << 31), dict(cols=1 << 30), dict(rows=(1 << 31) - 1, cols=1 << 12, ldc=1 << 12),
               dict(dtype=3), dict(x=None), dict(codes=None), dict(exponents=None), dict(ldx=69), dict(ldc=64), dict(ldc=97), dict(lde=2),
               dict(x=U, code=lib.OPTIM_EALIGN), dict(codes=P + 8, code=lib.OPTIM_EALIGN)):
        code = kw.pop("code", lib.OPTIM_EINVAL)
        a = {**ok, **kw}
        refused(lib, lib.act_pack_i8, code, *a.values())
        refused(lib, lib.act_unpack_i8, code, *(a[k] for k in ("codes", "ldc", "exponents", "lde", "x", "ldx", "rows", "cols", "dtype")))


def test_swiglu(lib):  # noqa: F811
    ok = dict(gate_up=P, ldg=140, h=P, ldh=70, codes=P, ldc=96, exponents=P, lde=3, rows=4, cols=70, dtype=0)
    for kw in (dict(rows=-1), dict(cols=0), dict(gate_up=None), dict(h=None), dict(ldg=139), dict(ldh=69), dict(codes=None),
               dict(exponents=None), dict(ldc=64), dict(lde=1), dict(gate_up=U, code=lib.OPTIM_EALIGN), dict(h=U, code=lib.OPTIM_EALIGN)):
        code = kw.pop("code", lib.OPTIM_EINVAL)
        refused(lib, lib.act_swiglu_forward, code, *{**ok, **kw}.values())
    ok = dict(dh=P, lddh=70, codes=P, ldc=96, exponents=P, lde=3, d=P, ldg=140, h=P, ldh=70, rows=4, cols=70, dtype=1)
    for kw in (dict(dh=None), dict(d=None), dict(lddh=1), dict(ldg=139), dict(ldh=2), dict(codes=None), dict(exponents=None),
               dict(dh=P + 2, code=lib.OPTIM_EALIGN), dict(h=P + 2, code=lib.OPTIM_EALIGN), dict(codes=P + 4, code=lib.OPTIM_EALIGN)):
        code = kw.pop("code", lib.OPTIM_EINVAL)
        refused(lib, lib.act_swiglu_backward, code, *{**ok, **kw}.values())


S, SK = (P, 256, 64), (P, 128, 64)
ATTN = dict(rows=10, heads=4, kv_heads=2, dim=64, scale=0.125)
BAD_SIZES = (dict(rows=-1), dict(rows=1 << 31), dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(heads=1 << 17, kv_heads=1),
             dict(dim=0), dict(dim=4), dict(dim=60), dict(dim=136), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
             dict(scale=float("nan")), dict(sequences=-1), dict(sequences=(1 << 30) + 1), dict(cu=None, sequences=3), dict(cu=None, sequences=0),
             dict(rows=(1 << 31) - 600, heads=1024))


def test_attention_forward(lib):  # noqa: F811
    ok = dict(q=S, k=SK, v=SK, out=S, lse=P, cu=P, sequences=2, **ATTN)
    call = lambda **kw: (lib.attn_forward, kw.pop("code", lib.OPTIM_EINVAL), *{**ok, **kw}.values())
    align = dict(code=lib.OPTIM_EALIGN)
    for kw in BAD_SIZES + (dict(q=(None, 256, 64)), dict(k=(None, 128, 64)), dict(v=(None, 128, 64)), dict(out=(None, 256, 64)), dict(lse=None),
                           dict(q=(P, 256, 56)), dict(q=(P, 0, 64)), dict(k=(P, 56, 64)), dict(out=(P, 64, 64)), dict(q=(P, 1 << 38, 64)),
                           dict(q=(P + 8, 256, 64), **align), dict(k=(P, 132, 64), **align), dict(v=(P, 128, 68), **align),
                           dict(out=(P + 2, 256, 64), **align), dict(lse=P + 2, **align), dict(cu=P + 2, **align)):
        refused(lib, *call(**kw))


def test_attention_backward(lib):  # noqa: F811
    ok = dict(do=S, q=S, k=SK, v=SK, out=S, lse=P, dq=S, dk=SK, dv=SK, cu=P, sequences=2, **ATTN, work=P, nbytes=1 << 30)
    call = lambda **kw: (lib.attn_backward, kw.pop("code", lib.OPTIM_EINVAL), *{**ok, **kw}.values())
    none, align = (None, 0, 0), dict(code=lib.OPTIM_EALIGN)
    for kw in BAD_SIZES + (dict(do=none), dict(q=none), dict(k=none), dict(v=none), dict(out=none), dict(lse=None), dict(dk=none), dict(dv=none),
                           dict(dq=(P, 64, 64)), dict(dk=(P, 64, 64)), dict(dv=(P, 128, 32)), dict(work=None), dict(nbytes=100),
                           dict(do=(P + 4, 256, 64), **align), dict(dq=(P, 260, 64), **align), dict(dk=(P + 2, 128, 64), **align),
                           dict(work=P + 128, **align)):
        refused(lib, *call(**kw))


def test_attention_workspace(lib):  # noqa: F811
    for bad in ((-1, 10, 4, 2, 64), (2, -1, 4, 2, 64), (2, 10, 4, 3, 64), (2, 10, 4, 2, 100)):
        with pytest.raises(lib.LmoptError):
            lib.attn_workspace(P, *bad)
    # 8 bytes a row and head, and a block's worth for each sequence
    n = lib.attn_workspace(P, 16, 8192, 32, 8, 128)
    assert 8 * 8192 * 32 <= n <= 8 * 32 * (8192 + 64 * 19)
    assert lib.attn_workspace(None, 16, 8192, 32, 8, 128) == n
    c = ctypes.c_size_t()
    assert lib.load().attn_workspace(None, 1, 64, 4, 4, 64, None) == lib.OPTIM_EINVAL
    assert lib.load().attn_workspace(None, 1, 64, 4, 4, 64, ctypes.byref(c)) == lib.OPTIM_OK


def test_rotary_frequencies():
    from memory_lean_optimizer_gb300 import block
    f, a = block.rotary_frequencies(8)
    assert a == 1.0 and f == [10000.0 ** (-j / 4) for j in range(4)]
    assert block.rotary_frequencies(8, scaling="linear", factor=4.0)[0] == [x / 4 for x in f]
    # the slowest pair of a scaled base turns `factor` times slower, the fastest as before
    g, _ = block.rotary_frequencies(64, scaling="ntk", factor=4.0)
    base = block.rotary_frequencies(64)[0]
    assert g[0] == 1.0 and math.isclose(g[-1], base[-1] / 4, rel_tol=1e-12)
    y, a = block.rotary_frequencies(64, scaling="yarn", factor=4.0, original_length=4096)
    assert math.isclose(a, 1 + 0.1 * math.log(4))
    for new, old in zip(y, base):
        turns = 4096 * old / (2 * math.pi)
        assert new == old if turns > 32 else math.isclose(new, old / 4) if turns < 1 else old / 4 <= new <= old
    for bad in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, base=-1.0), dict(rotary_dim=8, scaling="yarn", factor=2.0), dict(rotary_dim=8, base=float("inf"))):
        with pytest.raises(ValueError):
            block.rotary_frequencies(**bad)


def test_rotary_turns_are_the_frequencies():
    from memory_lean_optimizer_gb300 import block
    plan = block.RotaryPlan(64, device="cpu")
    for t, f in zip(plan.turns.tolist(), block.rotary_frequencies(64)[0]):
        turns = Fraction(t % 2 ** 64, 2 ** 64)
        assert abs(turns * 2 * block._PI - Fraction(f)) <= Fraction(8, 2 ** 64)
    # a frequency of a whole turn and more keeps its fraction
    fast = block.RotaryPlan(4, base=1e-3, device="cpu").turns.tolist()[1] % 2 ** 64
    f = Fraction(block.rotary_frequencies(4, base=1e-3)[0][1]) / (2 * block._PI)
    assert abs(Fraction(fast, 2 ** 64) - f % 1) <= Fraction(1, 2 ** 64)


def test_tensors_are_checked():
    """Refusals of the tensor calls that come before a GPU is needed."""
    from memory_lean_optimizer_gb300 import block
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        block.attention_forward(torch.zeros(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64))
    for call in (lambda: block.attention_forward(bf(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64)),
                 lambda: block.attention_forward(bf(1, 4, 2, 64), bf(1, 4, 1, 64), bf(1, 4, 1, 64), torch.zeros(2, dtype=torch.int32)),
                 lambda: block.attention_forward(bf(2, 4, 2, 64), bf(1, 4, 1, 64), bf(2, 4, 1, 64)),
                 lambda: block.attention_backward(bf(4, 2, 32), bf(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64), bf(4, 2, 64), torch.zeros(2, 4)),
                 lambda: block.rotary_forward(bf(4, 2, 64), bf(4, 1, 64), torch.arange(4), block.RotaryPlan(64, device="cpu")),
                 lambda: block.pack_activation(bf(4, 64)), lambda: block.swiglu_forward(bf(4, 64)),
                 lambda: block.gated_mlp(bf(4, 64), bf(96, 64), bf(64, 40)),
                 lambda: block.PackedActivation(torch.zeros(2, 32, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.uint8), (2, 32), torch.bfloat16),
                 lambda: block.PackedActivation(torch.zeros(2, 33, dtype=torch.int8), torch.zeros(2, 1, dtype=torch.uint8), (2, 32), torch.bfloat16),
                 lambda: block.TransformerBlock(100, 3, device="cpu"), lambda: block.TransformerBlock(128, 2, 3, device="cpu")):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        block.pack_activation(torch.zeros(4, 64, dtype=torch.float16))


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 0, None), (128, 2, 0), (0, 1, None), (128, -2, None), (128, 2, -1), (24, 6, 6), (512, 2, 2)])
def test_blocks_that_do_not_divide_are_refused(dim, heads, kv_heads):
    from memory_lean_optimizer_gb300 import block
    with pytest.raises(ValueError):
        block.TransformerBlock(dim, heads, kv_heads, device="cpu")
