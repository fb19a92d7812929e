"""The inside of a transformer block's training step over liblmopt.so: causal attention over packed sequences with
grouped heads, rotary positions, and activations kept in 8 bits between the forward and the backward pass,
alone and in the gated activation that reads them.  With ``head`` (norm, loss) and the optimizer groups they are a
memory-lean training step.

The ``*_forward`` / ``*_backward`` functions and ``pack_activation`` / ``unpack_activation`` are the library calls on
tensors; each takes ``stream`` (a torch stream the caller has ordered after its inputs; default: the
current one).  ``attention``, ``rotary``, ``swiglu``, ``gated_mlp`` are the same with autograd and run on
the current stream.  PyTorch supplies device memory, streams, the graph and plain matrix products.
All of them can be captured into a CUDA graph.  With autograd, capture the forward and the backward pass together, and let no
eager autograd graph of the same leaves live on at that time: its gradient accumulators belong to its own stream.
"""
from __future__ import annotations

import copy
import functools
import math
from fractions import Fraction

import torch
from torch.autograd.function import once_differentiable

from . import lmopt
from .head import _rows, _type, layer_norm


def _on_stream(stream, fn, *args):
    """A call's copies, allocations and kernels on a stream that is not the current one."""
    with torch.cuda.stream(stream):
        out = fn(*args)
    for a in args:                             # their memory is not given away before the stream is done with it
        for t in a.tensors() if isinstance(a, (PackedActivation, RotaryPlan)) else (a,):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
    return out


def _stream(device: int) -> int:
    return torch._C._cuda_getCurrentRawStream(device)


ACT_BLOCK = 32        # elements of a row that share an exponent (include/lmopt.h, act_pack_i8)


def _on_gpu(t: torch.Tensor, name: str) -> int:
    """The current GPU, where t has to be."""
    device = t.get_device()
    if device < 0 or device != torch._C._cuda_getDevice():
        raise ValueError(f"{name} must be on the current GPU")
    return device


# ----------------------------------------------------------------------------------------- attention
def _attn_side(t: torch.Tensor, name: str, device: int):
    """t [tokens, heads, dim], bf16, as the kernels read it: heads on 16 bytes, rows and heads apart; t itself, or a copy.  (t,
    its shape, its pointer and strides)"""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, not {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current GPU")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], not {list(t.shape)}")
    shape = t.shape
    rows, heads, dim = shape
    row, head, one = t.stride()
    at = t.data_ptr()
    if (at % 16 or rows > 1 and (row % 8 or row < dim) or heads > 1 and (head % 8 or head < dim) or dim > 1 and one != 1):
        t = t.clone(memory_format=torch.contiguous_format)
        at, row, head = t.data_ptr(), heads * dim, dim
    return t, shape, (at, row, head)


def _new_side(shape, like: torch.Tensor):
    """A new bf16 tensor of [tokens, heads, dim], and its pointer and strides."""
    t = torch.empty(shape, dtype=torch.bfloat16, device=like.device)
    return t, (t.data_ptr(), shape[1] * shape[2], shape[2])


_NO_SIDE = (None, 0, 0)


def _flat(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dim() != 4:
        raise ValueError(f"{name} must be [batch, length, heads, dim], not {list(t.shape)}")
    return t.reshape(-1, *t.shape[2:])


def _attn_args(q, k, v, cu_seqlens, scale):
    """(tensors that the call reads, shape of q, shape of k, sides of q, k, v, the call's sizes, the device) of [tokens, heads, dim] or, for
    sequences of one length, [batch, length, heads, dim]."""
    batch = 1
    if q.dim() == 4:
        if cu_seqlens is not None:
            raise ValueError("cu_seqlens are for [tokens, heads, dim]; [batch, length, heads, dim] are sequences of one length")
        if k.shape[:2] != q.shape[:2] or v.shape[:2] != q.shape[:2]:
            raise ValueError("q, k and v must have the same batch and length")
        batch = q.shape[0] or 1
        q, k, v = _flat(q, "q"), _flat(k, "k"), _flat(v, "v")
    if q.dtype is not torch.bfloat16:
        raise TypeError(f"q must be bfloat16, not {q.dtype}")
    device = _on_gpu(q, "q")
    q, q_shape, q_side = _attn_side(q, "q", device)
    k, k_shape, k_side = _attn_side(k, "k", device)
    v, v_shape, v_side = _attn_side(v, "v", device)
    rows, heads, dim = q_shape
    kv_heads = k_shape[1]
    if k_shape != v_shape or k_shape[0] != rows or k_shape[2] != dim:
        raise ValueError(f"q {list(q_shape)}, k {list(k_shape)} and v {list(v_shape)} do not fit")
    if heads < 1 or kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} query heads cannot share {kv_heads} key heads")
    if dim < 8 or dim > 128 or dim % 8:
        raise ValueError(f"heads must have 8 to 128 elements, a multiple of 8, not {dim}")
    borders = None
    if cu_seqlens is not None:
        if cu_seqlens.dtype is not torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.get_device() != device:
            raise ValueError(f"cu_seqlens must be int32 [sequences + 1] on {q.device}")
        if not cu_seqlens.is_contiguous():
            cu_seqlens = cu_seqlens.contiguous()
        borders, batch = cu_seqlens.data_ptr(), cu_seqlens.shape[0] - 1
    scale = dim ** -0.5 if scale is None else float(scale)
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale must be positive and finite")
    return (q, k, v, cu_seqlens), q_shape, k_shape, (q_side, k_side, v_side), (borders, batch, rows, heads, kv_heads, dim, scale), device


@functools.lru_cache(maxsize=256)
def _attn_bytes(packed: bool, sequences: int, rows: int, heads: int, kv_heads: int, dim: int) -> int:
    return lmopt.attn_workspace(256 if packed else None, sequences, rows, heads, kv_heads, dim)


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor | None = None,
                      scale: float | None = None, *, stream=None):
    """(out, lse): every query attends to the keys of its sequence up to its own, softmax(scale q k) v with scale
    dim^-1/2 by default.  q [tokens, heads, dim], k and v [tokens, kv_heads, dim] bf16 (dim a multiple of 8 up to 128, heads a multiple of
    kv_heads), sequence i rows cu_seqlens[i] to cu_seqlens[i + 1] - 1 (int32, on the device; None: one sequence), or all with
    a batch dimension before, sequences of one length.  lse, fp32 [heads, tokens], is the log of the softmax's
    denominator.  Rows of no sequence are 0 in both."""
    if stream is not None:
        return _on_stream(stream, attention_forward, q, k, v, cu_seqlens, scale)
    reads, shape, _, sides, args, device = _attn_args(q, k, v, cu_seqlens, scale)
    out, out_side = _new_side(shape, reads[0])
    lse = torch.empty((shape[1], shape[0]), dtype=torch.float32, device=out.device)
    lmopt.attn_forward(*sides, out_side, lse.data_ptr(), *args, _stream(device))
    return out.view(q.shape) if q.dim() == 4 else out, lse


def attention_backward(d_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
                       cu_seqlens: torch.Tensor | None = None, scale: float | None = None, need_q: bool = True, need_kv: bool = True, *,
                       stream=None):
    """(dq, dk, dv) from the gradient of out and what the forward call was given and returned; None for those that are not
    needed (dk and dv go together; dq's kernel runs for them too, they need what it sums).  Rows of no sequence get 0."""
    if stream is not None:
        return _on_stream(stream, attention_backward, d_out, q, k, v, out, lse, cu_seqlens, scale, need_q, need_kv)
    if d_out.shape != q.shape or out.shape != q.shape:
        raise ValueError(f"d_out and out must be {list(q.shape)}")
    batched = q.dim() == 4
    reads, q_shape, k_shape, sides, args, device = _attn_args(q, k, v, cu_seqlens, scale)
    d_out, _, do_side = _attn_side(_flat(d_out, "d_out") if batched else d_out, "d_out", device)
    out, _, out_side = _attn_side(_flat(out, "out") if batched else out, "out", device)
    if lse.dtype is not torch.float32 or lse.shape != (q_shape[1], q_shape[0]) or lse.get_device() != device:
        raise ValueError(f"lse must be float32 {[q_shape[1], q_shape[0]]} on {out.device}")
    if not lse.is_contiguous():
        lse = lse.contiguous()
    dq = dk = dv = None
    dq_side = dk_side = dv_side = _NO_SIDE
    if need_q:
        dq, dq_side = _new_side(q_shape, out)
    if need_kv:
        (dk, dk_side), (dv, dv_side) = _new_side(k_shape, out), _new_side(k_shape, out)
    borders, sequences, rows, heads, kv_heads, dim, _ = args
    nbytes = _attn_bytes(borders is not None, sequences, rows, heads, kv_heads, dim)
    work = torch.empty(nbytes, dtype=torch.uint8, device=out.device)
    lmopt.attn_backward(do_side, *sides, out_side, lse.data_ptr(), dq_side, dk_side, dv_side, *args, work.data_ptr(), nbytes,
                        _stream(device))
    if batched:
        dq, dk, dv = (None if t is None else t.view(s) for t, s in ((dq, q.shape), (dk, k.shape), (dv, v.shape)))
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale):
        out, lse = attention_forward(q, k, v, cu_seqlens, scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.scale = scale
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        need = ctx.needs_input_grad
        dq, dk, dv = attention_backward(d_out, q, k, v, out, lse, cu_seqlens, ctx.scale, need[0], need[1] or need[2])
        return dq, dk if need[1] else None, dv if need[2] else None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor | None = None, scale: float | None = None):
    """attention_forward's out with autograd (cu_seqlens must not change until the backward pass)."""
    return _Attention.apply(q, k, v, cu_seqlens, scale)


# ---------------------------------------------------------------------------------- rotary positions
_PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286208998, 10 ** 81)
_TURN_BITS = 256
_TURNS_PER_RADIAN = round(2 ** _TURN_BITS / (2 * _PI))


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None) -> tuple[list[float], float]:
    """Radians per position of each pair, base^(-2j/rotary_dim) scaled for `factor` times the length, and the factor on
    the rotated elements.
    scaling: None; "linear": positions divided by factor; "ntk": the base times factor^(d/(d-2)); "yarn": pairs
    that turn fewer than once in original_length are divided by factor, those that turn more than 32 times
    kept, in between in proportion, and the rotated elements times 0.1 ln(factor) + 1."""
    if rotary_dim < 0 or rotary_dim % 2:
        raise ValueError(f"rotary_dim must be even, not {rotary_dim}")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (base > 0 and math.isfinite(base)) or not (factor > 0 and math.isfinite(factor)):
        raise ValueError("base and factor must be positive")
    if scaling == "ntk" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    freq = [base ** (-2.0 * j / rotary_dim) for j in range(rotary_dim // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    if scaling == "yarn":
        if not original_length or original_length < 1:
            raise ValueError("yarn scaling needs original_length")
        keep = [min(max((original_length * f / (2 * math.pi) - 1.0) / 31.0, 0.0), 1.0) for f in freq]
        return [f * g + f / factor * (1.0 - g) for f, g in zip(freq, keep)], 1.0 + 0.1 * math.log(factor)
    return freq, 1.0


class RotaryPlan:
    """What rotary positions need of a model: the pairs' layout and their frequencies, on the device as turns per
    position in 64-bit fixed point.  Arguments as rotary_frequencies; interleaved: pairs are neighbours
    (2j, 2j + 1), not half the rotated part apart.  `rotary_dim` may be less than a head: the rest is kept."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str | None = None,
                 factor: float = 1.0, original_length: int | None = None, device="cuda"):
        freq, self.factor = rotary_frequencies(rotary_dim, base, scaling, factor, original_length)
        self.rotary_dim, self.interleaved = rotary_dim, interleaved
        turns = []
        for f in freq:
            num, den = f.as_integer_ratio()            # den is a power of two: the quotient is a shift
            shift = den.bit_length() - 1 + _TURN_BITS - 64
            turns.append((num * _TURNS_PER_RADIAN + (1 << shift - 1) >> shift) % 2 ** 64)
        self._turns = [t - (t >> 63 << 64) for t in turns]
        self.turns = torch.tensor(self._turns, dtype=torch.int64, device=device)

    def to(self, device) -> RotaryPlan:
        """The plan on a device: itself, or one like it."""
        if self.turns.device == torch.device(device):
            return self
        plan = copy.copy(self)
        plan.turns = torch.tensor(self._turns, dtype=torch.int64, device=device)
        return plan

    def tensors(self):
        return (self.turns,)


def _rope_side(t, name):
    """t [tokens, heads, dim] and a new tensor like it: (t or a copy, the new one, what a call takes of both)."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, dim], not {list(t.shape)}")
    shape = t.shape
    _, heads, dim = shape
    row, head, one = t.stride()
    if one != 1 and dim != 1:
        t = t.contiguous()
        row, head = heads * dim, dim
    o = torch.empty(shape, dtype=t.dtype, device=t.device)
    return t, o, (t.data_ptr(), row, head, o.data_ptr(), heads * dim, dim, heads)


def _rope(q, k, positions, plan, inverse, q_name, k_name):
    dtype = _type(q, q_name)
    device = _on_gpu(q, q_name)
    if k.get_device() != device:
        raise ValueError(f"{k_name} must be on the current GPU")
    q, q_out, q_side = _rope_side(q, q_name)
    k, k_out, k_side = _rope_side(k, k_name)
    rows, _, dim = q.shape
    if k.shape[0] != rows or k.shape[2] != dim or k.dtype is not q.dtype:
        raise ValueError(f"{q_name} and {k_name} must have the same tokens, head size and type")
    if plan.rotary_dim > dim:
        raise ValueError(f"{plan.rotary_dim} rotated elements in heads of {dim}")
    if positions.dtype is not torch.int64 or positions.shape != (rows,) or positions.get_device() != device:
        raise ValueError(f"positions must be int64 [{rows}] on {q.device}")
    if plan.turns.get_device() != device:
        raise ValueError("the plan is on another device")
    if not positions.is_contiguous():
        positions = positions.contiguous()
    lmopt.rope_apply(q_side, k_side, positions.data_ptr(), plan.turns.data_ptr(), rows, dim, plan.rotary_dim, plan.factor,
                     plan.interleaved, inverse, dtype, _stream(device))
    return q_out, k_out


def rotary_forward(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, plan: RotaryPlan, *, stream=None):
    """(q, k) turned by their tokens' positions.  q [tokens, heads, dim], k [tokens, kv_heads, dim] (bf16 or fp32, any strides;
    kv_heads may be 0), positions int64 [tokens], of any size.  New tensors."""
    if stream is not None:
        return _on_stream(stream, rotary_forward, q, k, positions, plan)
    return _rope(q, k, positions, plan, False, "q", "k")


def rotary_backward(dq: torch.Tensor, dk: torch.Tensor, positions: torch.Tensor, plan: RotaryPlan, *, stream=None):
    """Gradients of rotary_forward's inputs from those of its outputs."""
    if stream is not None:
        return _on_stream(stream, rotary_backward, dq, dk, positions, plan)
    return _rope(dq, dk, positions, plan, True, "dq", "dk")


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, plan):
        ctx.save_for_backward(positions)
        ctx.plan = plan
        return rotary_forward(q, k, positions, plan)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        return *rotary_backward(dq, dk, ctx.saved_tensors[0], ctx.plan), None, None


def rotary(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, plan: RotaryPlan):
    """rotary_forward with autograd."""
    return _Rotary.apply(q, k, positions, plan)


# ------------------------------------------------------------------------- activations kept in 8 bits
class PackedActivation:
    """An activation in 8 bits: int8 codes of rows of its last dimension, a uint8 exponent per 32 of them (the last block of a
    row is filled up with zeros), value = code * 2^(exponent - 133); the shape and type it was packed from.  Codes and
    exponents lie in one piece of memory, `data`; made from codes and exponents, it copies them there."""
    __slots__ = ("data", "rows", "width", "shape", "dtype")

    def __init__(self, codes: torch.Tensor, exponents: torch.Tensor, shape: torch.Size, dtype: torch.dtype):
        self._lay_out(shape, dtype)
        if (codes.dtype is not torch.int8 or codes.shape != (self.rows, self.width) or codes.device != exponents.device or
                exponents.dtype is not torch.uint8 or exponents.shape != (self.rows, self.width // ACT_BLOCK)):
            raise ValueError(f"codes and exponents do not fit {list(shape)}")
        self.data = torch.cat((codes.reshape(-1).view(torch.uint8), exponents.reshape(-1)))

    def _lay_out(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype
        self.rows, self.width = math.prod(shape[:-1]), -(-shape[-1] // ACT_BLOCK) * ACT_BLOCK

    @classmethod
    def _of(cls, data, shape, dtype):
        p = cls.__new__(cls)
        p._lay_out(shape, dtype)
        p.data = data
        return p

    @property
    def codes(self) -> torch.Tensor:
        return self.data[:self.rows * self.width].view(torch.int8).view(self.rows, self.width)

    @property
    def exponents(self) -> torch.Tensor:
        return self.data[self.rows * self.width:].view(self.rows, self.width // ACT_BLOCK)

    def tensors(self):
        return (self.data,)


def _new_packed(like: torch.Tensor, rows: int, cols: int, shape, dtype):
    """A PackedActivation of new memory, and what a call takes of it."""
    blocks = -(-cols // ACT_BLOCK)
    width = blocks * ACT_BLOCK
    p = PackedActivation.__new__(PackedActivation)
    p.data = torch.empty(rows * (width + blocks), dtype=torch.uint8, device=like.device)
    p.rows, p.width, p.shape, p.dtype = rows, width, shape, dtype
    at = p.data.data_ptr()
    return p, (at, width, at + rows * width, blocks)


def _packed_at(p: PackedActivation):
    """(what a call takes of a packed activation, its device)"""
    device = _on_gpu(p.data, "the packed activation")
    at, width = p.data.data_ptr(), p.width
    return (at, width, at + p.rows * width, width // ACT_BLOCK), device


def _matrix(t: torch.Tensor, name: str):
    """(t as a matrix of its last dimension's rows, its device)"""
    device = _on_gpu(t, name)
    return t if t.dim() == 2 and t.is_contiguous() else _rows(t, name), device


def pack_activation(x: torch.Tensor, *, stream=None) -> PackedActivation:
    """x (bf16 or fp32) in 8 bits: off by at most half a step of its block of 32 elements of the last dimension, which is 1/127.5
    (0.784 %) of the block's largest magnitude at most.  At the ends of the range a step has other limits: it is 2^-133 at least (blocks below 2^-126,
    of fp32), and in blocks from 127.5 2^121 on, where it cannot grow, their largest are off by less than a whole one.  A
    block with an infinity or a NaN comes back as NaN."""
    if stream is not None:
        return _on_stream(stream, pack_activation, x)
    dtype = _type(x, "x")
    m, device = _matrix(x, "x")
    rows, cols = m.shape
    if cols == 0:
        raise ValueError("x needs at least one element in a row")
    p, at = _new_packed(m, rows, cols, x.shape, x.dtype)
    lmopt.act_pack_i8(m.data_ptr(), m.stride(0), *at, rows, cols, dtype, _stream(device))
    return p


def unpack_activation(p: PackedActivation, *, stream=None) -> torch.Tensor:
    """The values that a packed activation stands for, in its shape and type."""
    if stream is not None:
        return _on_stream(stream, unpack_activation, p)
    at, device = _packed_at(p)
    shape = p.shape
    x = torch.empty(shape, dtype=p.dtype, device=p.data.device)
    lmopt.act_unpack_i8(*at, x.data_ptr(), shape[-1], p.rows, shape[-1], _type(x, "x"), _stream(device))
    return x


def swiglu_forward(gate_up: torch.Tensor, keep: bool = True, *, stream=None):
    """(h, packed): h = g sigmoid(g) u of gate_up [..., 2 n], g its first and u its last n elements, and both in 8
    bits ([..., 2, n]; None if keep is false) for swiglu_backward."""
    if stream is not None:
        return _on_stream(stream, swiglu_forward, gate_up, keep)
    dtype = _type(gate_up, "gate_up")
    m, device = _matrix(gate_up, "gate_up")
    rows, width = m.shape
    cols = width // 2
    if width != 2 * cols or cols == 0:
        raise ValueError(f"gate_up's last dimension must be even and not 0, not {width}")
    lead = gate_up.shape[:-1]
    h = torch.empty((*lead, cols), dtype=gate_up.dtype, device=m.device)
    packed, at = _new_packed(m, 2 * rows, cols, torch.Size((*lead, 2, cols)), gate_up.dtype) if keep else (None, (None, 0, None, 0))
    lmopt.act_swiglu_forward(m.data_ptr(), m.stride(0), h.data_ptr(), cols, *at, rows, cols, dtype, _stream(device))
    return h, packed


def swiglu_backward(dh: torch.Tensor, packed: PackedActivation, need_h: bool = False, *, stream=None):
    """(d_gate_up, h) from the gradient of h and what swiglu_forward kept: the gradients at the gate and up values that
    the codes stand for, and (need_h; else None) h of those values, for the next product's weight gradient."""
    if stream is not None:
        return _on_stream(stream, swiglu_backward, dh, packed, need_h)
    at, device = _packed_at(packed)
    if len(packed.shape) < 2 or packed.shape[-2] != 2:
        raise ValueError(f"a packed {list(packed.shape)} is not a gate and up pair")
    *lead, _, cols = packed.shape
    if dh.shape != (*lead, cols) or dh.dtype is not packed.dtype:
        raise ValueError(f"dh must be {packed.dtype} {[*lead, cols]} for a packed {list(packed.shape)}")
    d, _ = _matrix(dh, "dh")
    rows = d.shape[0]
    d_gate_up = torch.empty((*lead, 2 * cols), dtype=packed.dtype, device=d.device)
    h = torch.empty((*lead, cols), dtype=packed.dtype, device=d.device) if need_h else None
    lmopt.act_swiglu_backward(d.data_ptr(), d.stride(0), *at, d_gate_up.data_ptr(), 2 * cols, h.data_ptr() if need_h else None,
                              cols, rows, cols, _type(d, "dh"), _stream(device))
    return d_gate_up, h


class _SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate_up, keep):
        h, packed = swiglu_forward(gate_up, keep)
        if keep:
            ctx.save_for_backward(packed.data)
            ctx.kept = packed.shape, packed.dtype
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        return swiglu_backward(dh, PackedActivation._of(*ctx.saved_tensors, *ctx.kept))[0], None


def swiglu(gate_up: torch.Tensor) -> torch.Tensor:
    """g sigmoid(g) u with autograd; for the backward pass g and u are kept in 8 bits."""
    # always through the Function, which refuses forward-mode tangents: they come without requires_grad, and without grad mode too
    return _SwiGLU.apply(gate_up, torch.is_grad_enabled() and gate_up.requires_grad)


class _GatedMLP(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_in, w_out, keep):
        h, kept = swiglu_forward(torch.nn.functional.linear(x, w_in), keep)
        if keep:
            x8 = pack_activation(x) if ctx.needs_input_grad[1] else None
            ctx.save_for_backward(w_in, w_out, kept.data, x8.data if x8 else None)
            ctx.kept, ctx.x = (kept.shape, kept.dtype), (x.shape, x.dtype)
        return torch.nn.functional.linear(h, w_out)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        w_in, w_out, kept, x8 = ctx.saved_tensors
        need_x, need_in, need_out, _ = ctx.needs_input_grad
        d_gate_up, h = swiglu_backward(dy @ w_out, PackedActivation._of(kept, *ctx.kept), need_h=need_out)
        dx = d_in = d_out = None
        if need_out:
            d_out = dy.flatten(0, -2).t() @ h.flatten(0, -2)
            del h
        if need_in:
            d_in = d_gate_up.flatten(0, -2).t() @ unpack_activation(PackedActivation._of(x8, *ctx.x)).flatten(0, -2)
        if need_x:
            dx = d_gate_up @ w_in
        return dx, d_in, d_out, None


def gated_mlp(x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor) -> torch.Tensor:
    """swiglu(x w_in^T) w_out^T with autograd, w_in [2 n, dim], w_out [dim, n].  What is kept for the backward pass is x and
    the gate and up values in 8 bits (x for w_in's gradient; gate and up for everything else: h is formed again).  Under autocast
    (bf16) the three are cast first."""
    if x.dim() < 2 or w_in.dim() != 2 or w_out.dim() != 2 or w_in.shape[0] != 2 * w_out.shape[1] or x.shape[-1] != w_in.shape[1]:
        raise ValueError(f"x {list(x.shape)}, w_in {list(w_in.shape)} and w_out {list(w_out.shape)} do not fit")
    keep = torch.is_grad_enabled() and (x.requires_grad or w_in.requires_grad or w_out.requires_grad)
    if torch.is_autocast_enabled("cuda"):      # the casts are autograd's, outside of the Function, whose backward pass runs without autocast
        to = torch.get_autocast_dtype("cuda")
        x, w_in, w_out = (t.to(to) if t.dtype in (torch.float32, torch.bfloat16, torch.float16) else t for t in (x, w_in, w_out))
        with torch.autocast("cuda", enabled=False):
            return _GatedMLP.apply(x, w_in, w_out, keep)
    return _GatedMLP.apply(x, w_in, w_out, keep)


class TransformerBlock(torch.nn.Module):
    """x + attention(norm x), then x + mlp(norm x), over packed tokens [tokens, dim] in bf16: grouped heads with rotary
    positions, a gated MLP that keeps its activations in 8 bits.  Both output matrices start at zero, so that the block starts as the
    identity."""

    def __init__(self, dim: int, heads: int, kv_heads: int | None = None, hidden: int | None = None, rotary: RotaryPlan | None = None,
                 eps: float = 1e-5, device="cuda"):
        super().__init__()
        kv_heads = heads if kv_heads is None else kv_heads
        if heads < 1 or kv_heads < 1 or dim < 1 or dim % heads or dim // heads % 8 or dim // heads > 128 or heads % kv_heads:
            raise ValueError(f"width {dim} does not make {heads} heads of a multiple of 8, up to 128, that share {kv_heads}")
        hidden = 4 * dim if hidden is None else hidden
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.heads, self.kv_heads, self.head_dim, self.eps = heads, kv_heads, dim // heads, eps
        self.rotary = rotary or RotaryPlan(self.head_dim, device=device)
        new = lambda rows, cols: torch.nn.Parameter(torch.randn(rows, cols, **bf16) * cols ** -0.5)
        self.norm1, self.norm2 = torch.nn.Parameter(torch.ones(dim, **bf16)), torch.nn.Parameter(torch.ones(dim, **bf16))
        self.qkv = new((heads + 2 * kv_heads) * self.head_dim, dim)
        self.proj = torch.nn.Parameter(torch.zeros(dim, dim, **bf16))
        self.w_in = new(2 * hidden, dim)
        self.w_out = torch.nn.Parameter(torch.zeros(dim, hidden, **bf16))

    def _apply(self, fn, *args, **kw):
        super()._apply(fn, *args, **kw)
        self.rotary = self.rotary.to(fn(self.rotary.turns).device)      # where the parameters go
        return self

    def forward(self, x: torch.Tensor, positions: torch.Tensor, cu_seqlens: torch.Tensor | None = None) -> torch.Tensor:
        h, kv = self.heads, self.kv_heads
        qkv = torch.nn.functional.linear(layer_norm(x, self.norm1, None, self.eps), self.qkv).view(x.shape[0], h + 2 * kv, self.head_dim)
        q, k = rotary(qkv[:, :h], qkv[:, h:h + kv], positions, self.rotary)
        v = qkv[:, h + kv:]
        if v.requires_grad:
            v = v.contiguous()                 # kept for the backward pass: a view would keep q and k as they were, too
        y = attention(q, k, v, cu_seqlens)
        del qkv, q, k, v
        x = x + torch.nn.functional.linear(y.flatten(1), self.proj)
        return x + gated_mlp(layer_norm(x, self.norm2, None, self.eps), self.w_in, self.w_out)
