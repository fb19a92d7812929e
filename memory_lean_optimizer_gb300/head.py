"""The last layers of a language model's training step over liblmopt.so: layer norm and the softmax
cross entropy over the vocabulary, taken straight from the hidden states so that the logits are
never kept.  With ``engine.AdamWGroup`` (or ``hooks.attach_fused_adamw``) they are the memory-lean
tail of a training step: hidden states -> norm -> loss -> gradients -> optimizer.

The ``*_forward`` / ``*_backward`` functions are the library calls on tensors; each takes ``stream`` (a torch
stream the caller has ordered after its inputs; default: the current one).  ``layer_norm``,
``linear_cross_entropy`` and ``LMTail`` are the same with autograd and run on the current stream.  PyTorch supplies
device memory, streams and the graph.
"""
from __future__ import annotations

import functools

import torch
from torch.autograd.function import once_differentiable

from . import lmopt
from .engine import _stream_ptr

_TYPES = {torch.bfloat16: lmopt.OPTIM_BF16, torch.float32: lmopt.OPTIM_F32}


def _type(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _TYPES:
        raise TypeError(f"{name} must be bfloat16 or float32, not {t.dtype}")
    return _TYPES[t.dtype]


def _on_stream(fn):
    """Runs a call's copies, allocations and kernels on its `stream` argument (None: the current stream)."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        for t in (*args, *kw.values()):        # their memory is not given away before the stream is done with it
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        return out
    return call


def _rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """t as a matrix of its last dimension's rows, whose elements lie next to each other: a view where the
    strides allow one (rows may be apart), else a copy."""
    if not t.is_cuda or t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} must be on the current GPU")
    if t.dim() != 2:
        if t.dim() < 1:
            raise ValueError(f"{name} needs at least one dimension")
        t = t.reshape(-1, t.shape[-1])
    # a broadcast row (stride 0) is laid out too: the calls want rows at least their length apart
    rows, dim = t.shape
    ld, step = t.stride()
    if dim > 1 and step != 1 or rows > 1 and ld < dim:
        t = t.contiguous()
    return t


def _vector(t: torch.Tensor, n: int, like: torch.Tensor, dtype, name: str) -> torch.Tensor:
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be {n} values of {dtype} on {like.device}")
    return t if t.is_contiguous() else t.contiguous()


@functools.lru_cache(maxsize=256)
def _norm_bytes(rows: int, dim: int) -> int:
    return lmopt.norm_layer_workspace(rows, dim)


@_on_stream
def layer_norm_forward(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5):
    """(y, mean, rstd) of the layer norm over x's last dimension; mean and rstd are fp32, one per row."""
    xt, wt = _type(x, "x"), _type(weight, "weight")
    m = _rows(x, "x")
    rows, dim = m.shape
    weight = _vector(weight, dim, x, weight.dtype, "weight")
    if bias is not None:
        bias = _vector(bias, dim, x, weight.dtype, "bias")
    y = x.new_empty(x.shape)
    mean, rstd = x.new_empty(rows, dtype=torch.float32), x.new_empty(rows, dtype=torch.float32)
    lmopt.norm_layer_forward(m.data_ptr(), m.stride(0), weight.data_ptr(), None if bias is None else bias.data_ptr(),
                             y.data_ptr(), dim, mean.data_ptr(), rstd.data_ptr(), rows, dim, eps, xt, wt,
                             _stream_ptr(None))
    return y, mean, rstd


@_on_stream
def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, mean: torch.Tensor,
                        rstd: torch.Tensor, need_x: bool = True, need_weight: bool = True):
    """(dx, dweight, dbias) from the gradient of y and what the forward call returned; None for those that are not
    needed (dweight and dbias go together)."""
    xt, wt = _type(x, "x"), _type(weight, "weight")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must have x's shape and type")
    m, g = _rows(x, "x"), _rows(dy, "dy")
    rows, dim = m.shape
    weight = _vector(weight, dim, x, weight.dtype, "weight")
    mean, rstd = _vector(mean, rows, x, torch.float32, "mean"), _vector(rstd, rows, x, torch.float32, "rstd")
    dx = x.new_empty(x.shape) if need_x else None
    dweight, dbias = (weight.new_empty(dim), weight.new_empty(dim)) if need_weight else (None, None)
    nbytes = _norm_bytes(rows, dim)
    work = x.new_empty(nbytes, dtype=torch.uint8)
    lmopt.norm_layer_backward(g.data_ptr(), g.stride(0), m.data_ptr(), m.stride(0), weight.data_ptr(), mean.data_ptr(),
                              rstd.data_ptr(), dx.data_ptr() if need_x else None, dim,
                              dweight.data_ptr() if need_weight else None,
                              dbias.data_ptr() if need_weight else None, rows, dim, xt, wt, work.data_ptr(), nbytes,
                              _stream_ptr(None))
    return dx, dweight, dbias


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, mean, rstd = layer_norm_forward(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dweight, dbias = layer_norm_backward(dy, x, weight, mean, rstd, need[0], need[1] or need[2])
        return dx, dweight if need[1] else None, dbias if ctx.has_bias and need[2] else None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5):
    """Layer norm over x's last dimension, with autograd."""
    return _LayerNorm.apply(x, weight, bias, eps)


def _xent_args(hidden, weight, target):
    if hidden.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError(f"hidden and weight must be bfloat16, not {hidden.dtype} and {weight.dtype}")
    h, w = _rows(hidden, "hidden"), weight
    if w.dim() != 2 or w.shape[1] != h.shape[1]:
        raise ValueError(f"weight must be [vocabulary, {h.shape[1]}], not {list(weight.shape)}")
    w = _rows(w, "weight")
    if target.dtype != torch.int64 or target.shape != hidden.shape[:-1] or target.get_device() != hidden.get_device():
        raise ValueError(f"target must be int64 {list(hidden.shape[:-1])} on {hidden.device}")
    return h, w, target if target.dim() == 1 and target.is_contiguous() else target.reshape(-1).contiguous()


@functools.lru_cache(maxsize=256)
def _xent_bytes(rows: int, dim: int, vocab: int, off16: int, ldw: int, backward: bool) -> int:
    """Scratch bytes; of the weight's address only its place within 16 bytes counts."""
    return lmopt.loss_xent_workspace(rows, dim, vocab, 256 + off16, ldw, backward)


@_on_stream
def xent_forward(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, ignore_index: int = -100):
    """(loss, lse), fp32, one per row of hidden: the softmax cross entropy of hidden @ weight.T against target,
    and the log of the softmax's denominator.  Rows with ignore_index have 0 for both."""
    h, w, t = _xent_args(hidden, weight, target)
    (rows, dim), vocab = h.shape, w.shape[0]
    loss, lse = h.new_empty(target.shape, dtype=torch.float32), h.new_empty(target.shape, dtype=torch.float32)
    nbytes = _xent_bytes(rows, dim, vocab, w.data_ptr() % 16, w.stride(0), False)
    work = h.new_empty(nbytes, dtype=torch.uint8)
    lmopt.loss_xent_forward(h.data_ptr(), h.stride(0), w.data_ptr(), w.stride(0), t.data_ptr(), rows, dim, vocab,
                            ignore_index, loss.data_ptr(), lse.data_ptr(), work.data_ptr(), nbytes, _stream_ptr(None))
    return loss, lse


@_on_stream
def xent_backward(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, lse: torch.Tensor,
                  grad_loss: torch.Tensor, ignore_index: int = -100, need_hidden: bool = True, need_weight: bool = True):
    """(d_hidden, d_weight) of sum(grad_loss * loss), bf16; None for one that is not needed."""
    h, w, t = _xent_args(hidden, weight, target)
    (rows, dim), vocab = h.shape, w.shape[0]
    lse, g = (_vector(x if x.dim() == 1 else x.reshape(-1), rows, h, torch.float32, n)
              for x, n in ((lse, "lse"), (grad_loss, "grad_loss")))
    dh = h.new_empty(hidden.shape) if need_hidden else None
    dw = w.new_empty(weight.shape) if need_weight else None
    nbytes = _xent_bytes(rows, dim, vocab, w.data_ptr() % 16, w.stride(0), True)
    work = h.new_empty(nbytes, dtype=torch.uint8)
    lmopt.loss_xent_backward(h.data_ptr(), h.stride(0), w.data_ptr(), w.stride(0), t.data_ptr(), lse.data_ptr(),
                             g.data_ptr(), rows, dim, vocab, ignore_index, None if dh is None else dh.data_ptr(), dim,
                             None if dw is None else dw.data_ptr(), dim, work.data_ptr(), nbytes, _stream_ptr(None))
    return dh, dw


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, target, ignore_index):
        loss, lse = xent_forward(hidden, weight, target, ignore_index)
        ctx.save_for_backward(hidden, weight, target, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad):
        hidden, weight, target, lse = ctx.saved_tensors
        dh, dw = xent_backward(hidden, weight, target, lse, grad, ctx.ignore_index, ctx.needs_input_grad[0],
                               ctx.needs_input_grad[1])
        return dh, dw, None, None


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, target: torch.Tensor, ignore_index: int = -100,
                         reduction: str = "mean"):
    """Softmax cross entropy of hidden @ weight.T against target, with autograd and without the logits.
    reduction: "mean" over the rows that are not ignored (0 if there are none), "sum" or "none"."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError(f"unknown reduction {reduction!r}")
    loss = _LinearCrossEntropy.apply(hidden, weight, target, ignore_index)
    if reduction == "none":
        return loss
    total = loss.sum()
    return total if reduction == "sum" else total / (target != ignore_index).sum().clamp(min=1)


class LMTail(torch.nn.Module):
    """The last layers of a language model: layer norm, output matrix, cross entropy.  forward gives the loss of
    hidden states [..., dim] against targets [...]; neither it nor its backward pass holds logits."""

    def __init__(self, dim: int, vocab: int, eps: float = 1e-5, ignore_index: int = -100, device="cuda"):
        super().__init__()
        bf16 = dict(dtype=torch.bfloat16, device=device)
        self.norm_weight = torch.nn.Parameter(torch.ones(dim, **bf16))
        self.norm_bias = torch.nn.Parameter(torch.zeros(dim, **bf16))
        self.weight = torch.nn.Parameter(torch.randn(vocab, dim, **bf16) * dim ** -0.5)
        self.eps, self.ignore_index = eps, ignore_index

    def forward(self, hidden: torch.Tensor, target: torch.Tensor, reduction: str = "mean") -> torch.Tensor:
        y = layer_norm(hidden, self.norm_weight, self.norm_bias, self.eps)
        return linear_cross_entropy(y, self.weight, target, self.ignore_index, reduction)
