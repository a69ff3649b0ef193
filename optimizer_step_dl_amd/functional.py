"""Autograd forms of the vocabulary operators, for a torch training loop whose
step is FusedAdamW: the embedding lookup at one end of a model and the policy
or preference loss at the other.

    x = embedding(ids, table, scale=d ** 0.5, grad_buffer=table.grad)
    total, loss, logp = policy_loss(model(x), labels, advantages, old_logp=old)
    (total * loss_scale).backward()
    optimizer.step(gradient_scale=loss_scale)

All arithmetic runs in the library's kernels; these functions shape the
tensors, allocate outputs and workspaces and keep what the backward pass
needs.  Every call submits to its device's current stream and returns without
waiting; the backward passes run, as torch's own, on the stream of the forward
call.  Calls under graph capture raise RadamwError (as every entry point of
the library does); second derivatives raise.
"""
from __future__ import annotations

import threading
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _abi

__all__ = ["embedding", "policy_loss", "preference_loss"]


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as [n, width] with unit column stride and rows that do not overlap;
    copied only where it is not."""
    t = t.reshape(-1, t.shape[-1])
    row, col = t.stride()
    rows, cols = t.shape
    return t if (cols == 1 or col == 1) and (rows <= 1 or row >= cols) else t.contiguous()


def _flat32(t: Optional[torch.Tensor], what: str, n: int) -> Optional[torch.Tensor]:
    """A per-row or per-sequence input as n contiguous FP32 values, without
    its history."""
    if t is None:
        return None
    if t.numel() != n:
        raise ValueError(f"{what} has {t.numel()} values, expected {n}")
    return t.detach().reshape(-1).to(torch.float32).contiguous()


def _empty32(shape, device) -> torch.Tensor:
    """An FP32 output, whatever torch's default dtype."""
    return torch.empty(shape, dtype=torch.float32, device=device)


# --------------------------------------------------------------- embedding --

# Per device index, an event behind the last write into any grad_buffer.
_buffer_writes: dict = {}
_buffer_lock = threading.Lock()


def _write_in_order(ctx, device: torch.device, write) -> None:
    """Submit ``write``, which adds into a grad_buffer, from a backward pass.

    The engine orders streams along the gradients that nodes hand on, and
    there is none here.  So the write waits for the device's earlier ones,
    which may have run on other streams (into whichever buffer: two tensors
    may be the same memory); the table's own gradient node, which may add to
    the same memory, waits for it; and at the end of backward() so does the
    stream that called it.  9 us of host time (a lookup of 16 tokens with its
    backward takes 50 us instead of 41); nothing for the GPU where all of
    them are one stream."""
    stream = torch.cuda.current_stream(device)
    with _buffer_lock:
        last = _buffer_writes.get(device.index)
        if last is not None and not torch.cuda.is_current_stream_capturing():  # a capture is refused by the write
            stream.wait_event(last)
        write()
        done = torch.cuda.Event()
        done.record(stream)
        _buffer_writes[device.index] = done

    def wait(*_):
        if _abi._raw_stream is None or _abi._raw_stream(device.index) != stream.cuda_stream:
            torch.cuda.current_stream(device).wait_event(done)

    node = ctx.next_functions[0][0]
    if node is not None:  # a table that takes a gradient; only a model_copy may

        def before_node(*_):
            handle.remove()
            wait()

        handle = node.register_prehook(before_node)
    torch.autograd.Variable._execution_engine.queue_callback(wait)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, ids, values, scale, padding_id, out_dtype, grad_buffer):
        rows, dim = values.shape
        ids = ids.contiguous()
        out = torch.empty((ids.numel(), dim), dtype=out_dtype, device=values.device)
        _abi.radamw_embedding_lookup(values.detach(), ids, out, scale)
        ctx.save_for_backward(ids)
        ctx.scale, ctx.padding_id, ctx.grad_buffer = scale, padding_id, grad_buffer
        ctx.shape = (rows, dim)
        # the dtype a leaf keeps its gradient in, where this torch knows one
        ctx.grad_dtype = (getattr(table, "grad_dtype", None) if table.is_leaf else None) or table.dtype
        return out.view(*ids.shape, dim)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        ids, = ctx.saved_tensors
        rows, dim = ctx.shape
        grad_out = _rows(grad_out)
        into = ctx.grad_buffer
        grad = torch.empty((rows, dim), dtype=ctx.grad_dtype, device=grad_out.device) if into is None else into
        workspace = torch.empty(_abi.radamw_embedding_grad_workspace_bytes(ids.numel(), rows, dim), dtype=torch.uint8,
                                device=grad_out.device)
        if into is None:
            _abi.radamw_embedding_grad(grad_out, ids, grad, workspace, ctx.scale, ctx.padding_id, False)
            return (grad,) + (None,) * 6
        _write_in_order(ctx, grad.device, lambda: _abi.radamw_embedding_grad(
            grad_out, ids, grad, workspace, ctx.scale, ctx.padding_id, True))
        return (None,) * 7


def embedding(ids: torch.Tensor, table: torch.Tensor, *, scale: float = 1.0, padding_id: Optional[int] = None,
              out_dtype: Optional[torch.dtype] = None, model_copy: Optional[torch.Tensor] = None,
              grad_buffer: Optional[torch.Tensor] = None) -> torch.Tensor:
    """scale * table[ids], of shape ids.shape + (dim,); zeros where an id is
    outside the table.

    ``table`` [rows, dim] takes the gradient: the sum over tokens in a fixed
    order, tokens of ``padding_id`` left out, in ``table.grad_dtype`` where
    a leaf has that set, else the table's dtype.  ``model_copy`` is a float16 /
    bfloat16 tensor of the same shape to read instead of the table (the copy
    FusedAdamW rewrites at every step).  ``out_dtype`` defaults to what is
    read.  With ``grad_buffer`` (a [rows, dim] tensor, as ``table.grad`` of a
    flattened FusedAdamW group) the backward pass adds the rows that occur
    into that tensor and hands torch no gradient: nothing of the table's size
    is written, and hooks on the table do not run.  Such writes follow one
    another, whichever streams the forward passes ran on, and the stream that
    calls backward() goes on behind them."""
    if table.dim() != 2:
        raise ValueError("table must be [rows, dim]")
    values = table if model_copy is None else model_copy
    if values.shape != table.shape:
        raise ValueError(f"model_copy has shape {tuple(values.shape)}, expected {tuple(table.shape)}")
    if grad_buffer is not None and (grad_buffer.shape != table.shape or grad_buffer.requires_grad):
        raise ValueError("grad_buffer must be a tensor of the table's shape that takes no gradient itself")
    if padding_id is not None and not 0 <= padding_id < table.shape[0]:
        raise ValueError(f"padding_id {padding_id} is outside the table's {table.shape[0]} rows")
    return _Embedding.apply(table, ids, values, float(scale), padding_id, out_dtype or values.dtype, grad_buffer)


# ------------------------------------------------------------------ losses --

class _PolicyLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, old_logp, ref_logp, advantages, weights, opts):
        n, dev = logits.shape[0], logits.device
        total, loss, logp, stats = (_empty32(s, dev) for s in ((), n, n, (n, 4)))
        _abi.radamw_policy_loss(logits.detach(), labels, old_logp, advantages, opts, total, loss, logp,
                                ref_logp=ref_logp, weights=weights, row_stats=stats)
        ctx.save_for_backward(logits, labels, stats)
        ctx.mark_non_differentiable(loss, logp)
        ctx.set_materialize_grads(False)
        return total, loss, logp

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_total, *_):
        return (_logits_backward(ctx, grad_total),) + (None,) * 6


class _PreferenceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, labels, offsets, ref_logp, weights, opts):
        n, dev, pairs = logits.shape[0], logits.device, weights.numel()
        total, loss, seq_logp, logp, stats = (_empty32(s, dev) for s in ((), pairs, 2 * pairs, n, (n, 4)))
        _abi.radamw_preference_loss(logits.detach(), labels, offsets, ref_logp, opts, total, loss, seq_logp, logp,
                                    stats, weights=weights)
        ctx.save_for_backward(logits, labels, stats)
        ctx.mark_non_differentiable(loss, seq_logp)
        ctx.set_materialize_grads(False)
        return total, loss, seq_logp

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_total, *_):
        return (_logits_backward(ctx, grad_total),) + (None,) * 5


def _logits_backward(ctx, grad_total):
    if grad_total is None:
        return None
    logits, labels, stats = ctx.saved_tensors
    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    _abi.radamw_logits_grad(logits.detach(), labels, stats, grad, upstream=grad_total.to(torch.float32).contiguous())
    return grad


def _labels(logits: torch.Tensor, labels: torch.Tensor) -> torch.Tensor:
    if labels.shape != logits.shape[:-1]:
        raise ValueError(f"labels have shape {tuple(labels.shape)}, expected {tuple(logits.shape[:-1])}")
    return labels.reshape(-1).contiguous()


def policy_loss(logits: torch.Tensor, labels: torch.Tensor, advantages: torch.Tensor, *,
                old_logp: Optional[torch.Tensor] = None, ref_logp: Optional[torch.Tensor] = None,
                weights: Optional[torch.Tensor] = None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0):
    """(total, loss, logp) of the clipped policy loss with a KL term
    (radamw_policy_loss) over logits [..., vocab] and labels [...].

    ``total`` is differentiable with respect to the logits alone; ``loss`` and
    ``logp`` (of labels' shape, FP32) are not.  Rows whose label is outside
    the vocabulary (-100) take no part.  ``weights`` default to 1 / (number of
    rows that take part): the mean."""
    shape, vocab = labels.shape, logits.shape[-1]
    flat = _labels(logits, labels)
    n = flat.numel()
    if weights is None:
        taken = (flat >= 0) & (flat < vocab)
        w = taken.float() / taken.sum().clamp(min=1)
    else:
        w = _flat32(weights, "weights", n)
    opts = _abi.policy_options(clip_low, clip_high, kl_coef)
    total, loss, logp = _PolicyLoss.apply(_rows(logits), flat, _flat32(old_logp, "old_logp", n),
                                          _flat32(ref_logp, "ref_logp", n), _flat32(advantages, "advantages", n), w, opts)
    return total, loss.view(shape), logp.view(shape)


def preference_loss(logits: torch.Tensor, labels: torch.Tensor, offsets: torch.Tensor, ref_logp: torch.Tensor, *,
                    weights: Optional[torch.Tensor] = None, beta: float = 0.1, label_smoothing: float = 0.0):
    """(total, loss, seq_logp) of the preference loss
    (radamw_preference_loss) over packed rows of logits [n, vocab].

    ``offsets`` (2 * pairs + 1, device integers) give the rows of the chosen
    sequences, then of the rejected ones; ``ref_logp`` their summed
    log-probabilities under the reference model.  ``total`` is differentiable
    with respect to the logits alone.  ``weights`` default to 1 / pairs."""
    flat = _labels(logits, labels)
    if offsets.dim() != 1 or offsets.numel() < 3 or offsets.numel() % 2 == 0:
        raise ValueError(f"offsets must hold 2 * pairs + 1 entries (got {offsets.numel()})")
    pairs = offsets.numel() // 2
    if weights is None:
        w = torch.full((pairs,), 1.0 / pairs, dtype=torch.float32, device=logits.device)
    else:
        w = _flat32(weights, "weights", pairs)
    return _PreferenceLoss.apply(_rows(logits), flat, offsets.to(flat.dtype).contiguous(),
                                 _flat32(ref_logp, "ref_logp", 2 * pairs), w,
                                 _abi.preference_options(beta, label_smoothing))
