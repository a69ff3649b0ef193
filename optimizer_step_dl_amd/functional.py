"""Autograd forms of the vocabulary and block operators, for a torch training
loop whose step is FusedAdamW: the embedding lookup at one end of a model, the
residual stream's dropout and norms around each block, a router's balance
loss, and the policy or preference loss at the other end.

    x = embedding(ids, table, scale=d ** 0.5, grad_buffer=table.grad)
    x = dropout(x, 0.1, seed=run, offset=site(step, 0))
    y = residual_norm(x, None, pre_weight=norms[0])
    for i, block in enumerate(blocks):
        x, y = residual_norm(x, block(y), post_weight=posts[i], pre_weight=norms[i + 1], gate=gates[i], p=0.1,
                             seed=run, offset=site(step, i + 1))
    balance, *_ = balance_loss(router_logits, chosen_experts)
    total, loss, logp = policy_loss(head(y), labels, advantages, old_logp=old)
    ((total + balance) * loss_scale).backward()
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

__all__ = ["balance_loss", "dropout", "embedding", "policy_loss", "preference_loss", "residual_norm"]


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as [n, width] with unit column stride and rows that do not overlap;
    copied only where it is not."""
    t = t.reshape(-1, t.shape[-1])
    row, col = t.stride()
    rows, cols = t.shape
    if (cols == 1 or col == 1) and (rows <= 1 or row >= cols):
        return t
    # contiguous() would keep the strides of a tensor without rows, whatever they are
    return t.clone(memory_format=torch.contiguous_format)


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


# ------------------------------------------------------------------ blocks --

class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, opts):
        ctx.opts = opts
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        _abi.radamw_dropout(x.detach(), out, opts)
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out):
        grad = torch.empty(grad_out.shape, dtype=grad_out.dtype, device=grad_out.device)
        _abi.radamw_dropout(_rows(grad_out), grad, ctx.opts)
        return grad, None


def dropout(x: torch.Tensor, p: float, *, seed: int, offset: int = 0, first_row: int = 0,
            training: bool = True) -> torch.Tensor:
    """radamw_dropout of x [..., dim], whose leading dimensions are its rows:
    x / keep where the generator keeps an element, else 0.

    Which elements are kept depends on ``seed``, ``offset``, the row (counted
    from ``first_row``) and the column alone, so that a recomputed pass has the
    same ones; every use of a step and every step needs an offset of its own.
    No mask is stored.  Without ``training`` x itself is returned."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be within 0 .. 1 (got {p})")
    if not training or p == 0.0:
        return x
    if x.dim() == 0:
        raise ValueError("x must have at least one dimension")
    return _Dropout.apply(_rows(x), _abi.dropout_options(p, seed, offset, first_row)).view(x.shape)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, branch, gate, post_weight, pre_weight, opts, per, out_dtype):
        n, dim = x.shape
        dev = x.device
        rstd = _empty32((2, n), dev)
        h = None if branch is None else torch.empty((n, dim), dtype=x.dtype, device=dev)
        out = None if pre_weight is None else torch.empty((n, dim), dtype=out_dtype, device=dev)
        # without rows there is no gate row for the call to read
        given = [None if t is None else t.detach() for t in (x, branch, gate if n else None, post_weight, pre_weight)]
        _abi.radamw_residual_norm(given[0], given[1], opts, gate=given[2], rows_per_gate=per, post_weight=given[3],
                                  pre_weight=given[4], h=h, out=out, rstd=rstd)
        # h is read again by the norm before the next block alone
        ctx.save_for_backward(None if pre_weight is None else x if h is None else h, branch, gate, post_weight,
                              pre_weight, rstd)
        ctx.opts, ctx.per = opts, per
        ctx.set_materialize_grads(False)
        return h, out

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_h, grad_out):
        h, branch, gate, post_weight, pre_weight, rstd = ctx.saved_tensors
        like = grad_h if grad_h is not None else grad_out
        if like is None:
            return (None,) * 8
        n, dim = like.shape
        dev = like.device
        asked = ctx.needs_input_grad

        def empty(t, wanted=True):
            return torch.empty(t.shape, dtype=t.dtype, device=dev) if t is not None and wanted else None

        if grad_out is None:  # nothing came through the norm before the next block
            pre_weight = None
        stream = h.dtype if h is not None else grad_h.dtype
        grad_x = torch.empty((n, dim), dtype=stream, device=dev)
        grad_branch = empty(branch)
        grad_gate, grad_post, grad_pre = empty(gate, asked[2]), empty(post_weight, asked[3]), empty(pre_weight, asked[4])
        gate_out = grad_gate
        if n == 0:  # as in the forward call; the gate's gradient is a sum over no rows
            gate_out = gate = None
            if grad_gate is not None:
                grad_gate.zero_()
        need = _abi.radamw_residual_grad_workspace_bytes(n, dim, ctx.per or 1)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _abi.radamw_residual_norm_grad(
            h, branch, ctx.opts, rstd, workspace, gate=gate, rows_per_gate=ctx.per, post_weight=post_weight,
            pre_weight=pre_weight, grad_h=None if grad_h is None else _rows(grad_h),
            grad_out=None if grad_out is None else _rows(grad_out), grad_x=grad_x, grad_branch=grad_branch,
            grad_gate=gate_out, grad_post_weight=grad_post, grad_pre_weight=grad_pre)
        return grad_x, grad_branch, grad_gate, grad_post, grad_pre, None, None, None


def _gate_rows(gate: torch.Tensor, shape: torch.Size):
    """(gate as [rows, dim], rows of the stream that share one)."""
    g = (1,) * (len(shape) - gate.dim()) + tuple(gate.shape)
    k = len(shape) - 1
    while k > 0 and g[k - 1] == 1:
        k -= 1
    if len(g) != len(shape) or g[:k] != tuple(shape[:k]) or g[-1] != shape[-1]:
        raise ValueError(f"gate of shape {tuple(gate.shape)} is not the leading part of {tuple(shape)}: expected its "
                         "shape with trailing dimensions before the last one (or all) of size 1")
    per = 1
    for s in shape[k:-1]:
        per *= s
    return _rows(gate), max(1, per)


def residual_norm(x: torch.Tensor, branch: Optional[torch.Tensor], *, pre_weight: Optional[torch.Tensor] = None,
                  post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                  residual_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0, p: float = 0.0,
                  seed: int = 0, offset: int = 0, first_row: int = 0, training: bool = True,
                  out_dtype: Optional[torch.dtype] = None):
    """radamw_residual_norm of x and branch [..., dim]: with

        h = x + residual_scale * gate * dropout(norm(branch) * post_weight)
        out = norm(h) * pre_weight

    (h, out); h alone without a ``pre_weight``; out = norm(x) * pre_weight
    alone where ``branch`` is None.  No ``post_weight``: the branch as it is.
    The weights are (weight_offset + weight) [dim], of one dtype.

    ``gate`` broadcasts to x's shape along dimensions before the last: [dim],
    [batch, 1, dim] for x [batch, length, dim], or x's own shape.  Dropout as
    in dropout().  x has the branch's dtype or float32; out has the branch's
    (without a branch ``out_dtype``, by default x's).  Gradients reach x, the
    branch, the gate and both weights."""
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be within 0 .. 1 (got {p})")
    if branch is None:
        if pre_weight is None or gate is not None or post_weight is not None:
            raise ValueError("without a branch there is the norm with pre_weight alone")
        kind = out_dtype or x.dtype
    else:
        if branch.shape != x.shape:
            raise ValueError(f"branch has shape {tuple(branch.shape)}, expected {tuple(x.shape)}")
        kind = branch.dtype
        if out_dtype not in (None, kind):
            raise ValueError(f"out has the branch's dtype {kind} (got {out_dtype})")
    if x.dtype not in (kind, torch.float32):
        raise ValueError(f"x must be {kind} or float32 (got {x.dtype})")
    for w, what in ((post_weight, "post_weight"), (pre_weight, "pre_weight")):
        if w is not None and tuple(w.shape) != (x.shape[-1],):
            raise ValueError(f"{what} has shape {tuple(w.shape)}, expected {(x.shape[-1],)}")
    rows, per = (None, None) if gate is None else _gate_rows(gate, x.shape)
    drop = p if training and branch is not None else 0.0
    opts = _abi.residual_options(eps, weight_offset, residual_scale, drop, seed, offset, first_row)
    h, out = _ResidualNorm.apply(_rows(x), None if branch is None else _rows(branch), rows,
                                 None if post_weight is None else post_weight.contiguous(),
                                 None if pre_weight is None else pre_weight.contiguous(), opts, per, kind)
    if branch is None:
        return out.view(x.shape)
    return h.view(x.shape) if out is None else (h.view(x.shape), out.view(x.shape))


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, mask, offsets, weights, opts):
        n, experts = logits.shape
        dev = logits.device
        groups = weights.numel()
        total, loss, mean_prob = (_empty32(s, dev) for s in ((), groups, (groups, experts)))
        counts = torch.empty((groups, experts), dtype=torch.int32, device=dev)
        tokens = torch.empty(groups, dtype=torch.int32, device=dev)
        need = _abi.radamw_balance_workspace_bytes(n, experts, groups)
        _abi.radamw_balance_loss(logits.detach(), ids, opts, total, loss, counts, tokens, mean_prob,
                                 torch.empty(need, dtype=torch.uint8, device=dev), mask=mask, offsets=offsets,
                                 weights=weights)
        ctx.save_for_backward(logits, mask, offsets, weights, counts, tokens)
        ctx.opts, ctx.top_k = opts, ids.shape[1]
        ctx.mark_non_differentiable(loss, counts, mean_prob)
        ctx.set_materialize_grads(False)
        return total, loss, counts, mean_prob

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_total, *_):
        if grad_total is None:
            return (None,) * 6
        logits, mask, offsets, weights, counts, tokens = ctx.saved_tensors
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        _abi.radamw_balance_grad(logits.detach(), ctx.top_k, ctx.opts, counts, tokens, grad, mask=mask, offsets=offsets,
                                 weights=weights, upstream=grad_total.to(torch.float32).contiguous())
        return (grad,) + (None,) * 5


def balance_loss(logits: torch.Tensor, ids: torch.Tensor, *, mask: Optional[torch.Tensor] = None,
                 offsets: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                 balance_coef: float = 0.01, z_coef: float = 0.0, score: str = "softmax"):
    """(total, loss, counts, mean_prob) of a router's balance loss and z-loss
    (radamw_balance_loss) over logits [..., experts] and the chosen experts
    ids [..., top_k].

    ``mask`` [...] (bool) leaves out padding.  ``offsets`` (groups + 1, device
    integers) give groups of rows that are balanced each by itself; without
    them all rows are one group.  ``total`` is differentiable with respect to
    the logits alone; ``loss`` (groups), ``counts`` [groups, experts] (int32)
    and ``mean_prob`` [groups, experts] are not.  ``weights`` default to 1 /
    groups.  The counts are those of these rows: a loss over the rows of several
    processes takes radamw_balance_loss, sums of its counts and tokens, and
    radamw_balance_grad."""
    if ids.shape[:-1] != logits.shape[:-1]:
        raise ValueError(f"ids have shape {tuple(ids.shape)}, expected {tuple(logits.shape[:-1])} + (top_k,)")
    if mask is not None and mask.shape != logits.shape[:-1]:
        raise ValueError(f"mask has shape {tuple(mask.shape)}, expected {tuple(logits.shape[:-1])}")
    if offsets is not None and (offsets.dim() != 1 or offsets.numel() < 2):
        raise ValueError(f"offsets must hold groups + 1 entries (got {tuple(offsets.shape)})")
    groups = 1 if offsets is None else offsets.numel() - 1
    if weights is None:
        w = torch.full((groups,), 1.0 / groups, dtype=torch.float32, device=logits.device)
    else:
        w = _flat32(weights, "weights", groups)
    opts = _abi.balance_options(balance_coef, z_coef, score)
    chosen = ids.reshape(-1, ids.shape[-1]).contiguous()
    return _BalanceLoss.apply(_rows(logits), chosen, None if mask is None else mask.reshape(-1).contiguous(),
                              None if offsets is None else offsets.to(chosen.dtype).contiguous(), w, opts)
