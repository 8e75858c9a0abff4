"""torch.autograd integration of the fused head (page "mlx-bun 0.0.9 ->
0.0.10", src/train/loss.ts: the custom-VJP wrapper whose forward returns the
log-probabilities and keeps the lse, and whose backward turns the incoming
cotangent into dh).

Marshalling only: the forward is one qhead_fwd call, the backward one qhead_bwd
call with dlogp = the incoming gradient; nothing is computed in torch.  The
head is frozen (no gradient for it); dh is computed in fp32 and returned in the
dtype of h (bf16), as autograd requires.

The operators beside the head in the same manner: head_distill (the loss
against a teacher's top logits, differentiable in h), layer_norm
(differentiable in x, weight and bias) and embed (whose gradient is the
dequantized table's: it goes into the tensor given for it).  And the block between
them: linear (differentiable in x, weight, bias and residual) and add_norm (in x,
residual, weight and bias).

First derivatives only: a backward's result has no derivative of its own, and
differentiating it (a gradient penalty under create_graph) raises.  Every tensor
of the forward that the backward reads again, the mask among them, is saved, so
that one changed in place in between is noticed.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import qhead


class HeadLogp(torch.autograd.Function):
    """logp[m] = z[m, targets[m]] - lse[m] for every row of h (0 for rows the
    mask turns off); differentiable in h."""

    @staticmethod
    def forward(ctx, h: torch.Tensor, head: qhead.Head, targets: torch.Tensor,
                mask: torch.Tensor | None = None):
        logp, lse, _ = qhead.fwd(head, h, targets, mask, want_argmax=False)
        ctx.head = head
        ctx.save_for_backward(h, targets, lse, mask)
        return logp

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_logp: torch.Tensor):
        h, targets, lse, mask = ctx.saved_tensors
        dlogp = grad_logp.to(torch.float32).contiguous()
        dh = qhead.bwd(ctx.head, h, targets, lse, dlogp, mask)
        return dh.to(h.dtype), None, None, None


def head_logp(h: torch.Tensor, head: qhead.Head, targets: torch.Tensor,
              mask: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable per-row log-probabilities of the targets under the
    quantized head: a loss such as -head_logp(...).sum() backpropagates into h
    through the fused backward."""
    return HeadLogp.apply(h, head, targets, mask)


class HeadDistill(torch.autograd.Function):
    """loss[m] of the head against a teacher's top logits (0 for rows the mask
    turns off); differentiable in h."""

    @staticmethod
    def forward(ctx, h: torch.Tensor, head: qhead.Head, ids: torch.Tensor, tlogits: torch.Tensor,
                temperature: float = 1.0, mask: torch.Tensor | None = None):
        loss, lse, kept = qhead.distill_fwd(head, h, ids, tlogits, temperature, mask)
        ctx.head, ctx.temperature = head, temperature
        ctx.save_for_backward(h, ids, tlogits, lse, kept, mask)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss: torch.Tensor):
        h, ids, tlogits, lse, kept, mask = ctx.saved_tensors
        dloss = grad_loss.to(torch.float32).contiguous()
        dh = qhead.distill_bwd(ctx.head, h, ids, tlogits, kept, lse, dloss, ctx.temperature, mask)
        return dh, None, None, None, None, None


def head_distill(h: torch.Tensor, head: qhead.Head, ids: torch.Tensor, tlogits: torch.Tensor,
                 temperature: float = 1.0, mask: torch.Tensor | None = None) -> torch.Tensor:
    """Differentiable per-row distillation loss (qhead.distill_fwd): the cross
    entropy against the teacher's top logits less the teacher's entropy."""
    return HeadDistill.apply(h, head, ids, tlogits, temperature, mask)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t with contiguous rows that do not overlap (an expanded gradient's are not)."""
    if t.shape[1] > 1 and t.stride(1) != 1 or t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        return t.contiguous()
    return t


class LayerNorm(torch.autograd.Function):
    """y of qhead.layer_norm; differentiable in x, weight and bias."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None, eps: float,
                center: bool, out_dtype: torch.dtype):
        y, mean, rstd = qhead.layer_norm(x, weight, bias, eps, center=center, out_dtype=out_dtype)
        ctx.bias_type = None if bias is None else bias.dtype
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = qhead.layer_norm_bwd(x, weight, mean, rstd, _rows(dy),
                                          want_dbias=ctx.bias_type is not None)
        return (dx, dw.to(weight.dtype), None if db is None else db.to(ctx.bias_type), None, None,
                None)


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-6, *, center: bool = True,
               out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Differentiable layer norm of x's rows (center off: the root-mean-square
    form); in bfloat16 its result is the head's h."""
    return LayerNorm.apply(x, weight, bias, eps, center, out_dtype)


class AddNorm(torch.autograd.Function):
    """y and total of qhead.add_norm; differentiable in x, residual, weight and bias."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor,
                bias: torch.Tensor | None, eps: float, center: bool, out_dtype: torch.dtype):
        y, total, mean, rstd = qhead.add_norm(x, residual, weight, bias, eps, center=center,
                                              out_dtype=out_dtype)
        ctx.set_materialize_grads(False)
        ctx.x_type, ctx.bias_type = x.dtype, None if bias is None else bias.dtype
        ctx.save_for_backward(total, weight, mean, rstd)
        return y, total

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor | None, dtotal: torch.Tensor | None):
        total, weight, mean, rstd = ctx.saved_tensors
        if dy is None:  # only the sum is used: the norm has no part in it
            return None if dtotal is None else dtotal.to(ctx.x_type), dtotal, None, None, None, None, None
        if dtotal is not None:
            dtotal = _rows(dtotal)
        dx, dw, db = qhead.add_norm_bwd(total, weight, mean, rstd, _rows(dy), dtotal,
                                        want_dbias=ctx.bias_type is not None)
        return (dx.to(ctx.x_type), dx, dw.to(weight.dtype), None if db is None else db.to(ctx.bias_type), None, None,
                None)


def add_norm(x: torch.Tensor, residual: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
             eps: float = 1e-6, *, center: bool = True,
             out_dtype: torch.dtype = torch.bfloat16) -> tuple[torch.Tensor, torch.Tensor]:
    """Differentiable (y, total): total = x + residual and its norm (center off: the
    root-mean-square form).  The gradient of x is the residual's, formed in its type."""
    return AddNorm.apply(x, residual, weight, bias, eps, center, out_dtype)


class Linear(torch.autograd.Function):
    """y of qhead.linear; differentiable in x, weight, bias and residual."""

    @staticmethod
    def forward(ctx, x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None, act: str,
                residual: torch.Tensor | None, out_dtype: torch.dtype | None, graded: bool = True):
        keep = graded and act != "none" and any(ctx.needs_input_grad[:3])
        got = qhead.linear(x, weight, bias, act, residual, out_dtype=out_dtype, want_pre=keep)
        y, pre = got if keep else (got, None)
        ctx.act = act
        ctx.bias_type = None if bias is None else bias.dtype
        ctx.res_type = None if residual is None else residual.dtype
        ctx.save_for_backward(x, weight, pre)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy: torch.Tensor):
        x, weight, pre = ctx.saved_tensors
        want_dx, want_dw, want_db = ctx.needs_input_grad[:3]
        dx = dw = db = None
        if want_dx or want_dw or want_db:
            dx, dw, db = qhead.linear_bwd(x, weight, _rows(dy), pre, ctx.act, ctx.bias_type, want_dx=want_dx,
                                          want_dw=want_dw, want_dbias=want_db)
        return (dx, dw, None if db is None else db.to(ctx.bias_type), None,
                dy.to(ctx.res_type) if ctx.needs_input_grad[4] else None, None, None)


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None, act: str = "none",
           residual: torch.Tensor | None = None, *, out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """Differentiable act(x @ weight.T + bias) + residual (x and weight in bfloat16 or
    float16)."""
    # (parameters want gradients under no_grad too, and within forward no mode is on)
    return Linear.apply(x, weight, bias, act, residual, out_dtype, torch.is_grad_enabled())


class Embed(torch.autograd.Function):
    """Rows of the dequantized table; the gradient goes into `dw`."""

    @staticmethod
    def forward(ctx, anchor: torch.Tensor, head: qhead.Head, tokens: torch.Tensor, scale: float,
                mask: torch.Tensor | None, dw: torch.Tensor, out_dtype: torch.dtype):
        ctx.head, ctx.scale, ctx.dw = head, scale, dw
        ctx.save_for_backward(tokens, mask)
        return qhead.embed(head, tokens, scale, mask, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout: torch.Tensor):
        tokens, mask = ctx.saved_tensors
        qhead.embed_bwd(ctx.head, tokens, dout.contiguous(), ctx.scale, mask, dw=ctx.dw)
        return None, None, None, None, None, None, None


def embed(head: qhead.Head, tokens: torch.Tensor, scale: float = 1.0,
          mask: torch.Tensor | None = None, *, dw: torch.Tensor | None = None,
          out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """[M, H] rows of the dequantized table, times scale.  With dw (float32
    [V, H], as qhead.bwd_dw fills it) the result takes part in autograd: its
    backward adds the table's gradient into dw.  Without, the table is frozen."""
    if dw is None:
        return qhead.embed(head, tokens, scale, mask, out_dtype=out_dtype)
    anchor = torch.empty(0, device=tokens.device, requires_grad=True)
    return Embed.apply(anchor, head, tokens, scale, mask, dw, out_dtype)
