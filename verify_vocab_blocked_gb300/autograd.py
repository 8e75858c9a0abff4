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
dequantized table's: it goes into the tensor given for it).

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
        if dy.shape[1] > 1 and dy.stride(1) != 1 or dy.shape[0] > 1 and dy.stride(0) < dy.shape[1]:
            dy = dy.contiguous()  # (an expanded gradient)
        dx, dw, db = qhead.layer_norm_bwd(x, weight, mean, rstd, dy,
                                          want_dbias=ctx.bias_type is not None)
        return (dx, dw.to(weight.dtype), None if db is None else db.to(ctx.bias_type), None, None,
                None)


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
               eps: float = 1e-6, *, center: bool = True,
               out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Differentiable layer norm of x's rows (center off: the root-mean-square
    form); in bfloat16 its result is the head's h."""
    return LayerNorm.apply(x, weight, bias, eps, center, out_dtype)


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
