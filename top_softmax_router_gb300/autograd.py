"""torch.autograd wrappers over the C ABI: the MoE block, the vocabulary cross-entropy head and the operators
around them as differentiable functions, so they drop into a training loop.

Argument marshalling only: forward and backward call the library's moe_route / moe_forward /
moe_backward and moe_ce_forward / moe_ce_backward.  The library returns fp32 weight gradients;
autograd hands each gradient back in its parameter's dtype, so bf16 weights receive bf16
gradients.  (A caller that keeps fp32 master weights and wants the fp32 gradients uses MoEBlock /
VocabCE directly.)
"""
from __future__ import annotations

import functools

import torch

from .api import MoEBlock
from .ce import VocabCE
from .distill import VocabDistill
from .embed import TokenEmbedding
from .norm import LayerNorm
from .scores import ScoreRouter

__all__ = ["MoEFunction", "VocabCEFunction", "moe_block", "vocab_cross_entropy", "moe_experts", "expert_scores",
           "layer_norm", "token_embedding", "vocab_distill"]


class _Final(torch.autograd.Function):
    """The gradients as they are; differentiating them raises."""

    @staticmethod
    def forward(ctx, _anchor, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the library's gradients cannot be differentiated twice")


def _once(backward):
    """A backward pass that the library computes, without a graph.  Under create_graph its gradients would pass for
    constants; they raise instead, also where the upstream gradient is one (torch's once_differentiable lets those by)."""

    @functools.wraps(backward)
    def run(ctx, *upstream):
        with torch.no_grad():
            grads = backward(ctx, *upstream)
        if not torch.is_grad_enabled():
            return grads
        anchor = next((t for t in (*upstream, *ctx.saved_tensors) if t is not None and t.requires_grad), None)
        if anchor is None:
            return grads
        final = iter(_Final.apply(anchor, *(g for g in grads if g is not None)))
        return tuple(None if g is None else next(final) for g in grads)

    return run


class MoEFunction(torch.autograd.Function):
    """Y = MoE(X) with top-k softmax routing (Wr, bias), SwiGLU experts (Wg, Wu, Wd), chunked by (c, K_max).
    Gradients flow to X, Wr, Wg, Wu and Wd; the bias gets none (it only shifts the routing)."""

    @staticmethod
    def forward(ctx, X, Wr, bias, Wg, Wu, Wd, blk: MoEBlock):
        idx, gates = blk.route(X, Wr, bias)
        Y = blk.forward(X, idx, gates, Wg, Wu, Wd)
        ctx.blk = blk
        ctx.save_for_backward(X, Wr, Wg, Wu, Wd, idx, gates)
        return Y

    @staticmethod
    @_once
    def backward(ctx, dY):
        X, Wr, Wg, Wu, Wd, idx, gates = ctx.saved_tensors
        g = ctx.blk.backward(X, Wr, idx, gates, Wg, Wu, Wd, dY.contiguous(), want_dgates=False)
        return g["dX"], g["dWr"], None, g["dWg"], g["dWu"], g["dWd"], None


def moe_block(X, Wr, bias, Wg, Wu, Wd, blk: MoEBlock):
    """Differentiable MoE block over an MoEBlock's workspace (X [N,H] bf16; weights as in include/moe.h)."""
    return MoEFunction.apply(X, Wr, bias, Wg, Wu, Wd, blk)


class VocabCEFunction(torch.autograd.Function):
    """Mean cross-entropy of the logits X W^T against `targets`, without forming the logits."""

    @staticmethod
    def forward(ctx, X, W, targets, ce: VocabCE):
        loss, lse, mean = ce.forward(X, W, targets)
        ctx.ce = ce
        ctx.save_for_backward(X, W, targets, lse)
        return mean[0]

    @staticmethod
    @_once
    def backward(ctx, dmean):
        X, W, targets, lse = ctx.saved_tensors
        n = X.shape[0]
        dloss = (dmean.float() / max(n, 1)).expand(n).contiguous()
        dX, dW = ctx.ce.backward(X, W, targets, lse, dloss)
        return dX, dW, None, None


def vocab_cross_entropy(X, W, targets, ce: VocabCE):
    """Differentiable mean cross-entropy head over a VocabCE's workspace."""
    return VocabCEFunction.apply(X, W, targets, ce)


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, idx, gates, Wg, Wu, Wd, blk):
        ctx.blk = blk
        ctx.save_for_backward(X, idx, gates, Wg, Wu, Wd)
        return blk.forward(X, idx, gates, Wg, Wu, Wd)

    @staticmethod
    @_once
    def backward(ctx, dY):
        X, idx, gates, Wg, Wu, Wd = ctx.saved_tensors
        g = ctx.blk.experts_backward(X, idx, gates, Wg, Wu, Wd, dY.contiguous())
        return g["dX"], None, g["dgates"], g["dWg"], g["dWu"], g["dWd"], None


def moe_experts(X, idx, gates, Wg, Wu, Wd, blk: MoEBlock):
    """The experts for choices and gates that another router made (expert_scores): gradients flow to X, the gates,
    Wg, Wu and Wd."""
    return _Experts.apply(X, idx, gates, Wg, Wu, Wd, blk)


class _Scores(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, router):
        idx, weights, counts = router.forward(logits, bias)
        ctx.router = router
        ctx.save_for_backward(logits, idx)
        ctx.mark_non_differentiable(idx, counts)
        return idx, weights, counts

    @staticmethod
    @_once
    def backward(ctx, _idx, dweights, _counts):
        logits, idx = ctx.saved_tensors
        return ctx.router.backward(logits, idx, dweights.contiguous()), None, None


def expert_scores(logits, router: ScoreRouter, bias=None):
    """(idx, weights, counts) of a ScoreRouter; the weights' gradient flows to the logits, the bias gets none."""
    return _Scores.apply(logits, bias, router)


def _dense_rows(t):
    """`t` where the library can read it row by row (an expanded gradient, say, it cannot), else a copy."""
    n, h = t.shape
    return t if t.is_contiguous() or ((h < 2 or t.stride(1) == 1) and (n < 2 or t.stride(0) >= h)) else t.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, unit):
        y, mean, rstd = unit.forward(x, weight, bias)
        ctx.unit, ctx.bias_type = unit, None if bias is None else bias.dtype
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw, db = ctx.unit.backward(x, weight, mean, rstd, _dense_rows(dy), want_dx=need[0],
                                       want_dweight=need[1], want_dbias=need[2])
        return dx, dw if dw is None else dw.to(weight.dtype), db if db is None else db.to(ctx.bias_type), None


def layer_norm(x, weight, bias, unit: LayerNorm):
    """Differentiable layer norm of a matrix's rows over a LayerNorm's workspace."""
    return _LayerNorm.apply(x, weight, bias, unit)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, unit):
        ctx.unit, ctx.type = unit, table.dtype
        ctx.save_for_backward(ids)
        return unit.forward(ids, table)

    @staticmethod
    @_once
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        return None, ctx.unit.backward(ids, _dense_rows(dy)).to(ctx.type), None


def token_embedding(ids, table, unit: TokenEmbedding):
    """Differentiable lookup over a TokenEmbedding's workspace (a dense gradient, in the table's type)."""
    return _Embedding.apply(ids, table, unit)


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, X, W, ids, teacher, unit):
        loss, lse, mean = unit.forward(X, W, ids, teacher)
        ctx.unit = unit
        ctx.save_for_backward(X, W, ids, teacher, lse)
        return mean[0]

    @staticmethod
    @_once
    def backward(ctx, dmean):
        X, W, ids, teacher, lse = ctx.saved_tensors
        n = X.shape[0]
        dloss = (dmean.float() / max(n, 1)).expand(n).contiguous()
        dX, dW = ctx.unit.backward(X, W, ids, teacher, lse, dloss, dW_dtype=torch.bfloat16)
        return dX, dW, None, None, None


def vocab_distill(X, W, ids, teacher, unit: VocabDistill):
    """Differentiable mean distillation loss of the head X W^T against a teacher's top logits."""
    return _Distill.apply(X, W, ids, teacher, unit)
