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
from .blocks8 import Checkpoint8, Checkpoint8Config, pack_weight8
from .ce import VocabCE
from .distill import VocabDistill
from .embed import TokenEmbedding
from .linear import ExpertLinear
from .norm import LayerNorm
from .rmsnorm import RMSNorm
from .scores import ScoreRouter

__all__ = ["MoEFunction", "VocabCEFunction", "moe_block", "vocab_cross_entropy", "moe_experts", "expert_scores",
           "layer_norm", "token_embedding", "vocab_distill", "rms_norm", "expert_linear", "rms_norm_linear8"]


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


def _none_or_rows(t):
    return None if t is None else _dense_rows(t)


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, unit):
        y, h, rstd, _, _ = unit.forward(x, weight, residual)
        ctx.unit = unit
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, weight, rstd)
        return y if residual is None else (y, h)

    @staticmethod
    @_once
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dy = torch.zeros_like(h) if dy is None else _dense_rows(dy)
        dx, dw = ctx.unit.backward(h, weight, rstd, dy, _none_or_rows(dh), want_dx=need[0] or need[1],
                                   want_dweight=need[2])
        return dx if need[0] else None, dx if need[1] else None, dw if dw is None else dw.to(weight.dtype), None


def rms_norm(x, weight, unit: RMSNorm, residual=None):
    """Differentiable RMS norm over an RMSNorm's workspace: y, or with a residual (y, h), h = x + residual."""
    return _RMSNorm.apply(x, residual, weight, unit)


def _check_gradients8(w, unit: ExpertLinear, *others):
    """Refuses, before the forward pass, what the backward pass could not do with operands in 8 bits."""
    if not torch.is_grad_enabled():
        return
    if w.requires_grad and w.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("w: expected bfloat16 or float32, the types its gradient is made in")
    if any(t is not None and t.requires_grad for t in (w, *others)) and not unit.cfg.blocks8:
        raise ValueError("operands in 8 bits: the unit was made without blocks8")


class _ExpertLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets, unit, keep):
        xs = ws = None
        kept, held = x, w
        if keep == "nothing":
            kept = None
        elif keep != "bf16":
            kept, xs = Checkpoint8(Checkpoint8Config(N=unit.cfg.N, H=unit.cfg.K)).pack(x)
        if keep == "blocks8":
            held, ws = pack_weight8(w)
            y = unit.forward(kept, held, offsets, xs, ws)
        else:
            y = unit.forward(x, w, offsets)
        ctx.unit, ctx.type = unit, w.dtype
        ctx.save_for_backward(kept, xs, held, ws, offsets)
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        x, xs, w, ws, offsets = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dw = ctx.unit.backward(x, w, dy.contiguous(), offsets, xs, ws, want_dx=need[0], want_dw=need[1],
                                   dw_dtype=ctx.type)
        return dx, dw, None, None, None


def expert_linear(x, w, unit: ExpertLinear, offsets=None, keep="bf16"):
    """Differentiable product by expert over an ExpertLinear's workspace, x [n, K] and w [E, O, K] in bf16.  keep: "bf16"
    keeps x for the backward pass, "checkpoint8" keeps it in 8 bits (which dw then takes it from), "blocks8" also computes
    y and dx in 8 bits, with w (bf16 or fp32; fp16 only where it gets no gradient) and dy packed in each pass.  The two need
    a unit made with blocks8 where gradients are asked for."""
    if keep not in ("bf16", "checkpoint8", "blocks8"):
        raise ValueError("keep: expected 'bf16', 'checkpoint8' or 'blocks8'")
    if keep == "checkpoint8" and not (torch.is_grad_enabled() and w.requires_grad):
        keep = "nothing"                # x is kept for dw alone
    elif keep != "bf16":
        _check_gradients8(w, unit, *([x] if keep == "blocks8" else []))
    return _ExpertLinear.apply(x, w, offsets, unit, keep)


class _RMSNormLinear8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, w, offsets, norm, linear):
        _, h, rstd, codes, scales = norm.forward(x, weight, residual, want_y=False, want_codes=True)
        wc, ws = pack_weight8(w)
        out = linear.forward(codes, wc, offsets, scales, ws)
        ctx.norm, ctx.linear, ctx.type = norm, linear, w.dtype
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, weight, rstd, codes, scales, wc, ws, offsets)
        return out if residual is None else (out, h)

    @staticmethod
    @_once
    def backward(ctx, dout, dh=None):
        h, weight, rstd, codes, scales, wc, ws, offsets = ctx.saved_tensors
        need = ctx.needs_input_grad
        rows = need[0] or need[1]
        if dout is None:
            dout = torch.zeros(h.shape[0], wc.shape[1], dtype=torch.bfloat16, device=h.device)
        dy, dw = ctx.linear.backward(codes, wc, dout.contiguous(), offsets, scales, ws, want_dx=rows or need[2],
                                     want_dw=need[3], dw_dtype=ctx.type)
        dx = dweight = None
        if rows or need[2]:
            dx, dweight = ctx.norm.backward(h, weight, rstd, dy, _none_or_rows(dh), want_dx=rows, want_dweight=need[2])
        return (dx if need[0] else None, dx if need[1] else None,
                dweight if dweight is None else dweight.to(weight.dtype), dw, None, None, None)


def rms_norm_linear8(x, weight, w, norm: RMSNorm, linear: ExpertLinear, residual=None, offsets=None):
    """The product by expert, in 8 bits, of an RMS norm's output, which is never written but in 8 bits (and kept so for
    the backward pass): out, or with a residual (out, h).  x, residual and w in bf16; `linear` made with blocks8.  The norm
    is of every row: what rows of no expert hold enters `weight`'s gradient where it is no number (0 x NaN)."""
    if x.dtype != torch.bfloat16:
        raise TypeError("x: expected bfloat16")
    _check_gradients8(w, linear, x, weight, residual)
    return _RMSNormLinear8.apply(x, residual, weight, w, offsets, norm, linear)
