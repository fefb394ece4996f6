"""Optional autograd wrappers around the ftk ops, and the LoRA+ learning-rate
rule for building optimizer parameter groups.

Each Function runs the library's forward kernel, saves what the backward
kernel needs, and calls the backward kernel: argument marshalling only, no
arithmetic of its own (weight gradients, which the kernels produce in fp32,
are cast to the weight's dtype as autograd requires).  A step may be captured
into a CUDA graph, gradients included (torch.autograd.grad, or backward with no
earlier eager graph of the same leaves alive: torch ties a leaf's accumulation
to the stream that first used it, and a capture may not wait for another).

LoRA+ ("Chronicals", arXiv 2601.02609, abstract, optimisation (3)): the
adapter matrix B of every LoRA pair learns at 16 times the rate of A.
``lora_plus_param_groups`` turns that rule into parameter groups for any
torch optimizer.
"""
from __future__ import annotations

from typing import Iterable, List, Optional, Tuple

import numpy as np
import torch
from torch.autograd.function import once_differentiable

from . import ftk

LORA_PLUS_RATIO = 16.0


def _kept(table):
    """A copy of a host table for the backward pass: the caller's may change
    before it runs, and the angles have to be those of the forward."""
    return None if table is None else np.asarray(table).copy()


class RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, eps: float):
        y, rstd = ftk.rmsnorm_fwd(x, w, eps)
        ctx.save_for_backward(x, w, rstd)
        ctx.eps = eps
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w, rstd = ctx.saved_tensors
        dx, dw = ftk.rmsnorm_bwd(dy.contiguous(), x, w, rstd, ctx.eps)
        return dx, dw.to(w.dtype), None


class AddRMSNorm(torch.autograd.Function):
    """(h, y) = (x + res, rmsnorm(x + res) * w)."""

    @staticmethod
    def forward(ctx, x, res, w, eps: float):
        h, y, rstd = ftk.rmsnorm_add_fwd(x, res, w, eps)
        ctx.save_for_backward(h, w, rstd)
        ctx.eps = eps
        return h, y

    @staticmethod
    def backward(ctx, dh, dy):
        h, w, rstd = ctx.saved_tensors
        dh = torch.zeros_like(h) if dh is None else dh.contiguous()
        dy = torch.zeros_like(h) if dy is None else dy.contiguous()
        dx, dw = ftk.rmsnorm_add_bwd(dy, dh, h, w, rstd, ctx.eps)
        return dx, dx, dw.to(w.dtype), None


class SwiGLU(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g, u):
        ctx.save_for_backward(g, u)
        return ftk.swiglu_fwd(g, u)

    @staticmethod
    def backward(ctx, dh):
        g, u = ctx.saved_tensors
        dg, du = ftk.swiglu_bwd(dh.contiguous(), g, u)
        return dg, du


class QKRope(torch.autograd.Function):
    """Rotates copies of q [T, Hq, D] and k [T, Hkv, D]; inv_freq (host, D/2)
    replaces theta when given."""

    @staticmethod
    def forward(ctx, q, k, cu_seqlens, theta: float, inv_freq=None):
        q, k = q.clone(), k.clone()
        if inv_freq is None:
            ftk.qk_rope_fwd(q, k, cu_seqlens, theta)
        else:
            ftk.qk_rope_freq_fwd(q, k, cu_seqlens, inv_freq)
        ctx.save_for_backward(cu_seqlens)
        ctx.theta, ctx.inv_freq = theta, _kept(inv_freq)
        return q, k

    @staticmethod
    def backward(ctx, dq, dk):
        (cu,) = ctx.saved_tensors
        dq, dk = dq.contiguous().clone(), dk.contiguous().clone()
        if ctx.inv_freq is None:
            ftk.qk_rope_bwd(dq, dk, cu, ctx.theta)
        else:
            ftk.qk_rope_freq_bwd(dq, dk, cu, ctx.inv_freq)
        return dq, dk, None, None, None


class QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, cu_seqlens, eps: float, theta: float, inv_freq=None):
        qo, ko, rq, rk = ftk.qk_norm_rope_fwd(q, k, wq, wk, cu_seqlens, eps, theta=theta,
                                              inv_freq=inv_freq)
        ctx.save_for_backward(q, k, wq, wk, rq, rk, cu_seqlens)
        ctx.eps, ctx.theta, ctx.inv_freq = eps, theta, _kept(inv_freq)
        return qo, ko

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, wq, wk, rq, rk, cu = ctx.saved_tensors
        gq, gk, dwq, dwk = ftk.qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), q, k, wq, wk,
                                                rq, rk, cu, ctx.eps, theta=ctx.theta,
                                                inv_freq=ctx.inv_freq)
        return gq, gk, dwq.to(wq.dtype), dwk.to(wk.dtype), None, None, None, None


class QKMrope(torch.autograd.Function):
    """q [T, Hq, D] and k [T, Hkv, D] turned by positions on several axes
    (pos int32 [axes, T]; axis_of: D/2 axes on the host)."""

    @staticmethod
    def forward(ctx, q, k, pos, axis_of, theta: float, inv_freq=None):
        ctx.save_for_backward(pos)
        ctx.axis_of, ctx.theta, ctx.inv_freq = _kept(axis_of), theta, _kept(inv_freq)
        return ftk.qk_mrope_fwd(q, k, pos, axis_of, theta=theta, inv_freq=inv_freq)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        (pos,) = ctx.saved_tensors
        dq, dk = ftk.qk_mrope_bwd(dq.contiguous(), dk.contiguous(), pos, ctx.axis_of,
                                  theta=ctx.theta, inv_freq=ctx.inv_freq)
        return dq, dk, None, None, None, None


def _zeros(x):
    return torch.zeros(x.shape, dtype=x.dtype, device=x.device)


class Attention(torch.autograd.Function):
    """Attention inside every sequence of a packed batch (ftk.attn_fwd).  Tokens
    of no sequence (a batch padded past cu_seqlens[B]) get a zero output and
    zero gradients: where the sequences end is known on the device alone, so
    every result starts as zeros (ftk.attn_fwd and attn_bwd themselves leave such
    rows alone).  q, k and v of one projection are best taken with split along the
    heads: its backward joins the three gradients in one copy, that of three slices
    pads each to the projection's width and adds them.  Measured, bf16, 32/8 heads,
    direct calls, this, split, slices: forward 32,768 mixed tokens x 128 863 and 980
    us, 32,768 x 64 427 and 459; backward 3,040, 3,184, 3,459, 4,201 and 1,615,
    1,683, 1,818, 2,243."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale=None, causal: bool = True):
        o, lse = ftk.attn_fwd(q, k, v, cu_seqlens, scale=scale, causal=causal, o=_zeros(q))
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.scale, ctx.causal = scale, causal
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu = ctx.saved_tensors
        dq, dk, dv = ftk.attn_bwd(do.contiguous(), q, k, v, o, lse, cu, scale=ctx.scale,
                                  causal=ctx.causal, dq=_zeros(q), dk=_zeros(k), dv=_zeros(v))
        return dq, dk, dv, None, None, None


class CrossEntropyHead(torch.autograd.Function):
    """Mean cross-entropy of the logits h W^T against y (int32; y outside
    [0, V) is ignored), the logits never materialised."""

    @staticmethod
    def forward(ctx, h, W, y):
        loss, lse = ftk.cce_fwd(h, W, y)
        ctx.save_for_backward(h, W, y, lse)
        return loss.reshape(())

    @staticmethod
    def backward(ctx, dloss):
        h, W, y, lse = ctx.saved_tensors
        g = dloss.reshape(1).to(torch.float32).contiguous()
        dh, dW = ftk.cce_bwd(h, W, y, lse, g)
        return dh, dW.to(W.dtype), None


def rmsnorm(x, w, eps: float):
    return RMSNorm.apply(x, w, eps)


def add_rmsnorm(x, res, w, eps: float):
    return AddRMSNorm.apply(x, res, w, eps)


def swiglu(g, u):
    return SwiGLU.apply(g, u)


def qk_rope(q, k, cu_seqlens, theta: float, inv_freq=None):
    return QKRope.apply(q, k, cu_seqlens, theta, inv_freq)


def qk_norm_rope(q, k, wq, wk, cu_seqlens, eps: float, theta: float, inv_freq=None):
    return QKNormRope.apply(q, k, wq, wk, cu_seqlens, eps, theta, inv_freq)


def qk_mrope(q, k, pos, axis_of, theta: float, inv_freq=None):
    return QKMrope.apply(q, k, pos, axis_of, theta, inv_freq)


def attention(q, k, v, cu_seqlens, scale=None, causal: bool = True):
    return Attention.apply(q, k, v, cu_seqlens, scale, causal)


def cross_entropy_head(h, W, y):
    return CrossEntropyHead.apply(h, W, y)


def _is_lora_b(name: str) -> bool:
    parts = name.replace("/", ".").split(".")
    return any(p in ("lora_B", "lora_b", "B") for p in parts[-3:]) or name.endswith("lora_B")


def lora_plus_param_groups(named_parameters: Iterable[Tuple[str, torch.nn.Parameter]],
                           lr: float, ratio: float = LORA_PLUS_RATIO,
                           weight_decay: Optional[float] = None) -> List[dict]:
    """Parameter groups for the LoRA+ rule: every LoRA B matrix (a parameter
    whose dotted name has a ``lora_B`` (or ``B``) component) at lr * ratio,
    everything else trainable (the A matrices, biases, ...) at lr.  Frozen
    parameters are left out.  Pass the result to any torch optimizer."""
    a_params, b_params = [], []
    for name, p in named_parameters:
        if not p.requires_grad:
            continue
        (b_params if _is_lora_b(name) else a_params).append(p)
    groups = []
    extra = {} if weight_decay is None else {"weight_decay": weight_decay}
    if a_params:
        groups.append({"params": a_params, "lr": lr, **extra})
    if b_params:
        groups.append({"params": b_params, "lr": lr * ratio, **extra})
    return groups
