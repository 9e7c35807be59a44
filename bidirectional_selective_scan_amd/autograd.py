"""The recurrent block's operators as differentiable torch functions: forward and backward both run
the library's kernels (see ``block``). Gradients of gradients are not defined and raise."""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .block import GatedInputs, PreparedBlockNorm, PreparedBlockNormGrad, PreparedGated, PreparedGatedGrad


class _GatedRecurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, r, i, lam, h0, offsets, c, seg_len, reverse):
        inp = GatedInputs(x, r, i, lam, c, h0, seg_len, offsets, reverse)
        call = PreparedGated(inp, None, None, None, save_states=True)
        call()
        ctx.save_for_backward(x, r, i, lam, h0, offsets, call.states)
        ctx.scalars = (c, seg_len, reverse)
        ctx.set_materialize_grads(False)
        return call.y, call.h_last

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh_last):
        x, r, i, lam, h0, offsets, states = ctx.saved_tensors
        c, seg_len, reverse = ctx.scalars
        inp = GatedInputs(x, r, i, lam, c, h0, seg_len, offsets, reverse)
        dy = None if dy is None else dy.contiguous()
        dh_last = None if dh_last is None else dh_last.contiguous()
        g = PreparedGatedGrad(inp, dy, dh_last, states=states)
        g()
        return g.dx, g.dr, g.di, g.dlam, g.dh0, None, None, None, None


def gated_recurrence(x, r, i, lam, c: float = 8.0, h0=None, seg_len: int = 0, offsets=None, reverse: bool = False):
    """Differentiable (y, h_last) of the gated linear recurrence (arguments as ``PreparedGated``) in
    x, r, i, lam and h0."""
    return _GatedRecurrence.apply(x, r, i, lam, h0, offsets, float(c), int(seg_len), bool(reverse))


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, z, w_post, residual, gamma, w_pre, eps, gate_after, res_dtype):
        call = PreparedBlockNorm(x, z, w_post, residual, gamma, w_pre, eps, gate_after, res_dtype)
        call()
        ctx.save_for_backward(x, z, w_post, residual, gamma, w_pre)
        ctx.scalars = (eps, gate_after, res_dtype)
        ctx.set_materialize_grads(False)
        return call.sum, call.n

    @staticmethod
    @once_differentiable
    def backward(ctx, dsum, dn):
        x, z, w_post, residual, gamma, w_pre = ctx.saved_tensors
        eps, gate_after, res_dtype = ctx.scalars
        dsum = None if dsum is None else dsum.contiguous()
        dn = None if dn is None else dn.contiguous()
        g = PreparedBlockNormGrad(x, z, w_post, residual, gamma, w_pre, dsum, dn, eps, gate_after, res_dtype,
                                  weights=any(ctx.needs_input_grad[k] for k in (2, 4, 5)))
        g()
        return g.dx, g.dz, g.dw_post, g.dresidual, g.dgamma, g.dw_pre, None, None, None


def block_norm(x, z=None, w_post=None, residual=None, gamma=None, w_pre=None, eps: float = 1e-5,
               gate_after: bool = False, res_dtype=None):
    """Differentiable (sum, n) of the block norm (arguments as ``PreparedBlockNorm``; n is None without
    w_pre) in x, z, w_post, residual, gamma and w_pre."""
    return _BlockNorm.apply(x, z, w_post, residual, gamma, w_pre, float(eps), bool(gate_after), res_dtype)
