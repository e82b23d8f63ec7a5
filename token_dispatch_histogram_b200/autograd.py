"""Autograd functions for the path and the model around it (training).

The MoonEP page has the dispatched rows written straight into a static
communication buffer ("Online planning, zero copy και στατικά σχήματα"), which
the next dispatch or combine overwrites, so autograd must not keep such views
for the backward pass ("Ένα ρεαλιστικό πλαίσιο αξιολόγησης πριν από την
υιοθέτηση").  So:

- ep_dispatch_fn saves only the layout (pos); its backward is the unpermute,
  ep_dispatch_backward: dx[t] = sum_k dbuf[pos[t*K+k]] (fp32, one rounding).
- ep_combine_fn needs the expert rows y for the gate-weight gradient, so it
  saves y: the caller must keep y unchanged until the backward runs (a buffer
  per layer, or a copy).  Backward: ep_combine_backward, dy[pos[t*K+k]] =
  w[t,k] * dout[t] and dw[t,k] = <dout[t], y[pos[t*K+k]]>.
- ep_router_fn: router logits to (w, topk_ids); the backward gives dlogits from
  combine's dw.
- ep_experts_fn: dispatched rows through a layer's experts; the backward gives
  the rows' gradient and leaves the weights' in the layer's g_home and g_rep, in
  fp32, where grad_reduce and an optimizer take them (the weights are no leaves of
  the graph).  So its backward has to run wherever the layer holds such rows:
  then its result requires a gradient even if the rows do not (a frozen trunk
  under trained experts), and backward() reaches it.  It saves the rows and the
  plan's slots by reference: both must stay as they are until the backward (a
  buffer and a layer of their own, not the next step's).

The gradients of ep_router_fn and ep_experts_fn have no graph of their own: one
that would need it (create_graph) is refused.

Every step runs in libep.so's kernels; these classes only allocate outputs and
route tensors.
"""
import torch
from torch.autograd.function import once_differentiable

from . import (ep_combine, ep_combine_backward, ep_dispatch, ep_dispatch_backward, ep_expert_gemm, ep_expert_up,
               ep_router, ep_router_backward)


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, pos, K, buf):
        ep_dispatch(x, K, pos, buf)
        ctx.save_for_backward(pos)
        ctx.K, ctx.T = K, x.shape[0]
        ctx.mark_dirty(buf)
        return buf

    @staticmethod
    def backward(ctx, dbuf):
        (pos,) = ctx.saved_tensors
        dx = torch.empty((ctx.T, dbuf.shape[1]), dtype=dbuf.dtype, device=dbuf.device)
        ep_dispatch_backward(dbuf.contiguous(), pos, ctx.T, ctx.K, dx)
        return dx, None, None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, w, pos):
        T = w.shape[0]
        out = torch.empty((T, y.shape[1]), dtype=y.dtype, device=y.device)
        ep_combine(y, w, pos, out)
        ctx.save_for_backward(y, w, pos)
        return out

    @staticmethod
    def backward(ctx, dout):
        y, w, pos = ctx.saved_tensors
        dy = torch.zeros_like(y)  # rows no pair addresses get no gradient
        dw = torch.empty_like(w)
        ep_combine_backward(dout.contiguous(), w, y, pos, dy, dw)
        return dy, dw, None


class _Router(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, K, kw, dev_status):
        T = logits.shape[0]
        ids = torch.empty((T, K), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, K), dtype=torch.float32, device=logits.device)
        ep_router(logits, ids, w, dev_status=dev_status, **kw)
        ctx.save_for_backward(logits, ids)
        ctx.kw = {k: kw[k] for k in ("score", "renorm", "scale") if k in kw}
        ctx.mark_non_differentiable(ids)
        return w, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, dw, _):
        logits, ids = ctx.saved_tensors
        dlogits = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        ep_router_backward(dw.contiguous(), logits, ids, dlogits, **ctx.kw)
        return dlogits, None, None, None


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, w13, w2, layer, accumulate, anchor):
        P, I = rows.shape[0], w2.shape[2]
        like = dict(dtype=torch.bfloat16, device=rows.device)
        h, gu, y = torch.empty((P, I), **like), torch.empty((P, 2 * I), **like), torch.empty(rows.shape, **like)
        kw = dict(dev_status=layer.dev_status, **layer.slots())
        ep_expert_up(rows, w13, h=h, gu=gu, **kw)
        ep_expert_gemm(h, w2, y=y, **kw)
        ctx.save_for_backward(rows, w13, w2, gu)
        ctx.layer, ctx.accumulate = layer, accumulate
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, w13, w2, gu = ctx.saved_tensors
        dgu = torch.empty_like(gu)
        h = torch.empty((gu.shape[0], gu.shape[1] // 2), dtype=gu.dtype, device=gu.device)
        dx = torch.zeros_like(rows)  # rows of no slot get no gradient
        ctx.layer.experts_backward(dy.contiguous(), rows, w13, w2, gu, dgu, h, dx, ctx.accumulate)
        return dx, None, None, None, None, None


def ep_router_fn(logits, K, dev_status=None, **kw):
    """(w [T, K] fp32, topk_ids [T, K] int32) from router logits; kw as
    ep_router's.  The backward gives dlogits."""
    return _Router.apply(logits, K, kw, dev_status)


def ep_experts_fn(rows, w13, w2, layer, accumulate=False):
    """y = the rows [P, H] of a layer's dispatch through its experts (w13
    [E, 2I, H], w2 [E, H, I], over the layer's current plan).  The backward gives
    drows, and the weights' gradients into layer.g_home (added to what is there
    if accumulate) and layer.g_rep, which layer.grad_reduce() takes after each
    backward.  If the layer has those (grad_n = 3*H*I), y
    requires a gradient whether rows do or not; torch.autograd.grad() towards
    inputs that rows do not depend on leaves the weights' gradients out."""
    # a leaf that nobody sees makes autograd run the backward for the weights alone
    trained = torch.is_grad_enabled() and layer.grad_n == 3 * layer.H * w2.shape[2]
    anchor = torch.empty(0, device=rows.device, requires_grad=True) if trained else None
    return _Experts.apply(rows, w13, w2, layer, accumulate, anchor)


def ep_dispatch_fn(x, pos, K, buf):
    """buf[pos[p]] = x[p // K] into the static buffer buf (returned); the
    backward gives dx.  buf is overwritten in place and must not be kept."""
    return _Dispatch.apply(x, pos, K, buf)


def ep_combine_fn(y, w, pos):
    """out[t] = sum_k w[t,k] * y[pos[t*K+k]]; the backward gives dy and dw.
    y is saved for the backward and must stay unchanged until then."""
    return _Combine.apply(y, w, pos)
