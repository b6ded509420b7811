"""The operators around the chunk core (include/carve.h): the gated linear
scan, the norms of q and k with the position rotation, and the short causal
convolution.

Reached as ``carve.scan_fwd`` and so on.  The calls themselves are in the
compiled binding (csrc/mixer/binding.cpp, built into _mixer.so): CUDA tensors
in, the library's kernels enqueued on torch's current stream of the tensors'
device (which need not be the current device), no CPU fallback.  Token inputs
may be slices of a wider contiguous tensor (the channels of a token
contiguous, tokens evenly spaced); everything else is contiguous.  Outputs
that a call allocates are zero in the rows of a packed batch that belong to no
sequence; outputs that the caller passes keep theirs, and must not overlap what
the call reads.  Here are the autograd wrappers.

To capture a training step into a CUDA graph, capture the ``_fwd`` and ``_bwd``
calls: capturing ``backward()`` while an eager graph of the same leaves lives
can end the process inside torch.

A packed call with bad offsets writes no output: what it returns is memory as it
was allocated.  No call reads the status word back, which would wait for the
GPU; the wrappers hand on a workspace, whose word ``carve.get_status`` reads:

    ws = carve.scan_workspace(x, cu_seqlens)
    h, h_T = carve.scan(x, g, cu_seqlens=cu_seqlens, workspace=ws)
    y, state_T = carve.conv(x, w, cu_seqlens=cu_seqlens, workspace=ws2)  # 256 bytes
    carve.get_status(ws)
"""
import ctypes

import torch
from torch.autograd.function import once_differentiable


def _load():
    try:
        from . import _mixer
    except ImportError as e:
        raise RuntimeError(
            "the binding _mixer.so is not built or does not load (%s); run "
            "`python -m chunk_gated_delta_02_b200.build`" % e) from e
    return _mixer


def _late(name):
    # an entry point of a binding that was not built yet when this module was
    # imported
    def call(*args, **kwargs):
        return getattr(_load(), name)(*args, **kwargs)
    call.__name__ = name
    return call


try:
    from ._mixer import (
        conv_bwd, conv_fwd, conv_step, qk_rope_bwd, qk_rope_fwd, scan_bwd,
        scan_fwd, scan_step)
except ImportError:
    conv_bwd, conv_fwd, conv_step = map(_late, ("conv_bwd", "conv_fwd", "conv_step"))
    qk_rope_bwd, qk_rope_fwd = map(_late, ("qk_rope_bwd", "qk_rope_fwd"))
    scan_bwd, scan_fwd, scan_step = map(_late, ("scan_bwd", "scan_fwd", "scan_step"))


class ScanFunction(torch.autograd.Function):
    """Autograd wrapper of scan_fwd / scan_bwd (see scan)."""

    @staticmethod
    def forward(ctx, x, g, h0, cu_seqlens, decay_scale, complement, workspace):
        ctx.set_materialize_grads(False)
        train = any(ctx.needs_input_grad)
        h, h_T, ws = scan_fwd(x, g, h0, cu_seqlens, training=train,
                              workspace=workspace, decay_scale=decay_scale,
                              complement=complement)
        if train:
            ctx.save_for_backward(x, g, cu_seqlens, ws)
            ctx.opt = dict(decay_scale=decay_scale, complement=complement)
        return h, h_T

    @staticmethod
    @once_differentiable
    def backward(ctx, d_h, dh_T):
        x, g, cu_seqlens, ws = ctx.saved_tensors
        d_h = (torch.zeros(x.shape, dtype=x.dtype, device=x.device)
               if d_h is None else d_h.contiguous())
        gr = scan_bwd(x, g, d_h, ws, None if dh_T is None else
                      dh_T.contiguous(), cu_seqlens,
                      want_dh0=ctx.needs_input_grad[2], **ctx.opt)
        return gr["dx"], gr["dg"], gr["dh0"], None, None, None, None


def scan(x, g, h0=None, cu_seqlens=None, decay_scale=0.0, complement=False,
         workspace=None):
    """Differentiable gated linear scan; returns (h, h_T) (see scan_fwd).  The
    backward pass reads a workspace (scan_workspace) that is given: keep it for
    this call until then."""
    return ScanFunction.apply(x, g, h0, cu_seqlens, decay_scale, complement,
                              workspace)


def scan_workspace(x, cu_seqlens=None, training=True):
    """A workspace (uint8) for a scan over x: scan_fwd and scan take it, and its
    status word can be read afterwards."""
    from . import carve
    lead = 2 if cu_seqlens is None else 1
    shape = carve.ScanShape(
        B=x.shape[0] if lead == 2 else cu_seqlens.numel() - 1,
        T=x.shape[lead - 1], C=x.shape[lead:].numel(),
        dtype=carve.CARVE_BF16 if x.dtype == torch.bfloat16 else carve.CARVE_FP32)
    with torch.cuda.device(x.device):
        n = carve.lib().carve_scan_workspace_bytes(
            ctypes.byref(shape), int(lead == 1), int(bool(training)))
        if n == 0:
            raise carve.CarveError("carve_scan_workspace_bytes", 2)
        return torch.empty(n, dtype=torch.uint8, device=x.device)


def rope_freqs(dims, theta=10000.0, device="cuda"):
    """The usual rotation frequencies theta^(-2 i / dims), i < dims / 2, as
    the float64 tensor that qk_rope takes (radians per position)."""
    i = torch.arange(0, dims, 2, dtype=torch.float64)
    return (float(theta) ** (-i / max(dims, 1))).to(device)


class QkRopeFunction(torch.autograd.Function):
    """Autograd wrapper of qk_rope_fwd / qk_rope_bwd (see qk_rope)."""

    @staticmethod
    def forward(ctx, q, k, pos, freqs, w_q, w_k, eps, l2norm, interleaved):
        ctx.opt = dict(eps=eps, l2norm=l2norm, interleaved=interleaved)
        ctx.save_for_backward(q, k, pos, freqs, w_q, w_k)
        return qk_rope_fwd(q, k, pos, freqs, w_q, w_k, **ctx.opt)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, pos, freqs, w_q, w_k = ctx.saved_tensors
        gr = qk_rope_bwd(q, k, pos, freqs, dq_out.contiguous(),
                         None if k is None else dk_out.contiguous(), w_q, w_k,
                         **ctx.opt)
        return (gr["dq"], gr["dk"], None, None,
                None if w_q is None else gr["dw_q"].to(w_q.dtype),
                None if w_k is None else gr["dw_k"].to(w_k.dtype),
                None, None, None)


def qk_rope(q, k, pos, freqs, w_q=None, w_k=None, eps=1e-6, l2norm=False,
            interleaved=False):
    """Differentiable norms and rotation of q and k (see qk_rope_fwd)."""
    return QkRopeFunction.apply(q, k, pos, freqs, w_q, w_k, eps, l2norm,
                                interleaved)


class ConvFunction(torch.autograd.Function):
    """Autograd wrapper of conv_fwd / conv_bwd (see conv)."""

    @staticmethod
    def forward(ctx, x, w, bias, state, cu_seqlens, silu, workspace):
        ctx.set_materialize_grads(False)
        ctx.silu = silu
        ctx.save_for_backward(x, w, bias, state, cu_seqlens)
        return conv_fwd(x, w, bias, state, cu_seqlens, silu,
                        workspace=workspace)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dstate_T):
        x, w, bias, state, cu_seqlens = ctx.saved_tensors
        dy = (torch.zeros(x.shape, dtype=x.dtype, device=x.device)
              if dy is None else dy.contiguous())
        gr = conv_bwd(x, w, dy, bias, state, None if dstate_T is None else
                      dstate_T.contiguous(), cu_seqlens, ctx.silu)
        return (gr["dx"], gr["dw"].to(w.dtype),
                None if bias is None else gr["dbias"].to(bias.dtype),
                None if state is None else gr["dstate"], None, None, None)


def conv(x, w, bias=None, state=None, cu_seqlens=None, silu=False,
         workspace=None):
    """Differentiable short causal convolution; returns (y, state_T) (see
    conv_fwd, which the workspace goes to)."""
    return ConvFunction.apply(x, w, bias, state, cu_seqlens, silu, workspace)
