"""PyTorch-facing binding of the layer operators around the delta rule (same
names as include/kda.h): the short causal convolution, the selective state space
scan and the root-mean-square norm.

As in ``ops``: PyTorch provides device memory and the current stream, every step
runs in libkda.so's CUDA kernels. Token tensors are [B, T, ...]; inputs may be
slices of wider rows (the last axis dense, tokens evenly spaced), outputs are
contiguous. All tensors of a call lie on one device. A call with ``stream`` allocates
and runs on it; that its inputs are ready there, and its outputs where they are
used, is the caller's to order, as everywhere in PyTorch. Parameters and scan states
are fp32. The argument checks and the
calls are compiled (``csrc/binding.cpp``): a decoding step is short, and in
Python they would take longer than it.
"""

from __future__ import annotations

from typing import NamedTuple, Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib


class _Unloaded:
    """Stands for the compiled binding until its first use (the package is
    imported to build it); fails loudly if it has not been built."""

    def __getattr__(self, name):
        global _binding
        _lib.load()
        try:
            from . import _binding as module
        except ImportError as e:
            raise ImportError("_binding.so is not built for this torch (run `python -m chunkwise_delta_rule_gb300.build`); "
                              "the layer operators have no other entry from Python") from e
        _binding = module
        return getattr(module, name)


_binding = _Unloaded()


# ------------------------------------------------------------------ convolution

def make_conv_problem(x, weight, bias=None, *, silu: bool = True, initial_state: Optional[torch.Tensor] = None,
                      cu_seqlens: Optional[torch.Tensor] = None) -> "_binding.ConvProblem":
    """Describe one call of the short causal convolution: x [B, T, D] (bf16 or
    fp32), weight [D, W] fp32 with W = 2, 3 or 4, bias [D] fp32 or None,
    ``initial_state`` [N, W - 1, D] in x's type (each sequence's previous inputs,
    oldest first) or None."""
    return _binding.ConvProblem(x, weight, bias, silu, initial_state, cu_seqlens)


def kda_conv_workspace_size(p: "_binding.ConvProblem") -> int:
    return _binding.conv_workspace_size(p)


def kda_conv_fwd(p: "_binding.ConvProblem", *, output_final_state: bool = True, final_state: Optional[torch.Tensor] = None,
                 err: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, final state or None). ``final_state`` may be given, for example
    the initial state itself to update it in place; ``err`` is an optional int32
    device word (bit 0: inconsistent cu_seqlens)."""
    return _binding.conv_fwd(p, output_final_state, final_state, err, stream)


def kda_conv_bwd(p: "_binding.ConvProblem", dy: torch.Tensor, dfinal: Optional[torch.Tensor] = None, *,
                 workspace: Optional[torch.Tensor] = None, stream=None, need_dinit: Optional[bool] = None):
    """Backward of <dy, y> + <dfinal, final state>: (dx, dweight, dbias, dinit);
    dbias is None without a bias, dinit without an initial state (or with
    ``need_dinit`` False)."""
    return _binding.conv_bwd(p, dy, dfinal, workspace, stream, need_dinit)


# ------------------------------------------------------------------ scan

class SsmGrads(NamedTuple):
    """Gradients of a scan call; None where the input is absent."""

    dx: torch.Tensor
    ddt: torch.Tensor
    dA_log: torch.Tensor
    db: torch.Tensor
    dc: torch.Tensor
    dd_skip: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dh0: Optional[torch.Tensor]


def make_ssm_problem(x, dt, A_log, b, c, *, d_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                     dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
                     initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     save_policy: int = 0) -> "_binding.SsmProblem":
    """Describe one call of the selective state space scan: x, dt and the optional
    gate z [B, T, D], b and c [B, T, G, S] in one type (bf16 or fp32); A_log
    [D, S], d_skip and dt_bias [D], ``initial_state`` [N, D, S] in fp32. With
    ``save_policy`` 1 the forward keeps every 16th state for the backward."""
    return _binding.SsmProblem(x, dt, A_log, b, c, d_skip, z, dt_bias, dt_softplus, initial_state, cu_seqlens, save_policy)


def kda_ssm_workspace_size(p: "_binding.SsmProblem", for_backward: bool) -> int:
    return _binding.ssm_workspace_size(p, for_backward)


def kda_ssm_saved_size(p: "_binding.SsmProblem") -> int:
    return _binding.ssm_saved_size(p)


def kda_ssm_fwd(p: "_binding.SsmProblem", *, output_final_state: bool = True, ht: Optional[torch.Tensor] = None,
                saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, final states or None, saved or None). ``ht`` may be given, for
    example the initial state itself to update it in place; ``err`` is an optional
    int32 device word (bit 0: inconsistent cu_seqlens, bit 1: a bounded wait inside
    the kernel gave up)."""
    return _binding.ssm_fwd(p, output_final_state, ht, saved, workspace, err, stream)


def kda_ssm_bwd(p: "_binding.SsmProblem", dy: torch.Tensor, dht: Optional[torch.Tensor] = None, *,
                saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                need_dh0: Optional[bool] = None, err: Optional[torch.Tensor] = None) -> SsmGrads:
    """Backward of <dy, y> + <dht, final states>. With save_policy 1, ``saved`` is
    what the forward returned for the same inputs; ``err`` as in the forward."""
    return SsmGrads(*_binding.ssm_bwd(p, dy, dht, saved, workspace, stream, need_dh0, err))


# ------------------------------------------------------------------ norm

def make_norm_problem(x, weight, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6, out: str = "io",
                      group: int = 0) -> "_binding.NormProblem":
    """Describe one call of the root-mean-square norm over the last axis of x
    (contiguous, bf16 or fp32, up to 16384 wide) with weight [D] fp32, after
    adding ``residual`` (x's shape and type) if given. ``out``: "io" for x's type,
    "e4m3" for 8-bit values with one fp32 scale per ``group`` columns (32, 64,
    128, or 0 for the row)."""
    return _binding.NormProblem(x, weight, residual, eps, out, group)


def kda_norm_workspace_size(p: "_binding.NormProblem") -> int:
    return _binding.norm_workspace_size(p)


def kda_norm_fwd(p: "_binding.NormProblem", *, h: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, scale or None, h): y in x's type, or torch.float8_e4m3fn with
    scale [..., groups]; h is the sum with the residual in x's type (x itself
    without one). ``h`` may be given, for example the residual's own buffer."""
    return _binding.norm_fwd(p, h, stream)


def kda_norm_bwd(p: "_binding.NormProblem", dy: torch.Tensor, dres: Optional[torch.Tensor] = None, *,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward at x = the stored sum: (dx, dweight). ``dres`` is the gradient that
    reaches the sum past the norm; dx is the gradient of x and of the residual."""
    return _binding.norm_bwd(p, dy, dres, workspace, stream)


# ------------------------------------------------------------------ autograd

def _grad(t: Optional[torch.Tensor], shape=None, like: Optional[torch.Tensor] = None):
    """An output's gradient, dense; zeros of `shape` (None without one) where the output was not used."""
    if t is not None:
        return t.contiguous()
    return None if shape is None else torch.zeros(shape, dtype=like.dtype, device=like.device)


class ShortConvFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the CUDA library."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, silu, err):
        p = make_conv_problem(x, weight, bias, silu=silu, initial_state=initial_state, cu_seqlens=cu_seqlens)
        y, final = kda_conv_fwd(p, err=err)
        ctx.set_materialize_grads(False)   # an output nobody used has no gradient to read
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu = silu
        return y, final

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfinal):
        x, weight, bias, h0, cu = ctx.saved_tensors
        p = make_conv_problem(x, weight, bias, silu=ctx.silu, initial_state=h0, cu_seqlens=cu)
        dx, dw, db, dinit = kda_conv_bwd(p, _grad(dy, x.shape, x), _grad(dfinal))
        return dx, dw, db, dinit, None, None, None


def short_conv(x, weight, bias=None, *, silu: bool = True, initial_state: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None):
    """Differentiable short causal convolution. Returns (y, final_state). ``err``
    as in ``kda_conv_fwd``."""
    return ShortConvFunction.apply(x, weight, bias, initial_state, cu_seqlens, silu, err)


class SsmScanFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the CUDA library."""

    @staticmethod
    def forward(ctx, x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, dt_softplus, save_policy,
                err):
        p = make_ssm_problem(x, dt, A_log, b, c, d_skip=d_skip, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus,
                             initial_state=initial_state, cu_seqlens=cu_seqlens, save_policy=save_policy)
        y, ht, saved = kda_ssm_fwd(p, err=err)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, saved)
        ctx.meta = (dt_softplus, save_policy, err)
        return y, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dht):
        x, dt, A_log, b, c, d_skip, z, dt_bias, h0, cu, saved = ctx.saved_tensors
        p = make_ssm_problem(x, dt, A_log, b, c, d_skip=d_skip, z=z, dt_bias=dt_bias, dt_softplus=ctx.meta[0],
                             initial_state=h0, cu_seqlens=cu, save_policy=ctx.meta[1])
        g = kda_ssm_bwd(p, _grad(dy, x.shape, x), _grad(dht), saved=saved, err=ctx.meta[2])
        return (g.dx, g.ddt, g.dA_log, g.db, g.dc, g.dd_skip, g.dz, g.ddt_bias, g.dh0) + (None,) * 4


def ssm_scan(x, dt, A_log, b, c, *, d_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
             initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
             save_policy: int = 1, err: Optional[torch.Tensor] = None):
    """Differentiable selective state space scan. Returns (y, final_state). ``err``
    as in ``kda_ssm_fwd``; its backward sets it too."""
    return SsmScanFunction.apply(x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, dt_softplus,
                                 save_policy, err)


class RmsNormFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the CUDA library."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, _, h = kda_norm_fwd(make_norm_problem(x, weight, residual=residual, eps=eps))
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(h, weight)
        ctx.meta = (eps, residual is not None)
        return y, h if residual is not None else x.view_as(x)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        eps, has_residual = ctx.meta
        dx, dw = kda_norm_bwd(make_norm_problem(h, weight, eps=eps), _grad(dy, h.shape, h), _grad(dh))
        return dx, dw, dx if has_residual else None, None


def rms_norm(x, weight, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """Differentiable root-mean-square norm of x + residual. Returns (y, the sum):
    the sum is the residual stream that goes on."""
    return RmsNormFunction.apply(x, weight, residual, eps)
