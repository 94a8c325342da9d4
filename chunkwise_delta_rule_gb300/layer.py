"""PyTorch-facing binding of the layer operators around the delta rule (same
names as include/kda.h): the short causal convolution, the selective state space
scan, linear attention with a decay for each head, the root-mean-square norm, and
products in 8 bits.

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


# ------------------------------------------------------------------ linear attention

class LinGrads(NamedTuple):
    """Gradients of a linear attention call; dh0 is None where it was not asked for."""

    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dh0: Optional[torch.Tensor]


def make_lin_problem(q, k, v, decay: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                     initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None) -> "_binding.LinProblem":
    """Describe one call of linear attention: q and k [B, T, H, K], v [B, T, HV, V]
    in one type (bf16 or fp32; HV a multiple of H, value head j reading key head
    j // (HV // H); widths up to 256), ``decay`` [HV] fp32, the natural logarithm
    of each head's factor per token, or None for no decay, ``scale`` of the
    queries (K ** -0.5 by default), ``initial_state`` [N, HV, K, V] fp32 or None.
    ``include/kda.h`` says which of a call's values are rounded to bf16 on the
    tensor cores, and what a NaN in a token reaches. Single tokens of decoding are
    a call of their own, [N, 1, ...]; packed beside prompts they take longer."""
    return _binding.LinProblem(q, k, v, decay, scale, initial_state, cu_seqlens)


def kda_lin_workspace_size(p: "_binding.LinProblem", for_backward: bool) -> int:
    return _binding.lin_workspace_size(p, for_backward)


def kda_lin_fwd(p: "_binding.LinProblem", *, output_final_state: bool = True, ht: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, err: Optional[torch.Tensor] = None, stream=None):
    """Returns (o [B, T, HV, V], final states [N, HV, K, V] fp32 or None). ``ht`` may
    be given, for example the initial state itself to update it in place; ``err``
    is an optional int32 device word (bit 0: inconsistent cu_seqlens, bit 1: a
    bounded wait inside the kernel gave up)."""
    return _binding.lin_fwd(p, output_final_state, ht, workspace, err, stream)


def kda_lin_bwd(p: "_binding.LinProblem", do: torch.Tensor, dht: Optional[torch.Tensor] = None, *,
                workspace: Optional[torch.Tensor] = None, stream=None, need_dh0: Optional[bool] = None,
                err: Optional[torch.Tensor] = None) -> LinGrads:
    """Backward of <do, o> + <dht, final states> (the decay has no gradient); dh0
    comes with an initial state, or as ``need_dh0`` says; ``err`` as in the
    forward."""
    return LinGrads(*_binding.lin_bwd(p, do, dht, workspace, stream, need_dh0, err))


# ------------------------------------------------------------------ 8 bits

class Quant8(NamedTuple):
    """8-bit values and scales; None where they were not asked for."""

    q: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    qt: Optional[torch.Tensor]
    scale_t: Optional[torch.Tensor]


def make_quant8_problem(x, *, blocks: bool = False, rows: bool = True, transposed: bool = False) -> "_binding.Quant8Problem":
    """Describe one rounding of x [..., D] (bf16 or fp32) to e4m3: with ``rows`` in
    its own order, q [..., D] with a scale for each row and 128 columns (with
    ``blocks`` for each 128 rows and 128 columns); with ``transposed`` (also) as
    qt [D, R] over the R rows of all leading axes, with a scale for each 128 of
    them (with ``blocks`` the same values and scales)."""
    return _binding.Quant8Problem(x, blocks, rows, transposed)


def kda_quant8(p: "_binding.Quant8Problem", *, stream=None) -> Quant8:
    """Returns (q, scale, qt, scale_t). Rows of q and qt start every 16 bytes: they
    are views of wider rows where their width is no multiple of 16."""
    return Quant8(*_binding.quant8(p, stream))


def make_mm8_problem(a, scale_a, b, scale_b, *, out: str = "bf16") -> "_binding.Mm8Problem":
    """Describe the product a b^T of e4m3 values with scales: a [..., K] and scale_a
    [..., ceil(K / 128)] as ``kda_norm_fwd`` (out "e4m3", group 128) or
    ``kda_quant8`` give them, b [N, K] with scale_b [ceil(N / 128), ceil(K / 128)]
    (blocks) or [N, ceil(K / 128)] (rows), all scales fp32; ``out`` "bf16" or
    "fp32"."""
    return _binding.Mm8Problem(a, scale_a, b, scale_b, out)


def kda_mm8_workspace_size(p: "_binding.Mm8Problem") -> int:
    return _binding.mm8_workspace_size(p)


def kda_mm8(p: "_binding.Mm8Problem", *, y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            err: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Returns y [..., N]; ``err`` is an optional int32 device word (bit 1: a bounded
    wait inside the kernel gave up)."""
    return _binding.mm8(p, y, workspace, err, stream)


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


class LinearAttentionFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the CUDA library."""

    @staticmethod
    def forward(ctx, q, k, v, decay, scale, initial_state, cu_seqlens, err):
        p = make_lin_problem(q, k, v, decay, scale=scale, initial_state=initial_state, cu_seqlens=cu_seqlens)
        o, ht = kda_lin_fwd(p, err=err)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, decay, initial_state, cu_seqlens)
        ctx.meta = (scale, err)
        return o, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, do, dht):
        q, k, v, decay, h0, cu = ctx.saved_tensors
        if ctx.needs_input_grad[3]:
            raise RuntimeError("the decay has no gradient: it is a constant of the layer")
        p = make_lin_problem(q, k, v, decay, scale=ctx.meta[0], initial_state=h0, cu_seqlens=cu)
        g = kda_lin_bwd(p, _grad(do, v.shape, v), _grad(dht), err=ctx.meta[1])
        return g.dq, g.dk, g.dv, None, None, g.dh0, None, None


def linear_attention(q, k, v, decay: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                     initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     err: Optional[torch.Tensor] = None):
    """Differentiable linear attention with a decay for each head (a constant).
    Returns (o, final_state). ``err`` as in ``kda_lin_fwd``; its backward sets it
    too."""
    return LinearAttentionFunction.apply(q, k, v, decay, scale, initial_state, cu_seqlens, err)


class Linear8Function(torch.autograd.Function):
    """Autograd wrapper: the three products run in 8 bits."""

    @staticmethod
    def forward(ctx, x, weight, err, recorded):
        out = "bf16" if x.dtype == torch.bfloat16 else "fp32"
        a = kda_quant8(make_quant8_problem(x, transposed=recorded and ctx.needs_input_grad[1]))
        w = kda_quant8(make_quant8_problem(weight, blocks=True, transposed=recorded and ctx.needs_input_grad[0]))
        y = kda_mm8(make_mm8_problem(a.q, a.scale, w.q, w.scale, out=out), err=err)
        ctx.save_for_backward(a.qt, a.scale_t, w.qt, w.scale_t)
        ctx.meta = (out, weight.dtype, err)
        ctx.shape = weight.shape
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        xt, xt_scale, wt, wt_scale = ctx.saved_tensors
        out, wtype, err = ctx.meta
        need_x, need_w = ctx.needs_input_grad[:2]
        if dy.numel() == 0:   # no tokens: nothing to sum over
            dx = dy.new_zeros(dy.shape[:-1] + ctx.shape[1:]) if need_x else None
            return dx, dy.new_zeros(ctx.shape, dtype=wtype) if need_w else None, None, None
        d = kda_quant8(make_quant8_problem(dy.contiguous(), rows=need_x, transposed=need_w))
        dx = kda_mm8(make_mm8_problem(d.q, d.scale, wt, wt_scale, out=out), err=err) if need_x else None
        dw = None
        if need_w:
            wout = "bf16" if wtype == torch.bfloat16 else "fp32"
            dw = kda_mm8(make_mm8_problem(d.qt, d.scale_t, xt, xt_scale, out=wout), err=err)
        return dx, dw, None, None


def linear8(x, weight, *, err: Optional[torch.Tensor] = None):
    """Differentiable product x weight^T in 8 bits: x [..., K] and weight [N, K]
    (bf16 or fp32) are rounded to e4m3, x by rows and groups of 128 columns, weight
    by blocks of 128 x 128; the backward rounds the output's gradient by rows for
    x's gradient and by groups of 128 tokens, as x, for the weight's. The roundings
    pass their gradients through. y and dx come in x's type, the weight's gradient
    in its own. ``err`` as in ``kda_mm8``. The weight is rounded in every call:
    serving rounds it once with ``kda_quant8`` and calls ``kda_mm8``."""
    # (needs_input_grad says what the tensors ask for, not whether the call is recorded)
    return Linear8Function.apply(x, weight, err, torch.is_grad_enabled())
