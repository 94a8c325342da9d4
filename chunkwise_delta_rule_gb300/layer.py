"""PyTorch-facing binding of the layer operators around the delta rule (same
names as include/kda.h): the short causal convolution, the selective state space
scan and the root-mean-square norm.

As in ``ops``: PyTorch provides device memory and the current stream, every step
runs in libkda.so's CUDA kernels. Token tensors are [B, T, ...]; inputs may be
slices of wider rows (the last axis dense, tokens evenly spaced), outputs are
contiguous. Parameters and scan states are fp32.
"""

from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple, Optional

import torch

from . import _lib
from .ops import _buffer, _need, _stream

_IO = {torch.bfloat16: 0, torch.float32: 1}   # kda_dtype


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape, dtype) -> int:
    """Checks a [B, T, ...] input and returns the elements between its tokens."""
    _need(t.dtype == dtype and t.is_cuda and tuple(t.shape) == shape, f"{name} must be a CUDA tensor {list(shape)}, {dtype}")
    if t.is_contiguous():
        return 0
    st = t.stride()
    width = 1
    for size, step in zip(reversed(shape[2:]), reversed(st[2:])):
        _need(size == 1 or step == width, f"{name}'s rows must be dense")
        width *= size
    B, T = shape[:2]
    ld = st[1] if T > 1 else st[0] if B > 1 else width
    _need(ld >= width and (B == 1 or T == 1 or st[0] == T * ld), f"{name}'s tokens must be evenly spaced")
    return ld


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype):
    _need(t is None or (t.dtype == dtype and t.is_cuda and t.is_contiguous() and tuple(t.shape) == shape),
          f"{name} must be a contiguous CUDA tensor {list(shape)}, {dtype}")


def _axis(cu_seqlens, B):
    if cu_seqlens is None:
        return B, 0, None
    _need(cu_seqlens.dtype == torch.int32 and cu_seqlens.is_cuda and cu_seqlens.dim() == 1
          and cu_seqlens.is_contiguous() and cu_seqlens.numel() >= 2, "cu_seqlens must be an int32 CUDA vector")
    _need(B == 1, "packed sequences need B == 1")
    n = cu_seqlens.numel() - 1
    return n, n, cu_seqlens.data_ptr()


def _error_word(err):
    _need(err is None or (err.dtype == torch.int32 and err.is_cuda and err.numel() >= 1), "err must be an int32 CUDA tensor")


# ------------------------------------------------------------------ convolution

@dataclass
class ConvProblem:
    """A validated convolution call plus the tensors it points to."""

    c: _lib.ConvProblem
    x: torch.Tensor
    weight: torch.Tensor
    bias: Optional[torch.Tensor]
    h0: Optional[torch.Tensor]
    cu_seqlens: Optional[torch.Tensor]
    state_shape: tuple


def make_conv_problem(x, weight, bias=None, *, silu: bool = True, initial_state: Optional[torch.Tensor] = None,
                      cu_seqlens: Optional[torch.Tensor] = None) -> ConvProblem:
    """Describe one call of the short causal convolution: x [B, T, D] (bf16 or
    fp32), weight [D, W] fp32 with W = 2, 3 or 4, bias [D] fp32 or None,
    ``initial_state`` [N, W - 1, D] in x's type (each sequence's previous inputs,
    oldest first) or None."""
    _need(x.dim() == 3 and x.dtype in _IO, "x must be [B, T, D], bf16 or fp32")
    B, T, D = x.shape
    _need(weight.dim() == 2, "weight must be [D, W]")
    W = weight.shape[1]
    ldx = _rows(x, "x", (B, T, D), x.dtype)
    _dense(weight, "weight", (D, W), torch.float32)
    _dense(bias, "bias", (D,), torch.float32)
    n, packed, cu = _axis(cu_seqlens, B)
    shape = (n, W - 1, D)
    _dense(initial_state, "initial_state", shape, x.dtype)
    c = _lib.ConvProblem(B, T, D, W, packed, cu, _IO[x.dtype], 1 if silu else 0, ldx, x.data_ptr(), weight.data_ptr(),
                         _addr(bias), _addr(initial_state))
    return ConvProblem(c, x, weight, bias, initial_state, cu_seqlens, shape)


def kda_conv_workspace_size(p: ConvProblem) -> int:
    return int(_lib.load().kda_conv_workspace_size(ctypes.byref(p.c)))


def kda_conv_fwd(p: ConvProblem, *, output_final_state: bool = True, final_state: Optional[torch.Tensor] = None,
                 err: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, final state or None). ``final_state`` may be given, for example
    the initial state itself to update it in place."""
    x = p.x
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if final_state is not None:
        _dense(final_state, "final_state", p.state_shape, x.dtype)
    elif output_final_state:
        final_state = torch.empty(p.state_shape, dtype=x.dtype, device=x.device)
    _error_word(err)
    st = _lib.load().kda_conv_fwd(ctypes.byref(p.c), _addr(y), _addr(final_state), _addr(err), _stream(stream))
    _lib.check(st, "kda_conv_fwd")
    return y, final_state


def kda_conv_bwd(p: ConvProblem, dy: torch.Tensor, dfinal: Optional[torch.Tensor] = None, *,
                 workspace: Optional[torch.Tensor] = None, stream=None, need_dinit: Optional[bool] = None):
    """Backward of <dy, y> + <dfinal, final state>: (dx, dweight, dbias, dinit);
    dbias is None without a bias, dinit without an initial state (or with
    ``need_dinit`` False)."""
    x = p.x
    _dense(dy, "dy", tuple(x.shape), x.dtype)
    _dense(dfinal, "dfinal", p.state_shape, x.dtype)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(p.weight)
    db = None if p.bias is None else torch.empty_like(p.bias)
    dinit = None
    if need_dinit or (need_dinit is None and p.h0 is not None):
        dinit = torch.empty(p.state_shape, dtype=x.dtype, device=x.device)
    ws = _buffer(kda_conv_workspace_size(p), x.device, workspace)
    st = _lib.load().kda_conv_bwd(ctypes.byref(p.c), _addr(dy), _addr(dfinal), _addr(dx), _addr(dw), _addr(db),
                                  _addr(dinit), _addr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _lib.check(st, "kda_conv_bwd")
    return dx, dw, db, dinit


# ------------------------------------------------------------------ scan

@dataclass
class SsmProblem:
    """A validated scan call plus the tensors it points to."""

    c: _lib.SsmProblem
    x: torch.Tensor
    dt: torch.Tensor
    A_log: torch.Tensor
    b: torch.Tensor
    cm: torch.Tensor
    d_skip: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    dt_bias: Optional[torch.Tensor]
    h0: Optional[torch.Tensor]
    cu_seqlens: Optional[torch.Tensor]
    state_shape: tuple


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
                     save_policy: int = 0) -> SsmProblem:
    """Describe one call of the selective state space scan: x, dt and the optional
    gate z [B, T, D], b and c [B, T, G, S] in one type (bf16 or fp32); A_log
    [D, S], d_skip and dt_bias [D], ``initial_state`` [N, D, S] in fp32. With
    ``save_policy`` 1 the forward keeps every 16th state for the backward."""
    _need(x.dim() == 3 and x.dtype in _IO, "x must be [B, T, D], bf16 or fp32")
    B, T, D = x.shape
    _need(b.dim() == 4, "b must be [B, T, G, S]")
    G, S = b.shape[2:]
    dtype = x.dtype
    tok, bc = (B, T, D), (B, T, G, S)
    ldx, lddt = _rows(x, "x", tok, dtype), _rows(dt, "dt", tok, dtype)
    ldz = 0 if z is None else _rows(z, "z", tok, dtype)
    ldb, ldc = _rows(b, "b", bc, dtype), _rows(c, "c", bc, dtype)
    _dense(A_log, "A_log", (D, S), torch.float32)
    _dense(d_skip, "d_skip", (D,), torch.float32)
    _dense(dt_bias, "dt_bias", (D,), torch.float32)
    n, packed, cu = _axis(cu_seqlens, B)
    shape = (n, D, S)
    _dense(initial_state, "initial_state", shape, torch.float32)
    p = _lib.SsmProblem(B, T, D, S, G, packed, cu, _IO[dtype], 1 if dt_softplus else 0, int(save_policy), ldx, lddt,
                        ldz, ldb, ldc, x.data_ptr(), dt.data_ptr(), _addr(z), b.data_ptr(), c.data_ptr(),
                        A_log.data_ptr(), _addr(d_skip), _addr(dt_bias), _addr(initial_state))
    return SsmProblem(p, x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, shape)


def kda_ssm_workspace_size(p: SsmProblem, for_backward: bool) -> int:
    return int(_lib.load().kda_ssm_workspace_size(ctypes.byref(p.c), 1 if for_backward else 0))


def kda_ssm_saved_size(p: SsmProblem) -> int:
    return int(_lib.load().kda_ssm_saved_size(ctypes.byref(p.c)))


def kda_ssm_fwd(p: SsmProblem, *, output_final_state: bool = True, ht: Optional[torch.Tensor] = None,
                saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, final states or None, saved or None). ``ht`` may be given, for
    example the initial state itself to update it in place."""
    x = p.x
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if ht is not None:
        _dense(ht, "ht", p.state_shape, torch.float32)
    elif output_final_state:
        ht = torch.empty(p.state_shape, dtype=torch.float32, device=x.device)
    _error_word(err)
    ws = _buffer(kda_ssm_workspace_size(p, False), x.device, workspace)
    sv = _buffer(kda_ssm_saved_size(p), x.device, saved) if p.c.save_policy else None
    st = _lib.load().kda_ssm_fwd(ctypes.byref(p.c), _addr(y), _addr(ht), _addr(sv), _addr(ws),
                                 0 if ws is None else ws.numel() * ws.element_size(), _addr(err), _stream(stream))
    _lib.check(st, "kda_ssm_fwd")
    return y, ht, sv


def kda_ssm_bwd(p: SsmProblem, dy: torch.Tensor, dht: Optional[torch.Tensor] = None, *,
                saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                need_dh0: Optional[bool] = None) -> SsmGrads:
    """Backward of <dy, y> + <dht, final states>. With save_policy 1, ``saved`` is
    what the forward returned for the same inputs."""
    x, dev = p.x, p.x.device
    _dense(dy, "dy", tuple(x.shape), x.dtype)
    _dense(dht, "dht", p.state_shape, torch.float32)
    if p.c.save_policy:
        need = kda_ssm_saved_size(p)
        _need(need == 0 or (saved is not None and saved.numel() * saved.element_size() >= need),
              "save_policy 1 needs the forward's saved buffer")

    def like(t):
        return None if t is None else torch.empty(t.shape, dtype=t.dtype, device=dev)

    dh0 = None
    if need_dh0 or (need_dh0 is None and p.h0 is not None):
        dh0 = torch.empty(p.state_shape, dtype=torch.float32, device=dev)
    out = SsmGrads(like(x), like(p.dt), like(p.A_log), like(p.b), like(p.cm), like(p.d_skip), like(p.z),
                   like(p.dt_bias), dh0)
    g = _lib.SsmGrads(*(_addr(getattr(out, n)) for n, _ in _lib.SsmGrads._fields_))
    ws = _buffer(kda_ssm_workspace_size(p, True), dev, workspace)
    st = _lib.load().kda_ssm_bwd(ctypes.byref(p.c), _addr(dy), _addr(dht), _addr(saved if p.c.save_policy else None),
                                 ctypes.byref(g), _addr(ws), ws.numel() * ws.element_size(), _stream(stream))
    _lib.check(st, "kda_ssm_bwd")
    return out


# ------------------------------------------------------------------ norm

@dataclass
class NormProblem:
    """A validated norm call plus the tensors it points to."""

    c: _lib.NormProblem
    x: torch.Tensor
    weight: torch.Tensor
    residual: Optional[torch.Tensor]


def make_norm_problem(x, weight, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6, out: str = "io",
                      group: int = 0) -> NormProblem:
    """Describe one call of the root-mean-square norm over the last axis of x
    (contiguous, bf16 or fp32, up to 16384 wide) with weight [D] fp32, after
    adding ``residual`` (x's shape and type) if given. ``out``: "io" for x's type,
    "e4m3" for 8-bit values with one fp32 scale per ``group`` columns (32, 64,
    128, or 0 for the row)."""
    _need(x.dim() >= 1 and x.dtype in _IO, "x must be bf16 or fp32 rows")
    D = x.shape[-1]
    shape = tuple(x.shape)
    _dense(x, "x", shape, x.dtype)
    _dense(weight, "weight", (D,), torch.float32)
    _dense(residual, "residual", shape, x.dtype)
    _need(out in ("io", "e4m3"), 'out must be "io" or "e4m3"')
    c = _lib.NormProblem(x.numel() // D if D else 0, D, _IO[x.dtype], 0 if out == "io" else 1, int(group), float(eps),
                         x.data_ptr(), _addr(residual), weight.data_ptr())
    return NormProblem(c, x, weight, residual)


def kda_norm_workspace_size(p: NormProblem) -> int:
    return int(_lib.load().kda_norm_workspace_size(ctypes.byref(p.c)))


def kda_norm_fwd(p: NormProblem, *, h: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, scale or None, h): y in x's type, or torch.float8_e4m3fn with
    scale [..., groups]; h is the sum with the residual in x's type (x itself
    without one). ``h`` may be given, for example the residual's own buffer."""
    x = p.x
    dev, q8 = x.device, p.c.out == 1
    y = torch.empty(x.shape, dtype=torch.float8_e4m3fn if q8 else x.dtype, device=dev)
    scale = None
    if q8:
        D, group = p.c.D, p.c.group
        scale = torch.empty(x.shape[:-1] + ((D + group - 1) // group if group else 1,), dtype=torch.float32, device=dev)
    if p.residual is None:
        h = x
    elif h is None:
        h = torch.empty(x.shape, dtype=x.dtype, device=dev)
    else:
        _dense(h, "h", tuple(x.shape), x.dtype)
    st = _lib.load().kda_norm_fwd(ctypes.byref(p.c), _addr(y), _addr(scale), _addr(h), _stream(stream))
    _lib.check(st, "kda_norm_fwd")
    return y, scale, h


def kda_norm_bwd(p: NormProblem, dy: torch.Tensor, dres: Optional[torch.Tensor] = None, *,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward at x = the stored sum: (dx, dweight). ``dres`` is the gradient that
    reaches the sum past the norm; dx is the gradient of x and of the residual."""
    x = p.x
    _dense(dy, "dy", tuple(x.shape), x.dtype)
    _dense(dres, "dres", tuple(x.shape), x.dtype)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = torch.empty_like(p.weight)
    ws = _buffer(kda_norm_workspace_size(p), x.device, workspace)
    st = _lib.load().kda_norm_bwd(ctypes.byref(p.c), _addr(dy), _addr(dres), _addr(dx), _addr(dw), _addr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream))
    _lib.check(st, "kda_norm_bwd")
    return dx, dw


# ------------------------------------------------------------------ autograd

def _grad(t: Optional[torch.Tensor], shape=None, like: Optional[torch.Tensor] = None):
    """An output's gradient, dense; zeros of `shape` (None without one) where the output was not used."""
    if t is not None:
        return t.contiguous()
    return None if shape is None else torch.zeros(shape, dtype=like.dtype, device=like.device)


class ShortConvFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the CUDA library."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state, cu_seqlens, silu):
        p = make_conv_problem(x, weight, bias, silu=silu, initial_state=initial_state, cu_seqlens=cu_seqlens)
        y, final = kda_conv_fwd(p)
        ctx.set_materialize_grads(False)   # an output nobody used has no gradient to read
        ctx.save_for_backward(x, weight, bias, initial_state, cu_seqlens)
        ctx.silu = silu
        return y, final

    @staticmethod
    def backward(ctx, dy, dfinal):
        x, weight, bias, h0, cu = ctx.saved_tensors
        p = make_conv_problem(x, weight, bias, silu=ctx.silu, initial_state=h0, cu_seqlens=cu)
        dx, dw, db, dinit = kda_conv_bwd(p, _grad(dy, x.shape, x), _grad(dfinal))
        return dx, dw, db, dinit, None, None


def short_conv(x, weight, bias=None, *, silu: bool = True, initial_state: Optional[torch.Tensor] = None,
               cu_seqlens: Optional[torch.Tensor] = None):
    """Differentiable short causal convolution. Returns (y, final_state)."""
    return ShortConvFunction.apply(x, weight, bias, initial_state, cu_seqlens, silu)


class SsmScanFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run the CUDA library."""

    @staticmethod
    def forward(ctx, x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, dt_softplus, save_policy):
        p = make_ssm_problem(x, dt, A_log, b, c, d_skip=d_skip, z=z, dt_bias=dt_bias, dt_softplus=dt_softplus,
                             initial_state=initial_state, cu_seqlens=cu_seqlens, save_policy=save_policy)
        y, ht, saved = kda_ssm_fwd(p)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, saved)
        ctx.meta = (dt_softplus, save_policy)
        return y, ht

    @staticmethod
    def backward(ctx, dy, dht):
        x, dt, A_log, b, c, d_skip, z, dt_bias, h0, cu, saved = ctx.saved_tensors
        p = make_ssm_problem(x, dt, A_log, b, c, d_skip=d_skip, z=z, dt_bias=dt_bias, dt_softplus=ctx.meta[0],
                             initial_state=h0, cu_seqlens=cu, save_policy=ctx.meta[1])
        g = kda_ssm_bwd(p, _grad(dy, x.shape, x), _grad(dht), saved=saved)
        return g.dx, g.ddt, g.dA_log, g.db, g.dc, g.dd_skip, g.dz, g.ddt_bias, g.dh0, None, None, None


def ssm_scan(x, dt, A_log, b, c, *, d_skip: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = True,
             initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
             save_policy: int = 1):
    """Differentiable selective state space scan. Returns (y, final_state)."""
    return SsmScanFunction.apply(x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, dt_softplus,
                                 save_policy)


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
    def backward(ctx, dy, dh):
        h, weight = ctx.saved_tensors
        eps, has_residual = ctx.meta
        dx, dw = kda_norm_bwd(make_norm_problem(h, weight, eps=eps), _grad(dy, h.shape, h), _grad(dh))
        return dx, dw, dx if has_residual else None, None


def rms_norm(x, weight, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6):
    """Differentiable root-mean-square norm of x + residual. Returns (y, the sum):
    the sum is the residual stream that goes on."""
    return RmsNormFunction.apply(x, weight, residual, eps)
