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
from typing import NamedTuple, Optional

import torch

from . import _lib
from .ops import _buffer, _need

# A decoding step is a few microseconds on the device, so the checks here are kept to a few hundred nanoseconds per
# tensor: no message is formatted and no stream object made unless something is refused or asked for.

_IO = {torch.bfloat16: 0, torch.float32: 1}   # kda_dtype
_F32 = torch.float32
_byref = ctypes.byref
_empty = torch.empty
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream(stream, x: torch.Tensor) -> int:
    return _current_raw_stream(x.get_device()) if stream is None else stream.cuda_stream


def _refuse(name: str, what: str, shape, dtype):
    raise ValueError(f"{name} must be a {what}CUDA tensor {list(shape)}, {dtype}")


def _rows(t: torch.Tensor, name: str, shape, dtype) -> int:
    """Checks a [B, T, ...] input and returns the elements between its tokens (0: contiguous)."""
    if not (t.dtype is dtype and t.shape == shape and t.is_cuda):
        _refuse(name, "", shape, dtype)
    if t.is_contiguous():
        return 0
    st = t.stride()
    width = 1
    for size, step in zip(reversed(shape[2:]), reversed(st[2:])):
        if size != 1 and step != width:
            raise ValueError(f"{name}'s rows must be dense")
        width *= size
    B, T = shape[0], shape[1]
    ld = st[1] if T > 1 else st[0] if B > 1 else width
    if ld < width or (B > 1 and T > 1 and st[0] != T * ld):
        raise ValueError(f"{name}'s tokens must be evenly spaced")
    return ld


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype) -> Optional[int]:
    """Checks an optional contiguous tensor and returns its address."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous()):
        _refuse(name, "contiguous ", shape, dtype)
    return t.data_ptr()


def _axis(cu_seqlens, B):
    """(sequences, packed sequences, offsets' address)."""
    if cu_seqlens is None:
        return B, 0, None
    _need(cu_seqlens.dtype is torch.int32 and cu_seqlens.is_cuda and cu_seqlens.dim() == 1
          and cu_seqlens.is_contiguous() and cu_seqlens.numel() >= 2, "cu_seqlens must be an int32 CUDA vector")
    _need(B == 1, "packed sequences need B == 1")
    n = cu_seqlens.numel() - 1
    return n, n, cu_seqlens.data_ptr()


def _error_word(err) -> Optional[int]:
    if err is None:
        return None
    _need(err.dtype is torch.int32 and err.is_cuda and err.numel() >= 1, "err must be an int32 CUDA tensor")
    return err.data_ptr()


def _like(t: Optional[torch.Tensor]):
    return None if t is None else _empty(t.shape, dtype=t.dtype, device=t.device)


def _addr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _bytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


# ------------------------------------------------------------------ convolution

class ConvProblem(NamedTuple):
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
    dtype, shape = x.dtype, x.shape
    _need(len(shape) == 3 and dtype in _IO, "x must be [B, T, D], bf16 or fp32")
    _need(weight.dim() == 2, "weight must be [D, W]")
    B, T, D = shape
    W = weight.shape[1]
    ldx = _rows(x, "x", shape, dtype)
    n, packed, cu = _axis(cu_seqlens, B)
    state = (n, W - 1, D)
    c = _lib.ConvProblem(B, T, D, W, packed, cu, _IO[dtype], 1 if silu else 0, ldx, x.data_ptr(),
                         _dense(weight, "weight", (D, W), _F32), _dense(bias, "bias", (D,), _F32),
                         _dense(initial_state, "initial_state", state, dtype))
    return ConvProblem(c, x, weight, bias, initial_state, cu_seqlens, state)


def kda_conv_workspace_size(p: ConvProblem) -> int:
    return _lib.load().kda_conv_workspace_size(_byref(p.c))


def kda_conv_fwd(p: ConvProblem, *, output_final_state: bool = True, final_state: Optional[torch.Tensor] = None,
                 err: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, final state or None). ``final_state`` may be given, for example
    the initial state itself to update it in place."""
    x = p.x
    y = _like(x)
    if final_state is None and output_final_state:
        final_state = _empty(p.state_shape, dtype=x.dtype, device=x.device)
    st = _lib.load().kda_conv_fwd(_byref(p.c), y.data_ptr(), _dense(final_state, "final_state", p.state_shape, x.dtype),
                                  _error_word(err), _stream(stream, x))
    if st:
        _lib.check(st, "kda_conv_fwd")
    return y, final_state


def kda_conv_bwd(p: ConvProblem, dy: torch.Tensor, dfinal: Optional[torch.Tensor] = None, *,
                 workspace: Optional[torch.Tensor] = None, stream=None, need_dinit: Optional[bool] = None):
    """Backward of <dy, y> + <dfinal, final state>: (dx, dweight, dbias, dinit);
    dbias is None without a bias, dinit without an initial state (or with
    ``need_dinit`` False)."""
    x = p.x
    dx, dw, db = _like(x), _like(p.weight), _like(p.bias)
    dinit = None
    if need_dinit or (need_dinit is None and p.h0 is not None):
        dinit = _empty(p.state_shape, dtype=x.dtype, device=x.device)
    ws = _buffer(kda_conv_workspace_size(p), x.device, workspace)
    st = _lib.load().kda_conv_bwd(_byref(p.c), _dense(dy, "dy", x.shape, x.dtype),
                                  _dense(dfinal, "dfinal", p.state_shape, x.dtype), dx.data_ptr(), dw.data_ptr(),
                                  _addr(db), _addr(dinit), _addr(ws), _bytes(ws), _stream(stream, x))
    if st:
        _lib.check(st, "kda_conv_bwd")
    return dx, dw, db, dinit


# ------------------------------------------------------------------ scan

class SsmProblem(NamedTuple):
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
    dtype, tok, bc = x.dtype, x.shape, b.shape
    _need(len(tok) == 3 and dtype in _IO, "x must be [B, T, D], bf16 or fp32")
    _need(len(bc) == 4, "b must be [B, T, G, S]")
    B, T, D = tok
    G, S = bc[2], bc[3]
    if bc[0] != B or bc[1] != T:
        _refuse("b", "", (B, T, G, S), dtype)
    n, packed, cu = _axis(cu_seqlens, B)
    state = (n, D, S)
    p = _lib.SsmProblem(B, T, D, S, G, packed, cu, _IO[dtype], 1 if dt_softplus else 0, int(save_policy),
                        _rows(x, "x", tok, dtype), _rows(dt, "dt", tok, dtype),
                        0 if z is None else _rows(z, "z", tok, dtype), _rows(b, "b", bc, dtype),
                        _rows(c, "c", bc, dtype), x.data_ptr(), dt.data_ptr(), None if z is None else z.data_ptr(),
                        b.data_ptr(), c.data_ptr(), _dense(A_log, "A_log", (D, S), _F32),
                        _dense(d_skip, "d_skip", (D,), _F32), _dense(dt_bias, "dt_bias", (D,), _F32),
                        _dense(initial_state, "initial_state", state, _F32))
    return SsmProblem(p, x, dt, A_log, b, c, d_skip, z, dt_bias, initial_state, cu_seqlens, state)


def kda_ssm_workspace_size(p: SsmProblem, for_backward: bool) -> int:
    return _lib.load().kda_ssm_workspace_size(_byref(p.c), 1 if for_backward else 0)


def kda_ssm_saved_size(p: SsmProblem) -> int:
    return _lib.load().kda_ssm_saved_size(_byref(p.c))


def kda_ssm_fwd(p: SsmProblem, *, output_final_state: bool = True, ht: Optional[torch.Tensor] = None,
                saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                err: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, final states or None, saved or None). ``ht`` may be given, for
    example the initial state itself to update it in place."""
    x = p.x
    dev = x.device
    y = _like(x)
    if ht is None and output_final_state:
        ht = _empty(p.state_shape, dtype=_F32, device=dev)
    ws = _buffer(kda_ssm_workspace_size(p, False), dev, workspace)
    sv = _buffer(kda_ssm_saved_size(p), dev, saved) if p.c.save_policy else None
    st = _lib.load().kda_ssm_fwd(_byref(p.c), y.data_ptr(), _dense(ht, "ht", p.state_shape, _F32), _addr(sv), _addr(ws),
                                 _bytes(ws), _error_word(err), _stream(stream, x))
    if st:
        _lib.check(st, "kda_ssm_fwd")
    return y, ht, sv


def kda_ssm_bwd(p: SsmProblem, dy: torch.Tensor, dht: Optional[torch.Tensor] = None, *,
                saved: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None,
                need_dh0: Optional[bool] = None) -> SsmGrads:
    """Backward of <dy, y> + <dht, final states>. With save_policy 1, ``saved`` is
    what the forward returned for the same inputs."""
    x = p.x
    dev = x.device
    if p.c.save_policy:
        need = kda_ssm_saved_size(p)
        _need(need == 0 or (saved is not None and _bytes(saved) >= need),
              "save_policy 1 needs the forward's saved buffer")
    else:
        saved = None
    dh0 = None
    if need_dh0 or (need_dh0 is None and p.h0 is not None):
        dh0 = _empty(p.state_shape, dtype=_F32, device=dev)
    out = SsmGrads(_like(x), _like(p.dt), _like(p.A_log), _like(p.b), _like(p.cm), _like(p.d_skip), _like(p.z),
                   _like(p.dt_bias), dh0)
    g = _lib.SsmGrads(out.dx.data_ptr(), out.ddt.data_ptr(), _addr(out.dz), out.db.data_ptr(), out.dc.data_ptr(),
                      out.dA_log.data_ptr(), _addr(out.dd_skip), _addr(out.ddt_bias), _addr(dh0))
    ws = _buffer(kda_ssm_workspace_size(p, True), dev, workspace)
    st = _lib.load().kda_ssm_bwd(_byref(p.c), _dense(dy, "dy", x.shape, x.dtype), _dense(dht, "dht", p.state_shape, _F32),
                                 _addr(saved), _byref(g), _addr(ws), _bytes(ws), _stream(stream, x))
    if st:
        _lib.check(st, "kda_ssm_bwd")
    return out


# ------------------------------------------------------------------ norm

class NormProblem(NamedTuple):
    """A validated norm call plus the tensors it points to."""

    c: _lib.NormProblem
    x: torch.Tensor
    weight: torch.Tensor
    residual: Optional[torch.Tensor]
    scale_shape: Optional[tuple]


def make_norm_problem(x, weight, *, residual: Optional[torch.Tensor] = None, eps: float = 1e-6, out: str = "io",
                      group: int = 0) -> NormProblem:
    """Describe one call of the root-mean-square norm over the last axis of x
    (contiguous, bf16 or fp32, up to 16384 wide) with weight [D] fp32, after
    adding ``residual`` (x's shape and type) if given. ``out``: "io" for x's type,
    "e4m3" for 8-bit values with one fp32 scale per ``group`` columns (32, 64,
    128, or 0 for the row)."""
    dtype, shape = x.dtype, x.shape
    _need(len(shape) >= 1 and dtype in _IO, "x must be bf16 or fp32 rows")
    D = shape[-1]
    scales = None
    if out == "e4m3":
        scales = (*shape[:-1], -(-D // group) if group > 0 else 1)
    else:
        _need(out == "io", 'out must be "io" or "e4m3"')
    c = _lib.NormProblem(x.numel() // D if D else 0, D, _IO[dtype], 0 if scales is None else 1, group, eps,
                         _dense(x, "x", shape, dtype), _dense(residual, "residual", shape, dtype),
                         _dense(weight, "weight", (D,), _F32))
    return NormProblem(c, x, weight, residual, scales)


def kda_norm_workspace_size(p: NormProblem) -> int:
    return _lib.load().kda_norm_workspace_size(_byref(p.c))


def kda_norm_fwd(p: NormProblem, *, h: Optional[torch.Tensor] = None, stream=None):
    """Returns (y, scale or None, h): y in x's type, or torch.float8_e4m3fn with
    scale [..., groups]; h is the sum with the residual in x's type (x itself
    without one). ``h`` may be given, for example the residual's own buffer."""
    x = p.x
    scale = None
    if p.scale_shape is None:
        y = torch.empty_like(x)
    else:
        y = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        scale = _empty(p.scale_shape, dtype=_F32, device=x.device)
    if p.residual is None:
        h = x
    elif h is None:
        h = torch.empty_like(x)
    else:
        _dense(h, "h", x.shape, x.dtype)
    st = _lib.load().kda_norm_fwd(_byref(p.c), y.data_ptr(), _addr(scale), h.data_ptr(), _stream(stream, x))
    if st:
        _lib.check(st, "kda_norm_fwd")
    return y, scale, h


def kda_norm_bwd(p: NormProblem, dy: torch.Tensor, dres: Optional[torch.Tensor] = None, *,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward at x = the stored sum: (dx, dweight). ``dres`` is the gradient that
    reaches the sum past the norm; dx is the gradient of x and of the residual."""
    x = p.x
    dx, dw = torch.empty_like(x), torch.empty_like(p.weight)
    ws = _buffer(kda_norm_workspace_size(p), x.device, workspace)
    st = _lib.load().kda_norm_bwd(_byref(p.c), _dense(dy, "dy", x.shape, x.dtype), _dense(dres, "dres", x.shape, x.dtype),
                                  dx.data_ptr(), dw.data_ptr(), _addr(ws), _bytes(ws), _stream(stream, x))
    if st:
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
