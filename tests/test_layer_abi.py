"""Host-side checks of the layer operators' C ABI and binding: refusals and
workspace sizes (no GPU needed: no call here reaches CUDA)."""

import ctypes

import pytest
import torch

import chunkwise_delta_rule_gb300 as kda
from chunkwise_delta_rule_gb300 import _lib

X = 0x10000   # a stand-in for a device pointer; never dereferenced
VP = ctypes.c_void_p


def conv(**kw):
    f = dict(B=2, T=10, D=16, W=4, N=0, cu_seqlens=None, io=0, silu=1, ldx=0, x=X, weight=X, bias=None, h0=None)
    return _lib.ConvProblem(**dict(f, **kw))


def ssm(**kw):
    f = dict(B=2, T=10, D=16, S=16, G=1, N=0, cu_seqlens=None, io=0, dt_softplus=1, save_policy=0, ldx=0, lddt=0, ldz=0,
             ldb=0, ldc=0, x=X, dt=X, z=None, b=X, c=X, A_log=X, d_skip=None, dt_bias=None, h0=None)
    return _lib.SsmProblem(**dict(f, **kw))


def norm(**kw):
    f = dict(rows=4, D=64, io=0, out=0, group=0, eps=1e-6, x=X, residual=None, weight=X)
    return _lib.NormProblem(**dict(f, **kw))


BAD_AXIS = [(dict(B=0), 1), (dict(T=-1), 1), (dict(D=0), 1), (dict(io=2), 1), (dict(cu_seqlens=X, N=2), 1),
            (dict(B=1, cu_seqlens=X, N=0), 1), (dict(B=1 << 16, T=1 << 16), 2)]


@pytest.mark.parametrize("kw,status", BAD_AXIS + [(dict(W=1), 2), (dict(W=5), 2), (dict(silu=2), 1), (dict(ldx=15), 1),
                                                  (dict(weight=None), 1), (dict(x=None), 1)])
def test_conv_refusals(kw, status):
    lib = _lib.load()
    p = conv(**kw)
    assert lib.kda_conv_fwd(ctypes.byref(p), VP(X), None, None, None) == status and _lib.last_error()
    assert lib.kda_conv_bwd(ctypes.byref(p), VP(X), None, VP(X), VP(X), None, None, VP(X), 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", BAD_AXIS + [
    (dict(S=0), 1), (dict(S=65), 2), (dict(G=3), 1), (dict(G=0), 1), (dict(dt_softplus=2), 1), (dict(save_policy=2), 1),
    (dict(lddt=15), 1), (dict(ldb=15), 1), (dict(A_log=None), 1), (dict(dt=None), 1), (dict(b=None), 1)])
def test_scan_refusals(kw, status):
    lib = _lib.load()
    p = ssm(**kw)
    g = _lib.SsmGrads(**{n: X for n, _ in _lib.SsmGrads._fields_})
    assert lib.kda_ssm_fwd(ctypes.byref(p), VP(X), None, None, VP(X), 1 << 40, None, None) == status and _lib.last_error()
    assert lib.kda_ssm_bwd(ctypes.byref(p), VP(X), None, None, ctypes.byref(g), VP(X), 1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [(dict(rows=-1), 1), (dict(D=0), 1), (dict(D=16385), 2), (dict(io=3), 1),
                                       (dict(out=2), 1), (dict(group=16), 2), (dict(eps=-1.0), 1),
                                       (dict(eps=float("nan")), 1), (dict(x=None), 1), (dict(weight=None), 1)])
def test_norm_refusals(kw, status):
    lib = _lib.load()
    p = norm(**kw)
    assert lib.kda_norm_fwd(ctypes.byref(p), VP(X), VP(X), None, None) == status and _lib.last_error()
    assert lib.kda_norm_bwd(ctypes.byref(p), VP(X), None, VP(X), VP(X), VP(X), 1 << 40, None) == status


def test_missing_outputs_and_workspaces():
    lib = _lib.load()
    c, s, n = conv(), ssm(), norm()
    big = 1 << 40
    assert lib.kda_conv_fwd(ctypes.byref(c), None, None, None, None) == 1
    assert lib.kda_conv_bwd(ctypes.byref(c), None, None, VP(X), VP(X), None, None, VP(X), big, None) == 1
    for ws, size in ((None, 0), (VP(X + 16), big), (VP(X), lib.kda_conv_workspace_size(ctypes.byref(c)) - 1)):
        assert lib.kda_conv_bwd(ctypes.byref(c), VP(X), None, VP(X), VP(X), None, None, ws, size, None) == 3
    g = _lib.SsmGrads(**{f: X for f, _ in _lib.SsmGrads._fields_})
    assert lib.kda_ssm_fwd(ctypes.byref(s), None, None, None, None, 0, None, None) == 1
    assert lib.kda_ssm_bwd(ctypes.byref(s), VP(X), None, None, ctypes.byref(g), None, 0, None) == 3
    g.dx = None
    assert lib.kda_ssm_bwd(ctypes.byref(s), VP(X), None, None, ctypes.byref(g), VP(X), big, None) == 1
    z = ssm(z=X)
    g.dx, g.dz = X, None
    assert lib.kda_ssm_bwd(ctypes.byref(z), VP(X), None, None, ctypes.byref(g), VP(X), big, None) == 1
    a = ssm(save_policy=1)
    assert lib.kda_ssm_fwd(ctypes.byref(a), VP(X), None, None, VP(X), big, None, None) == 3
    assert lib.kda_norm_fwd(ctypes.byref(n), None, None, None, None) == 1
    assert lib.kda_norm_fwd(ctypes.byref(norm(out=1)), VP(X), None, None, None) == 1
    assert lib.kda_norm_fwd(ctypes.byref(norm(residual=X)), VP(X), None, None, None) == 1
    assert lib.kda_norm_bwd(ctypes.byref(norm(residual=X)), VP(X), None, VP(X), VP(X), VP(X), big, None) == 1
    assert lib.kda_norm_bwd(ctypes.byref(n), VP(X), None, VP(X), VP(X), None, 0, None) == 3


def test_sizes():
    lib = _lib.load()
    for bad in (conv(W=9), conv(B=0)):
        assert lib.kda_conv_workspace_size(ctypes.byref(bad)) == 0
    assert lib.kda_conv_workspace_size(ctypes.byref(conv())) % 256 == 0
    assert lib.kda_ssm_saved_size(ctypes.byref(ssm())) == 0
    # every 16th state: one per row of 10 tokens
    assert lib.kda_ssm_saved_size(ctypes.byref(ssm(save_policy=1))) == 2 * 16 * 16 * 4
    assert lib.kda_ssm_saved_size(ctypes.byref(ssm(save_policy=1, T=17))) == 2 * 2 * 16 * 16 * 4
    assert lib.kda_ssm_workspace_size(ctypes.byref(ssm(S=99)), 1) == 0
    assert lib.kda_norm_workspace_size(ctypes.byref(norm(D=0))) == 0


def test_the_binding_refuses_what_the_kernels_do_not_take():
    x = torch.zeros(2, 10, 16)
    w = torch.zeros(16, 4)
    with pytest.raises(ValueError):
        kda.make_conv_problem(x, w)                       # not on a GPU
    with pytest.raises(ValueError):
        kda.make_conv_problem(x.half(), w)
    with pytest.raises(ValueError):
        kda.make_ssm_problem(x, x, torch.zeros(16, 16), torch.zeros(2, 10, 16), torch.zeros(2, 10, 16))
    with pytest.raises(ValueError):
        kda.make_norm_problem(x, torch.zeros(16))
    with pytest.raises(ValueError):
        kda.make_norm_problem(x.double(), torch.zeros(16))
