"""Host-side checks of the C ABI and binding of linear attention and of the 8-bit
quantiser and product: refusals and workspace sizes (no GPU needed: no call here
reaches CUDA)."""

import ctypes

import pytest
import torch

import chunkwise_delta_rule_gb300 as kda
from chunkwise_delta_rule_gb300 import _lib
from tests.test_layer_abi import BAD_AXIS, VP, X

BIG = 1 << 40


def lin(**kw):
    f = dict(B=2, T=10, H=2, K=16, V=16, N=0, cu_seqlens=None, io=0, HV=0, scale=0.0, ldq=0, ldk=0, ldv=0, q=X, k=X, v=X,
             decay=X, h0=None)
    return _lib.LinProblem(**dict(f, **kw))


def quant(**kw):
    f = dict(rows=4, D=64, io=0, blocks=0, ldx=0, ldq=0, ldqt=0, x=X)
    return _lib.Quant8Problem(**dict(f, **kw))


def mm(**kw):
    f = dict(M=4, N=64, K=64, out=0, b_rows=0, lda=0, ldb=0, a=X, b=X, scale_a=X, scale_b=X)
    return _lib.Mm8Problem(**dict(f, **kw))


LIN_AXIS = [(dict(k, **({"K": k["D"]} if "D" in k else {})), s) for k, s in BAD_AXIS]


@pytest.mark.parametrize("kw,status", [({n: v for n, v in k.items() if n != "D"}, s) for k, s in LIN_AXIS] + [
    (dict(H=0), 1), (dict(V=0), 1), (dict(K=257), 2), (dict(V=257), 2), (dict(HV=3), 1), (dict(HV=1), 1), (dict(HV=-2), 1),
    (dict(H=1 << 17), 2), (dict(ldq=31), 1), (dict(ldk=31), 1), (dict(ldv=31), 1), (dict(HV=4, ldv=63), 1), (dict(q=None), 1),
    (dict(k=None), 1), (dict(v=None), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1)])
def test_lin_refusals(kw, status):
    lib = _lib.load()
    p = lin(**kw)
    assert lib.kda_lin_fwd(ctypes.byref(p), VP(X), None, VP(X), BIG, None, None) == status and _lib.last_error()
    assert lib.kda_lin_bwd(ctypes.byref(p), VP(X), None, VP(X), VP(X), VP(X), None, VP(X), BIG, None, None) == status


def test_lin_missing_outputs_and_workspaces():
    lib = _lib.load()
    p = lin()
    assert lib.kda_lin_fwd(ctypes.byref(p), None, None, VP(X), BIG, None, None) == 1
    for i in range(4):
        a = [VP(X)] * 4
        a[i] = None
        assert lib.kda_lin_bwd(ctypes.byref(p), a[0], None, a[1], a[2], a[3], None, VP(X), BIG, None, None) == 1
    # dh0 over dht or h0, which other calls of the same backward still read
    assert lib.kda_lin_bwd(ctypes.byref(p), VP(X), VP(X), VP(X), VP(X), VP(X), VP(X), VP(X), BIG, None, None) == 1
    assert lib.kda_lin_bwd(ctypes.byref(lin(h0=2 * X)), VP(X), None, VP(X), VP(X), VP(X), VP(2 * X), VP(X), BIG, None, None) == 1
    g = lin(HV=4)
    for p, back in ((lin(B=1, T=5000), False), (g, True)):
        need = lib.kda_lin_workspace_size(ctypes.byref(p), back)
        assert need > 0 and need % 256 == 0
        for ws, size in ((None, 0), (VP(X + 16), BIG), (VP(X), need - 1)):
            if back:
                assert lib.kda_lin_bwd(ctypes.byref(p), VP(X), None, VP(X), VP(X), VP(X), None, ws, size, None, None) == 3
            else:
                assert lib.kda_lin_fwd(ctypes.byref(p), VP(X), None, ws, size, None, None) == 3
    assert lib.kda_lin_workspace_size(ctypes.byref(lin(K=999)), 1) == 0


@pytest.mark.parametrize("kw,status", [(dict(rows=-1), 1), (dict(D=0), 1), (dict(rows=(1 << 22) + 1), 2), (dict(D=(1 << 20) + 1), 2),
                                       (dict(io=2), 1), (dict(blocks=2), 1), (dict(ldx=63), 1), (dict(ldq=63), 1),
                                       (dict(ldqt=3), 1), (dict(x=None), 1)])
def test_quant8_refusals(kw, status):
    lib = _lib.load()
    assert lib.kda_quant8(ctypes.byref(quant(**kw)), VP(X), VP(X), VP(X), VP(X), None) == status and _lib.last_error()


def test_quant8_outputs_come_in_pairs():
    lib = _lib.load()
    for a in ((None,) * 4, (VP(X), None, None, None), (None, VP(X), VP(X), VP(X)), (VP(X), VP(X), VP(X), None),
              (VP(X), VP(X), None, VP(X))):
        assert lib.kda_quant8(ctypes.byref(quant()), *a, None) == 1 and _lib.last_error()


@pytest.mark.parametrize("kw,status", [(dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(M=(1 << 22) + 1), 2),
                                       (dict(N=(1 << 20) + 1), 2), (dict(K=(1 << 22) + 1), 2), (dict(out=2), 1),
                                       (dict(b_rows=2), 1), (dict(lda=63), 1), (dict(ldb=63), 1), (dict(a=None), 1),
                                       (dict(b=None), 1), (dict(scale_a=None), 1), (dict(scale_b=None), 1)])
def test_mm8_refusals(kw, status):
    lib = _lib.load()
    p = mm(**kw)
    assert lib.kda_mm8(ctypes.byref(p), VP(X), VP(X), BIG, None, None) == status and _lib.last_error()
    if status == 2 or not any(v is None for v in kw.values()):
        assert lib.kda_mm8_workspace_size(ctypes.byref(p)) == 0


def test_mm8_without_an_output_is_refused():
    assert _lib.load().kda_mm8(ctypes.byref(mm()), None, VP(X), BIG, None, None) == 1


def test_the_binding_refuses_what_the_kernels_do_not_take():
    q = torch.zeros(2, 10, 2, 16)
    for bad in (q.half(), q[0], q.double()):
        with pytest.raises(ValueError, match=r"q must be \[B, T, H, K\], bf16 or fp32"):
            kda.make_lin_problem(bad, q, q)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kda.make_lin_problem(q, q, q)
    with pytest.raises(ValueError, match=r"v must be \[B, T, HV, V\]"):
        kda.make_lin_problem(q, q, q[0])
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="x must be bf16 or fp32 rows"):
        kda.make_quant8_problem(x.half())
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.make_quant8_problem(x)
    a, s = x.to(torch.float8_e4m3fn), torch.ones(4, 1)
    with pytest.raises(ValueError, match="a must be e4m3 rows"):
        kda.make_mm8_problem(x, s, a, s)
    with pytest.raises(ValueError, match="b must be e4m3"):
        kda.make_mm8_problem(a, s, x, s)
    with pytest.raises(ValueError, match="out must be"):
        kda.make_mm8_problem(a, s, a, s, out="fp16")
    with pytest.raises(ValueError, match="a must be a CUDA tensor"):
        kda.make_mm8_problem(a, s, a, s)
