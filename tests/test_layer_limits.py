"""Host-side limits of the layer operators (no GPU needed: no call here reaches
CUDA)."""

import ctypes

import pytest
import torch

import chunkwise_delta_rule_gb300 as kda
from chunkwise_delta_rule_gb300 import _lib
from tests.test_layer_abi import VP, X, norm, ssm


@pytest.mark.parametrize("rows", [(1 << 30) + 1, (1 << 31) - 1])
def test_norm_rows_beyond_the_kernels_counters_are_refused(rows):
    """A row counter steps past the last row by a grid's rows: near 2^31 it would come out negative."""
    lib = _lib.load()
    p = norm(rows=rows, D=1)
    assert lib.kda_norm_fwd(ctypes.byref(p), VP(X), VP(X), None, None) == 2 and "rows" in _lib.last_error()
    assert lib.kda_norm_bwd(ctypes.byref(p), VP(X), None, VP(X), VP(X), VP(X), 1 << 40, None) == 2
    assert lib.kda_norm_workspace_size(ctypes.byref(p)) == 0
    assert lib.kda_norm_workspace_size(ctypes.byref(norm(rows=1 << 30, D=1))) > 0


def test_the_scans_backward_with_an_error_word_refuses_what_it_refuses_without():
    lib = _lib.load()
    g = _lib.SsmGrads(**{n: X for n, _ in _lib.SsmGrads._fields_})
    for kw, status in ((dict(S=0), 1), (dict(S=65), 2), (dict(A_log=None), 1), (dict(G=3), 1)):
        p = ssm(**kw)
        assert lib.kda_ssm_bwd_err(ctypes.byref(p), VP(X), None, None, ctypes.byref(g), VP(X), 1 << 40, VP(X), None) == status
    p = ssm()
    assert lib.kda_ssm_bwd_err(ctypes.byref(p), VP(X), None, None, ctypes.byref(g), None, 0, VP(X), None) == 3


def test_the_binding_names_what_it_refuses():
    """Types and ranks are told apart from tensors that are not on a GPU."""
    x, w = torch.zeros(2, 10, 16), torch.zeros(16, 4)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.make_conv_problem(x, w)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        kda.make_ssm_problem(x, x, torch.zeros(16, 16), torch.zeros(2, 10, 1, 16), torch.zeros(2, 10, 1, 16))
    with pytest.raises(ValueError, match="x must be a contiguous CUDA tensor"):
        kda.make_norm_problem(x, torch.zeros(16))
    for bad in (x.half(), x.double(), x[0]):
        with pytest.raises(ValueError, match=r"x must be \[B, T, D\], bf16 or fp32"):
            kda.make_conv_problem(bad, w)
        with pytest.raises(ValueError, match=r"x must be \[B, T, D\], bf16 or fp32"):
            kda.make_ssm_problem(bad, bad, torch.zeros(16, 16), torch.zeros(2, 10, 1, 16), torch.zeros(2, 10, 1, 16))
    for bad in (x.half(), x.double(), torch.zeros(())):
        with pytest.raises(ValueError, match="x must be bf16 or fp32 rows"):
            kda.make_norm_problem(bad, torch.zeros(16))
    with pytest.raises(ValueError, match=r"weight must be \[D, W\]"):
        kda.make_conv_problem(x, w[0])
    with pytest.raises(ValueError, match=r"b must be \[B, T, G, S\]"):
        kda.make_ssm_problem(x, x, torch.zeros(16, 16), torch.zeros(2, 10, 16), torch.zeros(2, 10, 16))
    with pytest.raises(ValueError, match="out must be"):
        kda.make_norm_problem(x, torch.zeros(16), out="fp8")
