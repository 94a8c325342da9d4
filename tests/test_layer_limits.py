"""Host-side limits of the layer operators (no GPU needed: no call here reaches
CUDA)."""

import ctypes

import pytest

from chunkwise_delta_rule_gb300 import _lib
from tests.test_layer_abi import VP, X, norm


@pytest.mark.parametrize("rows", [(1 << 30) + 1, (1 << 31) - 1])
def test_norm_rows_beyond_the_kernels_counters_are_refused(rows):
    """A row counter steps past the last row by a grid's rows: near 2^31 it would come out negative."""
    lib = _lib.load()
    p = norm(rows=rows, D=1)
    assert lib.kda_norm_fwd(ctypes.byref(p), VP(X), VP(X), None, None) == 2 and "rows" in _lib.last_error()
    assert lib.kda_norm_bwd(ctypes.byref(p), VP(X), None, VP(X), VP(X), VP(X), 1 << 40, None) == 2
    assert lib.kda_norm_workspace_size(ctypes.byref(p)) == 0
    assert lib.kda_norm_workspace_size(ctypes.byref(norm(rows=1 << 30, D=1))) > 0
