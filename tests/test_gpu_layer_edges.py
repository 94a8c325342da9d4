"""GPU tests of the layer operators where their callers differ from the ordinary
ones: rows of unlike alignment, streams, buffers and refusals. Oracle and
tolerances as in test_gpu_layer."""

import pytest
import torch

from tests.helpers import check_close, np64
from tests.test_gpu_layer import scan_case, scan_problem, tol, wide_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,S", [("bf16", 16), ("bf16", 12), ("fp32", 16), ("fp32", 5)])
@pytest.mark.parametrize("name", ["x", "dt", "z", "b", "c"])
def test_scan_with_one_tensor_off_its_alignment(io, S, name):
    """One input starts one element off, the others on whole accesses; rows, tiles and states end raggedly, so that
    some copies are of nothing. (A copy of nothing still has to name an address that its access may have.)"""
    import chunkwise_delta_rule_gb300 as kda
    k, c, _, ref = scan_case(dict(io=io, B=2, T=37, D=72, S=S, state=True), 71)
    t = c[name].cpu()
    c[name] = wide_rows(t, 1) if t.dim() == 3 else wide_rows(t.flatten(2), 1).unflatten(-1, (1, S))
    for save in (0, 1):
        p = scan_problem(k, c, None, save)
        y, ht, saved = kda.kda_ssm_fwd(p)
        g = kda.kda_ssm_bwd(p, c["dy"], c["dht"], saved=saved)
        got = dict(y=y, ht=ht, dx=g.dx, ddt=g.ddt, dA_log=g.dA_log, db=g.db, dc=g.dc, dd_skip=g.dd_skip, dz=g.dz,
                   ddt_bias=g.ddt_bias, dh0=g.dh0)
        for n, v in got.items():
            check_close(n, np64(v).reshape(ref[n].shape), ref[n], tol(v, True))
