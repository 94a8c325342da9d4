"""The 8-bit product where a pair of SMs takes more than one tile, where outputs do
not start on whole accesses, and in graphs: paths beside those of the oracle's
cases, with their tolerances."""

import pytest
import torch

from tests.helpers import check_close, np64
from tests.test_gpu_fp8 import cuda, mm_case, mm_ref
from tests.test_gpu_lin_edges import launched

pytestmark = pytest.mark.gpu


# 110 tiles of 256 x 256, more than a device has pairs of SMs, 9 groups (two rounds of scales, more than the stages hold):
# whole rows of outputs, and rows that start on any address; 256 tiles, some pairs walk four of them, of copied rows
@pytest.mark.parametrize("M,N,K", [(2500, 2752, 1040), (2500, 2750, 1040), (4000, 3850, 700)])
@pytest.mark.parametrize("b", ["blocks", "rows"])
def test_several_tiles_to_a_pair(M, N, K, b):
    import chunkwise_delta_rule_gb300 as kda
    c = mm_case(M, N, K, b, 91)
    ref = mm_ref(*c)
    c = cuda(*c)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for out, tol in (("fp32", 1e-5), ("bf16", 4e-3)):
        p = kda.make_mm8_problem(*c, out=out)
        y, names = launched(lambda: kda.kda_mm8(p, err=err))
        assert names - {"k_mm8_align"} == {"k_mm8_pair"}
        check_close(out, np64(y), ref, tol)
        assert torch.equal(y, kda.kda_mm8(p, err=err))
    assert int(err) == 0


@pytest.mark.parametrize("M,N,K,kernel", [(1, 5000, 1040, "rows"), (16, 20001, 272, "rows"), (64, 8200, 400, "rows"), (65, 4500, 272, "pair"),
                                          (256, 4096, 144, "rows"), (512, 4096, 144, "pair")])
@pytest.mark.parametrize("b", ["blocks", "rows"])
def test_few_rows_of_a_and_many_of_b(M, N, K, kernel, b):
    """Both sides of the rule that chooses the kernel: up to 64 rows never go through tiles of 256."""
    import chunkwise_delta_rule_gb300 as kda
    c = mm_case(M, N, K, b, 96)
    y, names = launched(lambda: kda.kda_mm8(kda.make_mm8_problem(*cuda(*c), out="fp32")))
    assert names == {"k_mm8_" + kernel}
    check_close("y", np64(y), mm_ref(*c), 1e-5)


@pytest.mark.parametrize("M,N,K", [(40, 64, 256), (2000, 1300, 300)])
@pytest.mark.parametrize("out", ["bf16", "fp32"])
def test_an_output_off_16_bytes(M, N, K, out):
    """Behind and before the given rows nothing is written."""
    import chunkwise_delta_rule_gb300 as kda
    c = mm_case(M, N, K, "blocks", 92)
    p = kda.make_mm8_problem(*cuda(*c), out=out)
    flat = torch.full((M * N + 2,), -7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    y = kda.kda_mm8(p, y=flat[1:-1].view(M, N))
    assert y.data_ptr() % 16 == flat.element_size()
    check_close(out, np64(y), mm_ref(*c), 4e-3 if out == "bf16" else 1e-5)
    assert torch.equal(y, kda.kda_mm8(p)) and flat[0] == -7 and flat[-1] == -7


@pytest.mark.parametrize("b", ["blocks", "rows"])
def test_many_rows_in_a_graph(b):
    import chunkwise_delta_rule_gb300 as kda
    M, N, K = 2500, 2752, 1040
    c = cuda(*mm_case(M, N, K, b, 93))
    p = kda.make_mm8_problem(*c)
    assert launched(lambda: kda.kda_mm8(p))[1] == {"k_mm8_pair"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = kda.kda_mm8(p)
    for seed in (94, 95):
        for t, new in zip(c, mm_case(M, N, K, b, seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, kda.kda_mm8(p))


@pytest.mark.parametrize("no_grad", [torch.no_grad, torch.inference_mode])
def test_linear8_rounds_rows_only_without_gradients(no_grad):
    """The same values as a recorded call's; the weight a parameter."""
    import chunkwise_delta_rule_gb300 as kda
    x = torch.randn(100, 264, device="cuda").bfloat16()
    w = torch.nn.Parameter(torch.randn(200, 264, device="cuda"))
    y = kda.linear8(x, w)
    with no_grad():
        z = kda.linear8(x, w)
    assert y.requires_grad and not z.requires_grad and torch.equal(y.detach(), z)
