"""The example runs the operators together: it learns, and serving agrees with
one pass over the whole sequences.

Tolerances on the logits (normwise), four layers deep:
- fp32: the chunked and the token-by-token delta rule and the scan each stay
  within 1e-4 of their definition, four of them in a row with norms that keep
  the size: 1e-3;
- bf16: about ten roundings of 2^-9 a layer on each side that differ between the
  two orders of computation, 80 in all: sqrt(80) x 2^-9 = 1.7e-2, three times
  that as the bound: 5e-2.
"""

import math

import pytest
import torch

from examples import hybrid_stack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-3), (torch.bfloat16, 5e-2)])
def test_serving_agrees_with_one_pass(dtype, tol):
    torch.manual_seed(3)
    model = hybrid_stack.HybridStack().cuda()
    diff, _ = hybrid_stack.agreement(model, dtype=dtype)
    assert diff < tol


def test_training_learns():
    torch.manual_seed(4)
    model = hybrid_stack.HybridStack().cuda()
    losses = hybrid_stack.train(model, 300)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 1.0 < losses[0]   # a guess has log(64) = 4.16
