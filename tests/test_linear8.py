"""What ``linear8`` asks of the rounding and the product, seen on the host: both are
stood in for by elementary operations that note their calls (no GPU needed)."""

import pytest
import torch

from chunkwise_delta_rule_gb300 import layer


@pytest.fixture
def asked(monkeypatch):
    """(rows, transposed) of every rounding, in order."""
    seen = []

    def quant(x, *, blocks=False, rows=True, transposed=False):
        seen.append((rows, transposed))
        t = x.reshape(-1, x.shape[-1])
        return layer.Quant8(x if rows else None, x if rows else None, t.t() if transposed else None, t.t() if transposed else None)

    monkeypatch.setattr(layer, "make_quant8_problem", quant)
    monkeypatch.setattr(layer, "kda_quant8", lambda p: p)
    monkeypatch.setattr(layer, "make_mm8_problem", lambda a, sa, b, sb, out: a @ b.t())
    monkeypatch.setattr(layer, "kda_mm8", lambda p, err=None: p)
    return seen


def leaves(need_x, need_w):
    g = torch.Generator().manual_seed(1)
    return torch.randn(2, 3, 8, generator=g).requires_grad_(need_x), torch.randn(5, 8, generator=g).requires_grad_(need_w)


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_no_transposed_copy_without_a_backward(asked, mode):
    """A parameter asks for its gradient in every mode; copies for a backward are made where one can come."""
    x, w = leaves(True, True)
    with mode():
        y = layer.linear8(x, w)
    assert not y.requires_grad and asked == [(True, False), (True, False)]


@pytest.mark.parametrize("need_x,need_w", [(False, False), (True, False), (False, True), (True, True)])
def test_copies_are_the_gradients(asked, need_x, need_w):
    x, w = leaves(need_x, need_w)
    y = layer.linear8(x, w)
    assert asked == [(True, need_w), (True, need_x)]
    if not (need_x or need_w):
        return
    dy = torch.ones_like(y)
    y.backward(dy)
    assert asked[2:] == [(need_x, need_w)]
    if need_x:
        assert torch.allclose(x.grad, dy @ w)
    if need_w:
        assert torch.allclose(w.grad, dy.flatten(0, 1).t() @ x.flatten(0, 1))
