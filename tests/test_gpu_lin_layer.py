"""The operators together, as a layer has them: norm with 8-bit rows, projections in
8 bits, linear attention over packed prompts, then token by token; and training
steps through the same parts, one of them captured."""

import numpy as np
import pytest
import torch

from oracle import layer
from tests.helpers import check_close, np64
from tests.test_gpu_layer import gen_of, starts_of

pytestmark = pytest.mark.gpu

D, H, HV, K, V = 256, 2, 4, 64, 64
INNER = 2 * H * K + HV * V


def weights(seed):
    g = gen_of(seed)
    return (torch.randn(INNER, D, generator=g) * D ** -0.5).cuda(), (torch.randn(D, HV * V, generator=g) * (HV * V) ** -0.5).cuda()


def heads(p):
    q, k, v = p.split([H * K, H * K, HV * V], -1)
    return q.unflatten(-1, (H, K)), k.unflatten(-1, (H, K)), v.unflatten(-1, (HV, V))


def test_serving_is_one_pass():
    """Packed prompts prefilled, then six tokens each one by one, the states in place: the layer's outputs are those of one
    pass over the whole sequences. Norm and projections are the same arithmetic row by row; linear attention differs by
    its roundings to bf16 only (2 x 2^-8), which the second projection's rounding of its rows to e4m3 (2^-4 a value at
    most, 2^-4 sqrt(2) / sqrt(3) of a row's norm) may turn into other 8-bit values."""
    import chunkwise_delta_rule_gb300 as kda
    inp, outp = weights(61)
    w, wo = (kda.kda_quant8(kda.make_quant8_problem(t, blocks=True)) for t in (inp, outp))
    norm = torch.ones(D, device="cuda")
    decay = -torch.exp2(-torch.arange(1.0, HV + 1, device="cuda"))

    def run(x, cu, state):
        y, s, _ = kda.kda_norm_fwd(kda.make_norm_problem(x, norm, out="e4m3", group=128))
        p = kda.kda_mm8(kda.make_mm8_problem(y, s, w.q, w.scale))
        o, ht = kda.kda_lin_fwd(kda.make_lin_problem(*heads(p), decay, initial_state=state, cu_seqlens=cu), ht=state)
        r = kda.kda_quant8(kda.make_quant8_problem(o.flatten(2)))
        return o, kda.kda_mm8(kda.make_mm8_problem(r.q, r.scale, wo.q, wo.scale)), ht

    lengths, steps = [37, 130, 1, 200], 6
    g = gen_of(62)
    x = [torch.randn(1, n + steps, D, generator=g).bfloat16().cuda() for n in lengths]
    _, cu = starts_of(1, 0, lengths)
    o, y, state = run(torch.cat([t[:, :n] for t, n in zip(x, lengths)], 1), cu, None)
    parts = [[a] for a in o.split(lengths, 1)], [[a] for a in y.split(lengths, 1)]
    for i in range(steps):
        o, y, _ = run(torch.stack([t[0, n + i] for t, n in zip(x, lengths)]).unsqueeze(1), None, state)
        for dst, t in zip(parts, (o, y)):
            for j, a in enumerate(t):
                dst[j].append(a[None])
    for j, t in enumerate(x):
        o, y, _ = run(t, None, None)
        check_close("o", np64(torch.cat(parts[0][j], 1)), np64(o), 2 * 7.9e-3)
        check_close("y", np64(torch.cat(parts[1][j], 1)), np64(y), 2.0 ** -4 * (2 / 3) ** 0.5)


def test_a_training_step():
    """Gradients through norm, 8-bit projections and linear attention: each operator's own backward, chained. The loss is
    linear in the layer's output; its slope along a direction of the attention's values is the gradient's."""
    import chunkwise_delta_rule_gb300 as kda
    inp, outp = (t.requires_grad_() for t in weights(63))
    norm = torch.ones(D, device="cuda", requires_grad=True)
    decay = -torch.exp2(-torch.arange(1.0, HV + 1, device="cuda"))
    _, cu = starts_of(1, 0, [150, 0, 33, 70])
    g = gen_of(64)
    x = torch.randn(1, 253, D, generator=g).bfloat16().cuda().requires_grad_()
    dy = torch.randn(1, 253, D, generator=g).bfloat16().cuda()
    h, _ = kda.rms_norm(x, norm)
    p = kda.linear8(h, inp)
    p.retain_grad()
    q, k, v = heads(p)
    o, _ = kda.linear_attention(q, k, v, decay, cu_seqlens=cu)
    o.retain_grad()
    y = kda.linear8(o.flatten(2), outp)
    y.backward(dy)
    for t in (x, norm, inp, outp):
        assert t.grad.shape == t.shape and torch.isfinite(t.grad).all() and t.grad.any()
    ref = layer.lin(*(np64(t)[0] for t in (q, k, v)), np64(decay), K ** -0.5, None, [0, 150, 150, 183, 253], np64(o.grad)[0])
    want = np.concatenate([ref["dq"].reshape(253, -1), ref["dk"].reshape(253, -1), ref["dv"].reshape(253, -1)], 1)
    check_close("dp", np64(p.grad)[0], want, 7.9e-3)
    # the output's gradient, of the values that the weight's rounding stands for
    r = kda.kda_quant8(kda.make_quant8_problem(outp.detach(), blocks=True))
    held = np64(r.q.float()) * np.repeat(np.repeat(np64(r.scale), 128, 0), 128, 1)[:D, :HV * V]
    d = kda.kda_quant8(kda.make_quant8_problem(dy[0]))
    hd = np64(d.q.float()) * np.repeat(np64(d.scale), 128, 1)[:, :D]
    check_close("do", np64(o.grad)[0].reshape(253, -1), hd @ held, 4e-3)


def test_a_captured_training_step():
    """Forward and backward of the projections and the attention in one graph: replays on new values give what the eager
    step gives, bit for bit (no sum goes by the order of arrival)."""
    import chunkwise_delta_rule_gb300 as kda
    inp, outp = (t.requires_grad_() for t in weights(65))
    decay = -torch.exp2(-torch.arange(1.0, HV + 1, device="cuda"))
    g = gen_of(66)
    x, dy = (torch.randn(2, 300, D, generator=g).bfloat16().cuda() for _ in range(2))
    x.requires_grad_()

    def step():
        o, _ = kda.linear_attention(*heads(kda.linear8(x, inp)), decay)
        return torch.autograd.grad(kda.linear8(o.flatten(2), outp), (x, inp, outp), dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        with torch.no_grad():
            x.copy_(torch.randn(x.shape, generator=g))
            dy.copy_(torch.randn(dy.shape, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        assert all(torch.equal(a, b) and a.any() for a, b in zip(kept, step()))
