"""GPU parity of linear attention with a decay for each head against its FP64
oracle, and its serving and training properties.

Tolerances (normwise relative error), from the formats:
- fp32 outputs and states: a value is the end of a chain of at most some 900
  additions and products (the tokens and groups behind it and the widths), each
  off by at most 2^-24 with a sign of its own: 30 x 6e-8 = 1.8e-6, and powers of
  the decay to two units; 1e-5;
- bf16 outputs: one rounding of the output, at most 2^-8 of the value, and on the
  tensor cores one of each score or of the state it is multiplied with, another
  2^-8 of terms that add up to the value: 2 x 3.91e-3 = 7.9e-3 with what the fp32
  arithmetic adds.
"""

import numpy as np
import pytest
import torch

from oracle import layer
from tests.helpers import check_close, np64
from tests.test_gpu_layer import DT, gen_of, opt64, starts_of, wide_rows

pytestmark = pytest.mark.gpu


def tol(t):
    return 7.9e-3 if t.dtype == torch.bfloat16 else 1e-5


def decays(kind, HV):
    if kind is None:
        return None
    if kind == "slopes":
        return -torch.exp2(-1 - 7 * torch.arange(HV) / max(1, HV - 1))
    if kind == "strong":
        return torch.tensor([-30.0, -200.0, float("-inf"), -2.0, -1e-4] * HV)[:HV].contiguous()
    return 0.003 * (torch.arange(HV) + 1.0)     # growing states


def lin_case(kw, seed):
    k = dict(dict(T=0, HV=None, state=False, lengths=None, pad=0, decay="slopes", scale=None), **kw)
    g = gen_of(seed)
    starts, cu = starts_of(k["B"], k["T"], k["lengths"])
    T = starts[-1] if cu is not None else k["T"]
    B, H, K, V, dt = k["B"], k["H"], k["K"], k["V"], DT[k["io"]]
    HV, n = k["HV"] or H, len(starts) - 1
    c = dict(q=torch.randn(B, T, H, K, generator=g).to(dt), k=torch.randn(B, T, H, K, generator=g).to(dt),
             v=torch.randn(B, T, HV, V, generator=g).to(dt), decay=decays(k["decay"], HV),
             h0=torch.randn(n, HV, K, V, generator=g) if k["state"] else None,
             do=torch.randn(B, T, HV, V, generator=g).to(dt), dht=torch.randn(n, HV, K, V, generator=g) if k["state"] else None)
    k["starts"] = starts
    gpu = {x: None if t is None else t.cuda() for x, t in c.items()}
    for x in ("q", "k", "v"):
        gpu[x] = wide_rows(c[x].flatten(2), k["pad"]).unflatten(-1, c[x].shape[2:])
    return k, gpu, cu, c


def lin_ref(k, c):
    def flat(t):
        return np64(t).reshape(-1, *t.shape[2:])
    with np.errstate(over="ignore", invalid="ignore"):
        return layer.lin(flat(c["q"]), flat(c["k"]), flat(c["v"]), opt64(c["decay"]), k["scale"] or k["K"] ** -0.5,
                         opt64(c["h0"]), k["starts"], flat(c["do"]), opt64(c["dht"]))


def problem(k, c, cu):
    import chunkwise_delta_rule_gb300 as kda
    return kda.make_lin_problem(c["q"], c["k"], c["v"], c["decay"], scale=k["scale"], initial_state=c["h0"], cu_seqlens=cu)


LENGTHS = [0, 1, 2, 0, 130, 64, 5, 0, 257, 128, 3, 0]
CASES = [dict(io=io, B=2, T=T, H=2, K=64, V=64, state=True) for io in ("bf16", "fp32") for T in (1, 2, 8, 9, 65, 127, 128, 129, 300)]
CASES += [dict(io=io, B=1, T=77, H=2, HV=HV, K=K, V=V, state=True) for io in ("bf16", "fp32") for HV, K, V in (
    (2, 1, 1), (4, 5, 3), (2, 40, 72), (2, 64, 128), (6, 128, 64), (2, 128, 128), (2, 128, 136), (2, 128, 256), (4, 136, 8),
    (2, 192, 160), (2, 256, 256), (2, 8, 8), (2, 16, 250))]
CASES += [dict(io=io, B=1, H=2, HV=4, K=64, V=72, state=s, lengths=LENGTHS) for io in ("bf16", "fp32") for s in (True, False)]
CASES += [dict(io=io, B=1, H=3, K=128, V=128, state=True, lengths=[700, 1, 0, 33]) for io in ("bf16", "fp32")]
CASES += [dict(io="bf16", B=3, T=150, H=2, K=64, V=64, pad=p) for p in (64, 8, 3)]
CASES += [dict(io="fp32", B=3, T=50, H=2, K=12, V=20, pad=p) for p in (4, 1)]
CASES += [dict(io=io, B=2, T=200, H=5, K=64, V=64, state=True, decay=d) for io in ("bf16", "fp32") for d in (None, "strong", "up")]
CASES += [dict(io=io, B=1, T=2100, H=1, K=64, V=64, state=True) for io in ("bf16", "fp32")]          # time windows
CASES += [dict(io=io, B=1, H=1, HV=2, K=40, V=24, state=True, lengths=[3, 1500, 0, 2, 640, 129]) for io in ("bf16", "fp32")]
CASES += [dict(io="bf16", B=1, T=T, H=1, HV=HV, K=K, V=V, state=True) for T, HV, K, V in ((4500, 1, 128, 128), (1000, 2, 120, 104), (513, 1, 72, 200))]
CASES += [dict(io="bf16", B=2, T=200, H=2, K=64, V=64, scale=0.3), dict(io="fp32", B=4, T=0, H=2, K=8, V=8, state=True)]


@pytest.mark.parametrize("kw", CASES, ids=str)
def test_matches_oracle(kw):
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(kw, 21)
    p = problem(k, g, cu)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, ht = kda.kda_lin_fwd(p, err=err)
    r = kda.kda_lin_bwd(p, g["do"], g["dht"], need_dh0=True, err=err)
    assert int(err) == 0
    ref = lin_ref(k, c)
    got = dict(o=o, ht=ht, dq=r.dq, dk=r.dk, dv=r.dv, dh0=r.dh0)
    for n, t in got.items():
        check_close(n, np64(t).reshape(ref[n].shape), ref[n], tol(t))


@pytest.mark.parametrize("kw", [dict(io="bf16", B=2, T=300, H=2, K=64, V=64), dict(io="bf16", B=1, T=2100, H=1, HV=2, K=128, V=128),
                                dict(io="bf16", B=1, H=2, K=64, V=72, lengths=LENGTHS), dict(io="fp32", B=1, T=900, H=1, K=40, V=24)], ids=str)
def test_without_states(kw):
    """Calls that return no state: outputs and gradients as with one."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(kw, state=True), 37)
    p = problem(k, g, cu)
    ref = lin_ref(k, c)
    o, ht = kda.kda_lin_fwd(p, output_final_state=False)
    r = kda.kda_lin_bwd(p, g["do"], g["dht"], need_dh0=False)
    assert ht is None and r.dh0 is None
    for n, t in dict(o=o, dq=r.dq, dk=r.dk, dv=r.dv).items():
        check_close(n, np64(t).reshape(ref[n].shape), ref[n], tol(t))


@pytest.mark.parametrize("kw", [CASES[0], CASES[8], CASES[-4], CASES[-3], CASES[44]], ids=str)
def test_state_in_place(kw):
    """Every window and sequence reads the initial states, whatever the call has written."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, _ = lin_case(dict(kw, state=True), 22)
    o, ht = kda.kda_lin_fwd(problem(k, g, cu))
    h = g["h0"].clone()
    o2, h2 = kda.kda_lin_fwd(problem(k, dict(g, h0=h), cu), ht=h)
    assert h2.data_ptr() == h.data_ptr() and torch.equal(h, ht) and torch.equal(o, o2)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (40, 24)])
def test_token_by_token_is_one_call(io, K, V):
    """300 tokens in one call, in two, and one after the other."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, _, c = lin_case(dict(io=io, B=2, T=300, H=2, K=K, V=V, state=True), 23)
    ref = lin_ref(k, c)
    for cuts in ([0, 300], [0, 133, 300], list(range(301))):
        h, outs = g["h0"].clone(), []
        for lo, hi in zip(cuts[:-1], cuts[1:]):
            p = kda.make_lin_problem(*(g[n][:, lo:hi] if hi - lo == 300 else g[n][:, lo:hi].contiguous() for n in ("q", "k", "v")),
                                     g["decay"], initial_state=h)
            outs.append(kda.kda_lin_fwd(p, ht=h)[0])
        check_close("o", np64(torch.cat(outs, 1)).reshape(ref["o"].shape), ref["o"], tol(outs[0]))
        check_close("ht", np64(h), ref["ht"], 1e-5)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_repeated_calls_agree_bitwise(io):
    import chunkwise_delta_rule_gb300 as kda
    for kw in (dict(io=io, B=1, T=1100, H=1, HV=2, K=64, V=64, state=True), dict(io=io, B=1, H=2, HV=4, K=64, V=72, lengths=LENGTHS)):
        k, g, cu, _ = lin_case(kw, 24)
        p = problem(k, g, cu)
        first = None
        for _ in range(3):
            now = [*kda.kda_lin_fwd(p), *kda.kda_lin_bwd(p, g["do"], g["dht"])]
            now = [t for t in now if t is not None]
            assert first is None or all(torch.equal(a, b) for a, b in zip(first, now))
            first = now


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_sequence_does_not_reach_its_neighbours(io, bad):
    """What a sequence holds stays in it: sequences that end inside tiles lie beside ones full of NaN or infinities."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=1, H=2, K=64, V=64, state=True, lengths=[70, 200, 9, 130, 1, 64]), 25)
    ref = lin_ref(k, c)
    s = k["starts"]
    for n in ("q", "k", "v", "do"):
        for i in (1, 3, 5):
            g[n][:, s[i]:s[i + 1]] = bad
    p = problem(k, g, cu)
    o, ht = kda.kda_lin_fwd(p)
    r = kda.kda_lin_bwd(p, g["do"], g["dht"])
    for n, t in dict(o=o, dq=r.dq, dk=r.dk, dv=r.dv).items():
        for i in (0, 2, 4):
            check_close(n, np64(t)[0, s[i]:s[i + 1]], ref[n][s[i]:s[i + 1]], tol(t))
    for n, t in dict(ht=ht, dh0=r.dh0).items():
        check_close(n, np64(t)[::2], ref[n][::2], 1e-5)


@pytest.mark.parametrize("cu", [[0, 50, 30, 100], [5, 50, 60, 100], [0, 50, 60, 99], [0, 200, -7, 100], [100, 100, 100, 100]])
@pytest.mark.parametrize("times", [1, 25])     # in one window, and in several
def test_inconsistent_offsets_are_reported(cu, times):
    import chunkwise_delta_rule_gb300 as kda
    for io in ("bf16", "fp32"):
        k, g, _, _ = lin_case(dict(io=io, B=1, H=2, K=64, V=64, state=True, lengths=[30 * times, 40 * times, 30 * times]), 26)
        p = problem(k, g, torch.tensor(cu, dtype=torch.int32, device="cuda") * times)
        err = torch.zeros(2, dtype=torch.int32, device="cuda")
        kda.kda_lin_fwd(p, err=err[:1])
        kda.kda_lin_bwd(p, g["do"], g["dht"], err=err[1:])
        assert err.tolist() == [1, 1]


def test_a_decay_does_not_drift():
    """A state that only decays is the decay's power: to 2^-24 a step of rounding, whatever the number of tokens."""
    import chunkwise_delta_rule_gb300 as kda
    d = -torch.exp2(-torch.arange(1, 13.0, device="cuda"))
    for io in ("bf16", "fp32"):
        for T in (1, 7, 600, 1300):
            z = torch.zeros(1, T, 12, 64, dtype=DT[io], device="cuda")
            p = kda.make_lin_problem(z, z, z, d, initial_state=torch.ones(1, 12, 64, 64, device="cuda"))
            ht = kda.kda_lin_fwd(p)[1]
            want = np.exp(np64(d) * T).reshape(1, 12, 1, 1)
            keep = want[0, :, 0, 0] > 1e-30
            off = np.abs(np64(ht) / want - 1)[:, keep]
            assert np.max(off) <= 2.0 ** -24 * (T / 8 + 4), (io, T, np.max(off))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_autograd(io):
    """Gradients through the function: the formula's, and without a final state's gradient or a state."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=1, H=2, HV=4, K=64, V=72, state=True, lengths=LENGTHS), 27)
    ref = lin_ref(k, c)
    leaves = [g[n].detach().requires_grad_() for n in ("q", "k", "v", "h0")]
    o, ht = kda.linear_attention(*leaves[:3], g["decay"], initial_state=leaves[3], cu_seqlens=cu)
    torch.autograd.backward([o, ht], [g["do"], g["dht"]])
    for n, t in zip(("dq", "dk", "dv", "dh0"), leaves):
        check_close(n, np64(t.grad).reshape(ref[n].shape), ref[n], tol(t))
    ref = lin_ref(k, dict(c, h0=None, dht=None))
    q = g["q"].detach().requires_grad_()
    kda.linear_attention(q, g["k"], g["v"], g["decay"], cu_seqlens=cu)[0].backward(g["do"])
    check_close("dq", np64(q.grad).reshape(ref["dq"].shape), ref["dq"], tol(q))
    with pytest.raises(RuntimeError, match="the decay has no gradient"):
        kda.linear_attention(q, g["k"], g["v"], g["decay"].clone().requires_grad_(), cu_seqlens=cu)[0].sum().backward()
    dq = torch.autograd.grad(kda.linear_attention(q, g["k"], g["v"], cu_seqlens=cu)[0].float().square().sum(), q, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        dq.float().sum().backward()


def test_gradients_are_the_slopes_of_the_loss():
    """fp32, central differences of <do, o> + <dht, ht> along random directions. The loss is linear in each of q, k (to
    second order the product of both), v and h0 along one of them, so a step of 2^-4 has no truncation; its value, of
    some 100, is summed in 64 bits of outputs that are off by 1e-6 of their norm."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, _ = lin_case(dict(io="fp32", B=1, H=2, HV=4, K=24, V=40, state=True, lengths=[9, 0, 140, 1]), 28)
    r = kda.kda_lin_bwd(problem(k, g, cu), g["do"], g["dht"])

    def loss(**kw):
        o, ht = kda.kda_lin_fwd(problem(k, dict(g, **kw), cu))
        return (o.double() * g["do"].double()).sum() + (ht.double() * g["dht"].double()).sum()

    size = (loss().abs() + g["do"].double().norm() * kda.kda_lin_fwd(problem(k, g, cu))[0].double().norm()).item()
    for n, grad in (("q", r.dq), ("k", r.dk), ("v", r.dv), ("h0", r.dh0)):
        d = torch.randn(g[n].shape, generator=gen_of(29)).cuda()
        h = 2.0 ** -4
        slope = (loss(**{n: g[n] + h * d}) - loss(**{n: g[n] - h * d})).item() / (2 * h)
        want = (grad.double() * d.double()).sum().item()
        assert abs(slope - want) <= 1e-6 * size / h, (n, slope, want)


# ------------------------------------------------------------------ callers

def test_graph_replay_with_new_inputs():
    import chunkwise_delta_rule_gb300 as kda
    for kw in (dict(io="bf16", B=2, T=300, H=2, K=64, V=64, state=True), dict(io="bf16", B=4, T=1, H=2, K=64, V=64, state=True),
               dict(io="fp32", B=1, T=900, H=1, HV=2, K=40, V=24, state=True)):
        k, g, cu, _ = lin_case(kw, 30)
        p = problem(k, g, cu)

        def call():
            return [*kda.kda_lin_fwd(p), *kda.kda_lin_bwd(p, g["do"], g["dht"])]

        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call()
        for seed in (31, 32):
            new = lin_case(kw, seed)[1]
            for n in ("q", "k", "v", "h0", "do", "dht"):
                g[n].copy_(new[n])
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, call()))


def test_two_streams_at_once():
    """Calls on several streams with buffers of their own do not meet."""
    import chunkwise_delta_rule_gb300 as kda
    cases = [lin_case(dict(io=io, B=1, T=1500, H=1, K=64, V=64, state=True), s) for io, s in (("bf16", 33), ("bf16", 34), ("fp32", 35))]
    want = [kda.kda_lin_bwd(problem(k, g, cu), g["do"], g["dht"]) for k, g, cu, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[kda.kda_lin_bwd(problem(k, g, cu), g["do"], g["dht"], stream=s) for (k, g, cu, _), s in zip(cases, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for row in got:
        assert all(torch.equal(a, b) for x, y in zip(row, want) for a, b in zip(x, y))


def test_refusals_of_otherwise_valid_calls():
    """One property off at a time."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, _, _ = lin_case(dict(io="bf16", B=2, T=10, H=2, HV=4, K=16, V=24, state=True), 36)

    def make(**kw):
        a = dict(g, **kw)
        return kda.make_lin_problem(a["q"], a["k"], a["v"], a["decay"], initial_state=a["h0"], cu_seqlens=kw.get("cu"),
                                    scale=kw.get("scale"))

    p = make()
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    for name, kw in (("k must be", dict(k=g["k"].float())), ("k must be", dict(k=g["k"][:, :, :1])), ("v must be", dict(v=g["v"].float())),
                     ("v must be", dict(v=g["v"][:1])), ("decay must be", dict(decay=g["decay"][:2])),
                     ("decay must be", dict(decay=g["decay"].double())), ("decay must be", dict(decay=g["decay"].cpu())),
                     ("initial_state must be", dict(h0=g["h0"].bfloat16())), ("initial_state must be", dict(h0=g["h0"][:1])),
                     ("scale must be", dict(scale=0.0)), ("scale must be", dict(scale=-1.0)), ("scale must be", dict(scale=float("nan"))),
                     ("scale must be", dict(scale=1e39)), ("packed sequences need B == 1", dict(cu=cu)),
                     ("q's rows must be dense", dict(q=torch.zeros(2, 10, 2, 32, dtype=torch.bfloat16, device="cuda")[..., ::2]))):
        with pytest.raises(ValueError, match=name):
            make(**kw)
    with pytest.raises(_lib_error(), match="HV must be a multiple of H"):
        kda.kda_lin_fwd(make(v=g["v"][:, :, :3].contiguous(), decay=g["decay"][:3].contiguous(), h0=g["h0"][:, :3].contiguous()))
    with pytest.raises(ValueError, match="do must be"):
        kda.kda_lin_bwd(p, g["do"].float())
    with pytest.raises(ValueError, match="dht must be"):
        kda.kda_lin_bwd(p, g["do"], g["dht"][:1])
    with pytest.raises(ValueError, match="ht must be"):
        kda.kda_lin_fwd(p, ht=g["h0"].transpose(2, 3))
    with pytest.raises(ValueError, match="err must be"):
        kda.kda_lin_fwd(p, err=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="workspace must be"):
        kda.kda_lin_bwd(p, g["do"], workspace=torch.empty(1 << 20, dtype=torch.uint8))


def _lib_error():
    from chunkwise_delta_rule_gb300 import _lib
    return _lib.KdaError
