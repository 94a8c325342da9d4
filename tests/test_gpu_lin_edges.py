"""Linear attention where its calls split into time windows, where its states and
widths keep it from its widest accesses, and what a token that is not finite
reaches. Which kernels a call launches is read off the library's own tracing, so
that a change of the rules that choose them cannot leave a test without its path."""

import ctypes

import numpy as np
import pytest
import torch

from tests.helpers import check_close, np64
from tests.test_gpu_layer import DT
from tests.test_gpu_lin import lin_case, lin_ref, problem, tol

pytestmark = pytest.mark.gpu


class KernelTime(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double)]


def launched(call):
    """The call's result and the names of the library's kernels that it launched."""
    from chunkwise_delta_rule_gb300 import _lib
    lib = _lib.load()
    lib.kda_profile_end.argtypes = [ctypes.POINTER(KernelTime), ctypes.c_int]
    lib.kda_profile_begin()
    try:
        r = call()
    finally:
        arr = (KernelTime * 32)()
        n = lib.kda_profile_end(arr, 32)
    assert n >= 0
    return r, {arr[i].name.decode() for i in range(n)}


TC, CORES = {"k_lin_tc_windows", "k_lin_join", "k_lin_tc"}, {"k_lin_windows", "k_lin_join", "k_lin"}
# cut into windows on the tensor cores, forwards and backwards, and on the CUDA cores
WINDOWS = [(dict(io="bf16", B=1, T=2100, H=1, K=64, V=64, state=True), TC),
           (dict(io="bf16", B=1, T=4500, H=1, K=128, V=128, state=True), TC),
           (dict(io="bf16", B=2, T=2600, H=1, HV=2, K=64, V=72, state=True), TC),
           (dict(io="bf16", B=1, H=1, HV=2, K=40, V=24, state=True, lengths=[3, 1500, 0, 2, 640, 129]), TC),
           (dict(io="fp32", B=1, T=2100, H=1, K=64, V=64, state=True), CORES),
           (dict(io="fp32", B=1, H=1, HV=2, K=40, V=24, state=True, lengths=[3, 1500, 0, 2, 640, 129]), CORES)]


@pytest.mark.parametrize("kw,kernels", WINDOWS, ids=str)
def test_windows_against_the_oracle_and_in_place(kw, kernels):
    """Outputs, states and gradients of calls in windows, the same with the final states written over the initial ones, and
    three times the same bits."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(kw, 71)
    p = problem(k, g, cu)
    (o, ht), names = launched(lambda: kda.kda_lin_fwd(p))
    assert names == kernels
    r, names = launched(lambda: kda.kda_lin_bwd(p, g["do"], g["dht"]))
    assert names - {"k_lin_heads"} == kernels and ("k_lin_heads" in names) == (k["HV"] not in (None, k["H"]))
    ref = lin_ref(k, c)
    for n, t in dict(o=o, ht=ht, dq=r.dq, dk=r.dk, dv=r.dv, dh0=r.dh0).items():
        check_close(n, np64(t).reshape(ref[n].shape), ref[n], tol(t))
    for _ in range(2):
        h = g["h0"].clone()
        (o2, h2), names = launched(lambda: kda.kda_lin_fwd(problem(k, dict(g, h0=h), cu), ht=h))
        assert names == kernels and h2.data_ptr() == h.data_ptr() and torch.equal(h, ht) and torch.equal(o, o2)
        again = kda.kda_lin_bwd(p, g["do"], g["dht"])
        assert all(torch.equal(a, b) for a, b in zip(r, again))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("decay", [None, "strong", "up"])
@pytest.mark.parametrize("lengths", [None, [1, 800, 0, 129, 1170]], ids=["one", "packed"])
def test_windows_of_other_decays(io, decay, lengths):
    """No decay, decays down to -infinity and growing states through joined windows, whole and partial."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=1, T=0 if lengths else 2100, H=5, K=64, V=64, state=True, decay=decay, lengths=lengths), 70)
    p = problem(k, g, cu)
    (o, ht), names = launched(lambda: kda.kda_lin_fwd(p))
    assert names == (TC if io == "bf16" else CORES)
    r = kda.kda_lin_bwd(p, g["do"], g["dht"])
    ref = lin_ref(k, c)
    for n, t in dict(o=o, ht=ht, dq=r.dq, dk=r.dk, dv=r.dv, dh0=r.dh0).items():
        check_close(n, np64(t).reshape(ref[n].shape), ref[n], tol(t))


def test_windows_on_streams_and_in_graphs():
    """Windows' states lie in workspaces: calls on several streams at once, and replays of two graphs, keep their own."""
    import chunkwise_delta_rule_gb300 as kda
    cases = [lin_case(WINDOWS[i][0], s) for i, s in ((1, 72), (3, 73), (4, 74))]

    def call(case, stream=None):
        k, g, cu, _ = case
        p = problem(k, g, cu)
        return [*kda.kda_lin_fwd(p, stream=stream), *kda.kda_lin_bwd(p, g["do"], g["dht"], stream=stream)]

    want = [call(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[call(c, s) for c, s in zip(cases, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for row in got:
        assert all(torch.equal(a, b) for x, y in zip(row, want) for a, b in zip(x, y))
    graphs = []
    for c in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(c)
        graphs.append((graph, out))
    for seeds in ((75, 76, 77), (78, 79, 80)):
        for c, i, s in zip(cases, (1, 3, 4), seeds):
            new = lin_case(WINDOWS[i][0], s)[1]
            for n in ("q", "k", "v", "h0", "do", "dht"):
                c[1][n].copy_(new[n])
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for c, (_, out) in zip(cases, graphs):
            assert all(torch.equal(a, b) for a, b in zip(out, call(c)))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_windows_keep_sequences_apart(io):
    """Sequences of several windows full of NaN, beside clean ones that share windows with their ends."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=1, H=1, HV=2, K=64, V=64, state=True, lengths=[70, 900, 450, 1300, 1, 64]), 81)
    ref = lin_ref(k, c)
    s = k["starts"]
    for n in ("q", "k", "v", "do"):
        for i in (1, 3):
            g[n][:, s[i]:s[i + 1]] = float("nan")
    p = problem(k, g, cu)
    (o, ht), names = launched(lambda: kda.kda_lin_fwd(p))
    assert names == (TC if io == "bf16" else CORES)
    r = kda.kda_lin_bwd(p, g["do"], g["dht"])
    keep = (0, 2, 4, 5)
    for n, t in dict(o=o, dq=r.dq, dk=r.dk, dv=r.dv).items():
        for i in keep:
            check_close(n, np64(t)[0, s[i]:s[i + 1]], ref[n][s[i]:s[i + 1]], tol(t))
    for n, t in dict(ht=ht, dh0=r.dh0).items():
        check_close(n, np64(t)[list(keep)], ref[n][list(keep)], 1e-5)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_what_a_token_reaches(io):
    """A NaN in a token's key and value reaches its own and all later outputs and the final state; on the tensor cores
    earlier outputs of the same chunk of 128 too, and none before. Backwards in time the same holds for a query and an
    output's gradient, chunks counted from the end; outputs and dq of other tokens do not see those."""
    import chunkwise_delta_rule_gb300 as kda
    T, at = 600, 300
    first, behind = (256, T - 2 * 128) if io == "bf16" else (at, at + 1)     # the chunk's first token; from the end, the first behind it
    k, g, cu, c = lin_case(dict(io=io, B=1, T=T, H=2, K=64, V=64, state=True), 82)
    ref = lin_ref(k, c)
    bad = dict(g, k=g["k"].clone(), v=g["v"].clone())
    bad["k"][:, at], bad["v"][:, at] = float("nan"), float("nan")
    o, ht = kda.kda_lin_fwd(problem(k, bad, cu))
    check_close("o", np64(o)[0, :first], ref["o"][:first], tol(o))
    assert torch.isnan(o[:, at:]).all() and torch.isnan(ht).all()
    bad = dict(g, q=g["q"].clone(), do=g["do"].clone())
    bad["q"][:, at], bad["do"][:, at] = float("nan"), float("nan")
    p = problem(k, bad, cu)
    o, ht = kda.kda_lin_fwd(p)
    r = kda.kda_lin_bwd(p, bad["do"], g["dht"])
    others = np.arange(T) != at
    check_close("o", np64(o)[0, others], ref["o"][others], tol(o))
    check_close("ht", np64(ht), ref["ht"], 1e-5)
    check_close("dq", np64(r.dq)[0, others], ref["dq"][others], tol(r.dq))
    for n, t in dict(dk=r.dk, dv=r.dv).items():
        check_close(n, np64(t)[0, behind:], ref[n][behind:], tol(t))
        assert torch.isnan(t[:, :at + 1]).all()
    assert torch.isnan(r.dh0).all()


def off_by_one(t):
    """The same values, contiguous, from an address 4 bytes behind a multiple of 16."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    flat[1:].copy_(t.flatten())
    return flat[1:].view(t.shape)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 9, 200, 2100])
def test_states_off_16_bytes(io, T):
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=1, T=T, H=1, HV=2, K=64, V=128, state=True), 83)
    ref = lin_ref(k, c)
    a = dict(g, h0=off_by_one(g["h0"]), dht=off_by_one(g["dht"]))
    assert a["h0"].data_ptr() % 16 == 4
    ht = off_by_one(torch.zeros_like(g["h0"]))
    o, _ = kda.kda_lin_fwd(problem(k, a, cu), ht=ht)
    r = kda.kda_lin_bwd(problem(k, a, cu), g["do"], a["dht"])
    h = a["h0"]
    o2, _ = kda.kda_lin_fwd(problem(k, a, cu), ht=h)      # in place
    assert torch.equal(o, o2) and torch.equal(h, ht)
    for n, t in dict(o=o, ht=ht, dq=r.dq, dk=r.dk, dv=r.dv, dh0=r.dh0).items():
        check_close(n, np64(t).reshape(ref[n].shape), ref[n], tol(t))


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V", [(136, 64), (256, 256), (64, 66), (128, 7), (130, 5), (1, 1)])
def test_single_tokens_of_other_widths(io, K, V):
    """Widths that the single tokens' kernel does not take: three tokens one by one, the states in place."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=3, T=3, H=2, HV=4, K=K, V=V, state=True), 84)
    ref = lin_ref(k, c)
    h, outs = g["h0"].clone(), []
    for t in range(3):
        p = kda.make_lin_problem(*(g[n][:, t:t + 1] for n in ("q", "k", "v")), g["decay"], initial_state=h)
        (o, _), names = launched(lambda: kda.kda_lin_fwd(p, ht=h))
        assert names == {"k_lin"}
        outs.append(o)
    check_close("o", np64(torch.cat(outs, 1)).reshape(ref["o"].shape), ref["o"], tol(outs[0]))
    check_close("ht", np64(h), ref["ht"], 1e-5)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("H,lengths,forward,backward", [
    (2, [1] * 10 + [900] + [1] * 7, True, True), (2, [1] * 20 + [900, 0, 1], False, True), (2, [1] * 100 + [900, 0, 1], False, False),
    (2, [48] * 5, True, True), (2, [47] * 5, False, True), (2, [24] * 5, False, True), (2, [23] * 5, False, False), (2, [1] * 70, False, False),
    (64, [1, 30, 0, 33], True, True), (64, [15] * 3, False, True), (64, [9] * 3, False, False)])
def test_packed_mixes(io, H, lengths, forward, backward):
    """Mixes of a serving step, and both sides of the mean lengths from which packed calls of few and of many heads take the
    tensor cores."""
    import chunkwise_delta_rule_gb300 as kda
    k, g, cu, c = lin_case(dict(io=io, B=1, H=H, HV=H, K=64, V=64, state=True, lengths=lengths), 85)
    ref = lin_ref(k, c)
    p = problem(k, g, cu)
    r, names = launched(lambda: kda.kda_lin_bwd(p, g["do"], g["dht"]))
    assert ("k_lin_tc" in names) == (io == "bf16" and backward)
    h = g["h0"].clone()
    (o, _), names = launched(lambda: kda.kda_lin_fwd(problem(k, dict(g, h0=h), cu), ht=h))
    assert ("k_lin_tc" in names) == (io == "bf16" and forward)
    for n, t in dict(o=o, ht=h, dq=r.dq, dk=r.dk, dv=r.dv, dh0=r.dh0).items():
        check_close(n, np64(t).reshape(ref[n].shape), ref[n], tol(t))


def step_bound(steps):
    """A state that only decays is rounded once a step, by at most 2^-24 of it with a sign of its own: eight standard
    deviations of a sum of `steps` of them, and 4 for the powers and their products themselves."""
    return 2.0 ** -24 * (8 * (steps / 3) ** 0.5 + 4)


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [33, 100, 127])
def test_a_decay_does_not_drift_over_calls(io, T):
    """A state carried through 400 calls of T tokens, each a partial chunk on the tensor cores."""
    import chunkwise_delta_rule_gb300 as kda
    calls = 400
    d = -torch.exp2(-torch.arange(9, 17.0, device="cuda"))
    z = torch.zeros(1, T, 8, 64, dtype=DT[io], device="cuda")
    h = torch.ones(1, 8, 64, 64, device="cuda")
    p = kda.make_lin_problem(z, z, z, d, initial_state=h)
    names = launched(lambda: kda.kda_lin_fwd(p, ht=h))[1]
    assert ("k_lin_tc" in names) == (io == "bf16")
    for _ in range(calls - 1):
        kda.kda_lin_fwd(p, ht=h)
    want = np.exp(np64(d) * T * calls).reshape(1, 8, 1, 1)
    keep = want[0, :, 0, 0] > 1e-30
    assert keep.sum() >= 7
    off = np.max(np.abs(np64(h) / want - 1)[:, keep])
    assert off <= step_bound(calls * (1 if io == "bf16" else -(-T // 8))), off * 2 ** 24


@pytest.mark.parametrize("io", ["bf16", "fp32"])
def test_a_decay_does_not_drift_over_windows(io):
    """A state carried through the windows of one long row; backwards in time the same of a final state's gradient."""
    import chunkwise_delta_rule_gb300 as kda
    T = 32768
    z = torch.zeros(1, T, 1, 64, dtype=DT[io], device="cuda")
    ones = torch.ones(1, 1, 64, 64, device="cuda")
    for e in range(9, 17):
        d = torch.full((1,), -2.0 ** -e, device="cuda")
        p = kda.make_lin_problem(z, z, z, d, initial_state=ones)
        (_, ht), names = launched(lambda: kda.kda_lin_fwd(p))
        assert names == (TC if io == "bf16" else CORES)
        dh0 = kda.kda_lin_bwd(p, z, ones).dh0
        want = np.exp(-2.0 ** -e * T)
        for n, t in (("ht", ht), ("dh0", dh0)):
            off = np.max(np.abs(np64(t) / want - 1))
            assert off <= step_bound(96 if io == "bf16" else 288), (n, e, off * 2 ** 24)
