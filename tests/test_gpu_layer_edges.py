"""GPU tests of the layer operators where their callers differ from the ordinary
ones: rows of unlike alignment, streams, buffers and refusals. Oracle and
tolerances as in test_gpu_layer."""

import numpy as np
import pytest
import torch

from chunkwise_delta_rule_gb300 import _lib
from oracle import layer
from tests.helpers import check_close, np64
from tests.test_gpu_layer import gen_of, scan_case, scan_problem, tol, wide_rows

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


# ------------------------------------------------------------------ streams

def busy():
    """About 20 ms of the current stream."""
    torch.cuda._sleep(40_000_000)


def stream_calls(kda):
    """name -> a call on a given stream (None: the current one) that makes its own outputs and workspace."""
    from tests.test_gpu_layer import conv_case, norm_case
    k, s, _, _ = scan_case(dict(io="fp32", B=1, T=2100, D=8, S=16, state=True), 72)      # in time pieces
    _, c, _, _ = conv_case(dict(io="fp32", B=2, T=600, D=48, W=4, state=True), 73)
    x, r, w, dy = norm_case("fp32", 300, 1000, 74)
    p0, p1 = scan_problem(k, s, None, 0), scan_problem(k, s, None, 1)
    pc = kda.make_conv_problem(c["x"], c["w"], c["bias"], initial_state=c["h0"])
    pn, pq = kda.make_norm_problem(x, w), kda.make_norm_problem(x, w, residual=r, out="e4m3", group=128)
    saved = kda.kda_ssm_fwd(p1)[2]
    return {"ssm_fwd": lambda st: kda.kda_ssm_fwd(p1, stream=st), "ssm_bwd": lambda st: kda.kda_ssm_bwd(p0, s["dy"], s["dht"], stream=st),
            "ssm_bwd_saved": lambda st: kda.kda_ssm_bwd(p1, s["dy"], s["dht"], saved=saved, stream=st),
            "conv_fwd": lambda st: kda.kda_conv_fwd(pc, stream=st),
            "conv_bwd": lambda st: kda.kda_conv_bwd(pc, c["dy"], c["df"], stream=st),
            "norm_fwd": lambda st: kda.kda_norm_fwd(pq, stream=st), "norm_bwd": lambda st: kda.kda_norm_bwd(pn, dy, stream=st)}


def tensors(out):
    return [t.float() for t in out if t is not None]


@pytest.mark.parametrize("name", ["ssm_fwd", "ssm_bwd", "ssm_bwd_saved", "conv_fwd", "conv_bwd", "norm_fwd", "norm_bwd"])
def test_a_given_stream_owns_what_the_call_allocates(name):
    """A call on a busy side stream: its workspace and outputs lie neither in blocks that earlier work of the current
    stream still writes, nor in blocks that its later tensors get; outputs dropped by the current stream are not given
    to the side stream's next call while they are still read."""
    import chunkwise_delta_rule_gb300 as kda
    call = stream_calls(kda)[name]
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    sizes = [1 << b for b in range(9, 23)] + [256 * i for i in range(1, 400, 7)]
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    # blocks that the current stream has freed but not finished with
    busy()
    late = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
    del late
    got = call(side)                         # side does not wait for them
    side.synchronize()
    first = [t.clone() for t in tensors(got)]
    # later tensors of the current stream, while the side stream is still to run
    with torch.cuda.stream(side):
        busy()
    got2 = call(side)
    later = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
    main.wait_stream(side)
    second = [t.clone() for t in tensors(got2)]
    # outputs dropped while the current stream is still to read them
    busy()
    third = [t.clone() for t in tensors(got2)]
    del got2
    with torch.cuda.stream(side):
        again = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes]
    torch.cuda.synchronize()
    del later, again
    for got in (first, second, third):
        assert all(torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) for a, b in zip(got, want))


# ------------------------------------------------------------------ refusals

def test_tensors_of_another_device_are_refused():
    """Every tensor of a call, buffers included, lies on x's device."""
    import chunkwise_delta_rule_gb300 as kda
    from tests.test_gpu_layer import conv_case, norm_case
    k, s, _, _ = scan_case(dict(io="fp32", B=1, T=2100, D=8, S=16, state=True), 75)
    p, ps = scan_problem(k, s, None), scan_problem(k, s, None, 1)
    n = max(kda.kda_ssm_workspace_size(p, b) for b in (False, True))
    host = torch.empty(n, dtype=torch.uint8)
    spread = torch.empty(256, dtype=torch.uint8, device="cuda").expand(-(-n // 256), 256)   # n bytes in 256 places
    for ws in (host, spread):
        with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
            kda.kda_ssm_fwd(p, workspace=ws)
        with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
            kda.kda_ssm_bwd(p, s["dy"], s["dht"], workspace=ws)
        with pytest.raises(ValueError, match="saved must be a contiguous CUDA tensor"):
            kda.kda_ssm_fwd(ps, saved=ws)
    saved = torch.empty(kda.kda_ssm_saved_size(ps), dtype=torch.uint8)
    with pytest.raises(ValueError, match="saved must be a contiguous CUDA tensor"):
        kda.kda_ssm_bwd(ps, s["dy"], s["dht"], saved=saved)
    with pytest.raises(ValueError, match="err must be an int32 CUDA tensor"):
        kda.kda_ssm_fwd(p, err=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="dy must be a contiguous CUDA tensor"):
        kda.kda_ssm_bwd(p, s["dy"].cpu(), stream=torch.cuda.Stream())
    with pytest.raises(ValueError, match="d_skip must be a contiguous CUDA tensor"):
        scan_problem(k, dict(s, d_skip=s["d_skip"].cpu()), None)
    _, c, _, _ = conv_case(dict(io="bf16", B=2, T=70, D=64, W=4, state=True), 76)
    pc = kda.make_conv_problem(c["x"], c["w"], c["bias"], initial_state=c["h0"])
    ws = torch.empty(kda.kda_conv_workspace_size(pc), dtype=torch.uint8)
    with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
        kda.kda_conv_bwd(pc, c["dy"], workspace=ws)
    with pytest.raises(ValueError, match="final_state must be a contiguous CUDA tensor"):
        kda.kda_conv_fwd(pc, final_state=c["h0"].cpu())
    x, r, w, dy = norm_case("fp32", 4, 64, 77)
    pn = kda.make_norm_problem(x, w)
    with pytest.raises(ValueError, match="workspace must be a contiguous CUDA tensor"):
        kda.kda_norm_bwd(pn, dy, workspace=torch.empty(kda.kda_norm_workspace_size(pn), dtype=torch.uint8))
    with pytest.raises(ValueError, match="residual must be a contiguous CUDA tensor"):
        kda.make_norm_problem(x, w, residual=r.cpu())


def test_refusals_of_otherwise_valid_calls():
    """One property off at a time."""
    import chunkwise_delta_rule_gb300 as kda
    from tests.test_gpu_layer import conv_case, norm_case
    _, c, _, _ = conv_case(dict(io="bf16", B=2, T=10, D=16, W=4, state=True), 79)
    k, s, _, _ = scan_case(dict(io="bf16", B=2, T=10, D=16, S=16, state=True), 79)
    x, r, w, dy = norm_case("fp32", 4, 64, 79)
    long = torch.zeros(2, 10, 32, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 10], dtype=torch.int32, device="cuda")

    def conv(**kw):
        a = dict(x=c["x"], weight=c["w"], bias=c["bias"], initial_state=c["h0"])
        return kda.make_conv_problem(**dict(a, **kw))

    def scan(save=0, **kw):
        return scan_problem(k, dict(s, **kw), None, save)

    conv(), scan()
    with pytest.raises(ValueError, match="x must be a CUDA tensor|x must be"):
        conv(x=c["x"].half())
    with pytest.raises(ValueError, match="weight must be a contiguous"):
        conv(weight=c["w"].bfloat16())
    with pytest.raises(ValueError, match="weight must be a contiguous"):
        conv(weight=c["w"][:8])
    with pytest.raises(ValueError, match="bias must be a contiguous"):
        conv(bias=c["bias"][:8])
    with pytest.raises(ValueError, match="initial_state must be a contiguous"):
        conv(initial_state=c["h0"][:, :2])
    with pytest.raises(ValueError, match="initial_state must be a contiguous"):
        conv(initial_state=c["h0"].float())
    with pytest.raises(ValueError, match="x's rows must be dense"):
        conv(x=long[..., ::2])
    with pytest.raises(ValueError, match="x's tokens must be evenly spaced"):
        conv(x=torch.zeros(2, 12, 16, dtype=torch.bfloat16, device="cuda")[:, :10])
    with pytest.raises(ValueError, match="x's tokens must be evenly spaced"):
        conv(x=c["x"][:, :1].expand(2, 10, 16))
    with pytest.raises(ValueError, match="dt must be a CUDA tensor"):
        scan(dt=s["dt"].float())
    with pytest.raises(ValueError, match="b must be a CUDA tensor|c must be a CUDA tensor"):
        scan(c=s["c"][..., :8])
    with pytest.raises(ValueError, match="z's rows must be dense"):
        scan(z=long[..., ::2])
    with pytest.raises(ValueError, match="A_log must be a contiguous"):
        scan(A_log=s["A_log"].double())
    one = {n: s[n][:1] for n in ("x", "dt", "b", "c", "z")}
    one["h0"] = s["h0"][:1]
    scan_problem(k, dict(s, **one), cu)
    with pytest.raises(ValueError, match="cu_seqlens must be an int32"):
        scan_problem(k, dict(s, **one), cu.long())
    with pytest.raises(ValueError, match="cu_seqlens must be an int32"):
        scan_problem(k, dict(s, **one), cu[:1])
    with pytest.raises(ValueError, match="packed sequences need B == 1"):
        scan_problem(k, s, cu)
    p = scan(1)
    with pytest.raises(ValueError, match="save_policy 1 needs the forward's saved buffer"):
        kda.kda_ssm_bwd(p, s["dy"])
    saved = kda.kda_ssm_fwd(p)[2]
    with pytest.raises(ValueError, match="save_policy 1 needs the forward's saved buffer"):
        kda.kda_ssm_bwd(p, s["dy"], saved=saved[:-1])
    with pytest.raises(ValueError, match="dy must be a contiguous"):
        kda.kda_ssm_bwd(scan(), s["dy"].float())
    with pytest.raises(ValueError, match="dht must be a contiguous"):
        kda.kda_ssm_bwd(scan(), s["dy"], s["dht"][:1])
    with pytest.raises(ValueError, match="ht must be a contiguous"):
        kda.kda_ssm_fwd(scan(), ht=s["h0"].transpose(1, 2))
    with pytest.raises(ValueError, match="x must be a contiguous"):
        kda.make_norm_problem(x[:, ::2], w[:32].contiguous())
    with pytest.raises(ValueError, match="weight must be a contiguous"):
        kda.make_norm_problem(x, w[:32])
    with pytest.raises(ValueError, match="residual must be a contiguous"):
        kda.make_norm_problem(x, w, residual=r.bfloat16())
    with pytest.raises(ValueError, match="h must be a contiguous"):
        kda.kda_norm_fwd(kda.make_norm_problem(x, w, residual=r), h=r[:2])
    with pytest.raises(_lib.KdaError, match="group must be"):
        kda.kda_norm_fwd(kda.make_norm_problem(x, w, out="e4m3", group=48))
    with pytest.raises(ValueError, match="dres must be a contiguous"):
        kda.kda_norm_bwd(kda.make_norm_problem(x, w), dy, r.bfloat16())


def test_sizes_beyond_32_bits_are_refused():
    """They do not fit the C interface; cut to 32 bits they would be other, smaller calls."""
    import chunkwise_delta_rule_gb300 as kda
    n = (1 << 32) + 1
    x = torch.empty(n, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(1, 4, device="cuda")
    with pytest.raises(ValueError, match="B is beyond 32 bits"):
        kda.make_conv_problem(x.view(n, 1, 1), w)
    with pytest.raises(ValueError, match="T is beyond 32 bits"):
        kda.make_conv_problem(x.view(1, n, 1), w)
    with pytest.raises(ValueError, match="T is beyond 32 bits"):
        kda.make_ssm_problem(x.view(1, n, 1), x.view(1, n, 1), w[:, :1].contiguous(), x.view(1, n, 1, 1), x.view(1, n, 1, 1))
    with pytest.raises(ValueError, match="the number of rows is beyond 32 bits"):
        kda.make_norm_problem(x.view(n, 1), w[0, :1].contiguous())
    with pytest.raises(ValueError, match="group is beyond 32 bits"):
        kda.make_norm_problem(x[:64].view(1, 64), torch.ones(64, device="cuda"), out="e4m3", group=(1 << 32) + 32)


# ------------------------------------------------------------------ norm, 8-bit output

def test_norm_8bit_of_the_largest_weights():
    """Groups whose largest value is near the end of fp32's range keep their values, as groups near its start do:
    value ~ scale * e4m3 to half a step."""
    import chunkwise_delta_rule_gb300 as kda
    x = torch.linspace(-1.7, 1.7, 512, device="cuda").repeat(3, 1)
    w = torch.ones(512, device="cuda")
    w[:128], w[128:256], w[256:384] = 1.9e38, 8.6e37, 8.4e37     # on both sides of 2^126
    for group in (128, 0):
        q, scale, _ = kda.kda_norm_fwd(kda.make_norm_problem(x, w, out="e4m3", group=group))
        ref = layer.norm(np64(x), np64(w), None, 1e-6)["y"]
        s = np64(scale.repeat_interleave(group or 512, 1))
        assert torch.isfinite(q.float()).all() and (q.float().abs().amax(1) == 448).all()
        assert np.all(np.abs(np64(q.float()) * s - ref) <= np.maximum(np.abs(ref) / 16, s / 1024) * (1 + 1e-4) + s * 448 * 1e-6)


def test_norm_8bit_values_are_the_nearest_ones():
    """An 8-bit value differs from the nearest one only where the exact quotient lies within the fp32 arithmetic's
    error of the middle between two: eight roundings of 2^-24 (sum, weight, product of the value and of its group's
    largest one, quotient, last product; the root is the same in both), 4.8e-7 of the value."""
    import chunkwise_delta_rule_gb300 as kda
    from tests.test_gpu_layer import norm_case
    x, r, w, _ = norm_case("fp32", 2000, 554, 78)
    for group in (0, 32):
        q, scale, _ = kda.kda_norm_fwd(kda.make_norm_problem(x, w, residual=r, out="e4m3", group=group))
        y = layer.norm(np64(x), np64(w), np64(r), 1e-6)["y"]
        gr = group or 554
        pad = np.zeros((2000, -(-554 // gr) * gr))
        pad[:, :554] = np.abs(y)
        amax = pad.reshape(2000, -1, gr).max(axis=2)
        v = y / np.repeat(amax, gr, axis=1)[:, :554] * 448.0
        step = np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6))) - 3)
        off = np.abs(np64(q.float()) - v) - step / 2       # beyond half a step
        assert np.max(off / np.maximum(np.abs(v), 2.0 ** -6)) <= 4.8e-7


# ------------------------------------------------------------------ scan, decays

@pytest.mark.parametrize("g", [0.35, 0.09, 0.02, 0.006, 0.0015])
def test_decays_do_not_drift(g):
    """A state that only decays is the product of its tokens' decays: an error with a mean grows with the tokens. The
    hardware's 2^x, with the constant that the exponent carries, is off by 1.2e-8 or less on the average at every
    size of exponent; what is random (2.5e-8 a token) and what differs by state (1e-7 of the exponents) averages out
    over 1024 states to 1e-9 a token. So at most 1.5e-8 a token, forward, backward and token by token."""
    import chunkwise_delta_rule_gb300 as kda
    gen = gen_of(81)
    D, S = 64, 16
    for T in (20, int(min(600, 100 / g))):
        A_log = torch.rand(D, S, generator=gen) * 0.5 - 0.25
        dt = ((torch.rand(1, T, D, generator=gen) + 0.5) * (g * np.log(2))).float()
        one = torch.ones(1, D, S, device="cuda")
        zero, bc = torch.zeros(1, T, D, device="cuda"), torch.zeros(1, T, 1, S, device="cuda")
        p = kda.make_ssm_problem(zero, dt.cuda(), A_log.cuda(), bc, bc, dt_softplus=False, initial_state=one)
        want = np.exp(-np.exp(np64(A_log)) * np64(dt).sum(axis=1).reshape(D, 1))
        _, ht, _ = kda.kda_ssm_fwd(p)
        dh0 = kda.kda_ssm_bwd(p, zero, one).dh0
        for t in (ht, dh0):
            drift = np.mean(np64(t)[0] / want - 1) / T
            assert abs(drift) <= 1.5e-8, (T, drift)


@pytest.mark.parametrize("softplus", [True, False])
def test_tokens_of_step_zero_leave_the_state_as_it_is(softplus):
    """Padding inside a row: the decay of a zero step is 1 and nothing is added, to the last bit, over thousands of
    tokens; the adjoint passes through too."""
    import chunkwise_delta_rule_gb300 as kda
    k, c, _, _ = scan_case(dict(io="fp32", B=2, T=3, D=40, S=16, state=True, bias=False, softplus=softplus), 89)
    for T in (6, 2000):
        x, b, cm, z = (torch.randn(2, T, *c[n].shape[2:], device="cuda") for n in ("x", "b", "c", "z"))
        dt = torch.full((2, T, 40), float("-inf") if softplus else 0.0, device="cuda")
        p = kda.make_ssm_problem(x, dt, c["A_log"], b, cm, z=z, dt_softplus=softplus, initial_state=c["h0"])
        assert torch.equal(kda.kda_ssm_fwd(p)[1], c["h0"])
        assert torch.equal(kda.kda_ssm_bwd(p, torch.zeros_like(x), c["dht"]).dh0, c["dht"])


@pytest.mark.parametrize("io", ["bf16", "fp32"])
@pytest.mark.parametrize("S", [16, 20])
def test_decoding_and_prefill_give_the_same_states(io, S):
    """The token-by-token kernel and the tiled one form rates, steps and states by the same operations: bitwise."""
    import chunkwise_delta_rule_gb300 as kda
    k, c, _, _ = scan_case(dict(io=io, B=1, T=6, D=72, S=S, state=True), 82)
    c["A_log"] = c["A_log"] * 3 - 4
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    tokens = kda.kda_ssm_fwd(scan_problem(k, c, None))[1]     # so few tokens are taken one by one
    tiles = kda.kda_ssm_fwd(scan_problem(k, c, cu))[1]        # packed sequences are not
    assert torch.equal(tokens, tiles)


def test_gradient_of_the_rates_sums_long_rows():
    """dA_log of long rows whose terms have one sign, in one piece (160 CTAs). Summed one token after another each of 4096
    addends would be rounded at the whole sum's size, about 0.58 x 64 x 1.7e-8 = 6.3e-7 of it; by tiles of 16 the sums' part
    is (4 + 16) x 0.58 x 1.7e-8 = 2e-7. The terms' own errors with a mean (a decay in three places, 3e-8 each at these
    exponents) add 1e-7, and the roundings of A, the product and the last one 1e-7: 4e-7."""
    import chunkwise_delta_rule_gb300 as kda
    B, T, D, S = 4, 4096, 2560, 4
    gen = torch.Generator(device="cuda").manual_seed(83)

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda") + 0.5

    x, dt, dy, b, c = rand(B, T, D), rand(B, T, D), rand(B, T, D), rand(B, T, 1, S), rand(B, T, 1, S)
    A_log = rand(D, S) - 1.0
    p = kda.make_ssm_problem(x, dt, A_log, b, c, dt_softplus=False, save_policy=1)
    got = kda.kda_ssm_bwd(p, dy, saved=kda.kda_ssm_fwd(p)[2]).dA_log
    A = -torch.exp(A_log.double())
    before = torch.empty(T, B, D, S, dtype=torch.float64, device="cuda")
    h = torch.zeros(B, D, S, dtype=torch.float64, device="cuda")
    for t in range(T):
        before[t] = h
        d = dt[:, t, :, None].double()
        h = torch.exp(d * A) * h + d * x[:, t, :, None].double() * b[:, t].double()
    g, dA = torch.zeros_like(h), torch.zeros_like(h)
    for t in reversed(range(T)):
        d = dt[:, t, :, None].double()
        g = (g + c[:, t].double() * dy[:, t, :, None].double()) * torch.exp(d * A)
        dA += g * before[t] * d
    want = A * dA.sum(0)
    err = float((got.double() - want).norm() / want.norm())
    assert err <= 4e-7, err


PIECES = [
    dict(io="bf16", B=1, T=1500, D=40, S=16, state=True, pad=3),
    dict(io="bf16", B=3, T=900, D=24, S=8, G=2),
    dict(io="fp32", B=2, T=700, D=34, S=6, G=2, state=True, pad=1, skip=False),
    dict(io="bf16", B=1, D=36, S=32, state=True, lengths=[0, 500, 1, 700, 33]),
    dict(io="fp32", B=1, T=600, D=10, S=64, G=2, state=True, gate=False, softplus=False, bias=False),
    dict(io="bf16", B=4, T=333, D=72, S=20, state=True),
    dict(io="fp32", B=1, D=33, S=41, state=True, lengths=[31, 1, 1, 800, 64]),
    dict(io="bf16", B=1, D=24, S=16, state=True, lengths=[1] * 300 + [400] + [1] * 20),
]


@pytest.mark.parametrize("kw", PIECES, ids=lambda kw: "-".join(f"{n}{v}" for n, v in kw.items() if n != "lengths"))
def test_scan_in_time_pieces(kw):
    """Few channels and long rows of every kind that is cut into time pieces: types, states per lane, groups, unaligned
    rows, several rows, packed ones, without gate, skip, bias or softplus; the states in place."""
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, ref = scan_case(kw, 88)
    for save in (0, 1):
        p = scan_problem(k, c, cu, save)
        assert kda.kda_ssm_workspace_size(p, False) > 0      # in pieces
        y, ht, saved = kda.kda_ssm_fwd(p)
        g = kda.kda_ssm_bwd(p, c["dy"], c["dht"], saved=saved, need_dh0=True)
        for name, t in dict(y=y, ht=ht, dx=g.dx, ddt=g.ddt, dA_log=g.dA_log, db=g.db, dc=g.dc, dd_skip=g.dd_skip,
                            dz=g.dz, ddt_bias=g.ddt_bias, dh0=g.dh0).items():
            if t is not None:
                check_close(name, np64(t).reshape(ref[name].shape), ref[name], tol(t, True))
    if c["h0"] is not None:
        c["state"] = c["h0"].clone()
        y2, _, _ = kda.kda_ssm_fwd(scan_problem(k, c, cu, h0="state"), ht=c["state"])
        assert torch.equal(y2, y) and torch.equal(c["state"], ht)


# ------------------------------------------------------------------ autograd

def test_second_derivatives_are_refused():
    """The backwards are kernels without one of their own: a second derivative through them is an error, not a term
    that is missing."""
    import chunkwise_delta_rule_gb300 as kda
    from tests.test_gpu_layer import conv_case, norm_case
    _, c, _, _ = conv_case(dict(io="fp32", B=2, T=20, D=24, W=4), 84)
    _, s, _, _ = scan_case(dict(io="fp32", B=2, T=20, D=24, S=16), 85)
    x, r, w, _ = norm_case("fp32", 6, 200, 86)
    q, k, v = (torch.randn(1, 20, 2, 64, device="cuda") for _ in range(3))
    g, beta = -torch.rand(1, 20, 2, 64, device="cuda"), torch.rand(1, 20, 2, device="cuda")
    calls = [(c["x"], lambda t: kda.short_conv(t, c["w"], c["bias"])[0]),
             (s["x"], lambda t: kda.ssm_scan(t, s["dt"], s["A_log"], s["b"], s["c"], z=s["z"], dt_bias=s["dt_bias"])[0]),
             (x, lambda t: kda.rms_norm(t, w, residual=r)[0]), (v, lambda t: kda.chunk_kda(q, k, t, g, beta)[0])]
    for leaf, f in calls:
        leaf = leaf.clone().requires_grad_(True)
        y = f(leaf)
        grad, = torch.autograd.grad((y * y).sum(), leaf, create_graph=True)   # a first one as ever
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (grad * grad).sum().backward()


@pytest.mark.parametrize("save", [0, 1])
def test_the_backward_and_autograd_report_on_the_error_word(save):
    """The recomputed forward of the backward, the backward itself and the autograd functions set the caller's word (its
    bit for offsets that do not fit: the same word takes the bit of a wait that gave up)."""
    import chunkwise_delta_rule_gb300 as kda
    from tests.test_gpu_layer import conv_case
    bad = torch.tensor([0, 9, 4, 12], dtype=torch.int32, device="cuda")
    k, s, good, _ = scan_case(dict(io="bf16", B=1, D=16, S=16, state=True, lengths=[4, 4, 4]), 87)
    _, c, _, _ = conv_case(dict(io="bf16", B=1, D=16, W=4, state=True, lengths=[4, 4, 4]), 87)
    for cu, want in ((good, 0), (bad, 1)):
        p = scan_problem(k, s, cu, save)
        saved = kda.kda_ssm_fwd(p)[2]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        kda.kda_ssm_bwd(p, s["dy"], s["dht"], saved=saved, err=err)
        assert int(err) == want
        err.zero_()
        x = s["x"].clone().requires_grad_(True)
        y, _ = kda.ssm_scan(x, s["dt"], s["A_log"], s["b"], s["c"], z=s["z"], dt_bias=s["dt_bias"], cu_seqlens=cu,
                            save_policy=save, err=err)
        assert int(err) == want
        err.zero_()
        y.sum().backward()
        assert int(err) == want
        err.zero_()
        kda.short_conv(c["x"], c["w"], c["bias"], cu_seqlens=cu, err=err)
        assert int(err) == want
