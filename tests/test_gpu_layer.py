"""GPU parity of the layer operators (short convolution, selective state space
scan, norm) against their FP64 oracle, and their serving and training properties.

Tolerances (normwise relative error), from the formats:
- a bf16 output carries one rounding of at most half a unit in the last of 8
  significant bits, 2^-8 = 3.91e-3 of a value just above a power of two: 4e-3 with
  what the fp32 arithmetic adds;
- an fp32 output of the convolution or the norm: a handful of fp32 roundings
  (6e-8 each) and one 2^-22 exponential, and sums whose rounding grows with the
  root of their few thousand terms: 1e-5;
- an fp32 output of the scan: each step's decay is exact to 2^-22 plus the
  rounding of its exponent, and a state remembers at most the row's length (at
  most about 400 tokens here): 400 x 2.4e-7 = 1e-4, the library's bar for fp32.
8-bit values are checked one by one: at most half a step of the format (2^-4 of
the value, or 2^-10 of the scale below the normal range).
"""

import numpy as np
import pytest
import torch

from oracle import layer
from tests.helpers import check_close, np64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def tol(t, scan=False):
    return 4e-3 if t.dtype == torch.bfloat16 else (1e-4 if scan else 1e-5)


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def wide_rows(t, pad):
    """The same values as a slice of rows `pad` elements wider."""
    if pad == 0:
        return t.cuda()
    w = torch.full(t.shape[:-1] + (t.shape[-1] + pad,), float("nan"), dtype=t.dtype, device="cuda")
    w[..., pad:] = t.cuda()
    return w[..., pad:]


def starts_of(B, T, lengths):
    if lengths is None:
        return [b * T for b in range(B + 1)], None
    s = [0] + list(np.cumsum(lengths))
    return [int(v) for v in s], torch.tensor(s, dtype=torch.int32, device="cuda")


def opt64(t):
    return None if t is None else np64(t)


# ------------------------------------------------------------------ convolution

CONV = [
    dict(io="bf16", B=2, T=150, D=64, W=4),
    dict(io="bf16", B=1, T=1, D=16, W=4),
    dict(io="bf16", B=5, T=1, D=264, W=4, state=True),
    dict(io="bf16", B=3, T=2, D=40, W=4, state=True),
    dict(io="bf16", B=2, T=67, D=37, W=3, state=True),
    dict(io="fp32", B=2, T=100, D=48, W=2, state=True, silu=False),
    dict(io="fp32", B=1, T=33, D=5, W=4, state=True),
    dict(io="bf16", B=2, T=70, D=64, W=4, pad=64),
    dict(io="bf16", B=2, T=70, D=64, W=4, pad=3),
    dict(io="fp32", B=2, T=9, D=12, W=3, pad=1, bias=False),
    dict(io="bf16", B=1, D=72, W=4, state=True, lengths=[0, 1, 2, 0, 3, 64, 65, 5, 0]),
    dict(io="fp32", B=1, D=9, W=4, state=True, lengths=[130, 1, 1, 1, 0, 40]),
    dict(io="bf16", B=1, D=64, W=3, lengths=[7, 200, 33]),
    dict(io="bf16", B=3, T=700, D=520, W=4, state=True),
]


def conv_case(kw, seed):
    k = dict(dict(T=0, silu=True, state=False, pad=0, bias=True, lengths=None), **kw)
    g = gen_of(seed)
    starts, cu = starts_of(k["B"], k["T"], k["lengths"])
    T = starts[-1] if cu is not None else k["T"]
    B, D, W, dt = k["B"], k["D"], k["W"], DT[k["io"]]
    n = len(starts) - 1
    c = dict(x=torch.randn(B, T, D, generator=g).to(dt), w=torch.randn(D, W, generator=g) * 0.6,
             bias=torch.randn(D, generator=g) if k["bias"] else None,
             h0=torch.randn(n, W - 1, D, generator=g).to(dt) if k["state"] else None,
             dy=torch.randn(B, T, D, generator=g).to(dt),
             df=torch.randn(n, W - 1, D, generator=g).to(dt) if k["state"] else None)
    ref = layer.conv(np64(c["x"]).reshape(-1, D), np64(c["w"]), opt64(c["bias"]), opt64(c["h0"]), starts, k["silu"],
                     np64(c["dy"]).reshape(-1, D), opt64(c["df"]))
    gpu = {name: None if t is None else t.cuda() for name, t in c.items()}
    gpu["x"] = wide_rows(c["x"], k["pad"])
    return k, gpu, cu, ref


@pytest.mark.parametrize("kw", CONV, ids=str)
def test_conv_matches_oracle(kw):
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, ref = conv_case(kw, 11)
    p = kda.make_conv_problem(c["x"], c["w"], c["bias"], silu=k["silu"], initial_state=c["h0"], cu_seqlens=cu)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, final = kda.kda_conv_fwd(p, err=err)
    dx, dw, db, dinit = kda.kda_conv_bwd(p, c["dy"], c["df"], need_dinit=True)
    assert int(err) == 0
    check_close("y", np64(y).reshape(ref["y"].shape), ref["y"], tol(y))
    assert np.array_equal(np64(final), ref["final"])     # copies of inputs
    check_close("dx", np64(dx).reshape(ref["dx"].shape), ref["dx"], tol(dx))
    check_close("dweight", np64(dw), ref["dweight"], tol(dw))
    if k["bias"]:
        check_close("dbias", np64(db), ref["dbias"], tol(db))
    check_close("dinit", np64(dinit), ref["dinit"], tol(dinit))


@pytest.mark.parametrize("kw", [CONV[2], CONV[3], CONV[10], CONV[13]], ids=str)
def test_conv_state_in_place(kw):
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, _ = conv_case(kw, 12)
    p = kda.make_conv_problem(c["x"], c["w"], c["bias"], silu=k["silu"], initial_state=c["h0"], cu_seqlens=cu)
    y1, f1 = kda.kda_conv_fwd(p)
    y2, f2 = kda.kda_conv_fwd(p, final_state=c["h0"])
    assert f2.data_ptr() == c["h0"].data_ptr()
    assert torch.equal(y1, y2) and torch.equal(f1, f2)


def test_conv_token_by_token_equals_one_call():
    import chunkwise_delta_rule_gb300 as kda
    k, c, _, _ = conv_case(dict(io="bf16", B=3, T=7, D=64, W=4, state=True), 13)
    y, final = kda.kda_conv_fwd(kda.make_conv_problem(c["x"], c["w"], c["bias"], initial_state=c["h0"]))
    state = c["h0"].clone()
    outs = []
    for t in range(7):
        p = kda.make_conv_problem(c["x"][:, t:t + 1], c["w"], c["bias"], initial_state=state)
        outs.append(kda.kda_conv_fwd(p, final_state=state)[0])
    assert torch.equal(torch.cat(outs, 1), y) and torch.equal(state, final)


def test_conv_keeps_a_bad_sequence_to_itself():
    """NaN and infinite inputs of one packed sequence reach no other."""
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, _ = conv_case(dict(io="fp32", B=1, D=8, W=4, state=True, lengths=[5, 6, 7]), 14)
    c["x"][0, 5:11] = float("nan")
    c["x"][0, 10] = float("inf")
    c["h0"][1] = float("inf")
    p = kda.make_conv_problem(c["x"], c["w"], c["bias"], initial_state=c["h0"], cu_seqlens=cu)
    y, final = kda.kda_conv_fwd(p)
    dx, _, _, dinit = kda.kda_conv_bwd(p, c["dy"], c["df"])
    for t in (y, dx):
        assert torch.isfinite(t[0, :5]).all() and torch.isfinite(t[0, 11:]).all()
    for t in (final, dinit):
        assert torch.isfinite(t[0]).all() and torch.isfinite(t[2]).all()


# ------------------------------------------------------------------ scan

SCAN = [
    dict(io="bf16", B=2, T=150, D=64, S=16),
    dict(io="bf16", B=1, T=1, D=32, S=16),
    dict(io="bf16", B=5, T=1, D=72, S=16, state=True),
    dict(io="fp32", B=2, T=100, D=40, S=16, state=True),
    dict(io="fp32", B=1, T=400, D=5, S=16, state=True),
    dict(io="fp32", B=2, T=70, D=36, S=5, G=2, state=True),
    dict(io="fp32", B=1, T=61, D=33, S=8),
    dict(io="bf16", B=2, T=65, D=48, S=32, G=2, state=True),
    dict(io="fp32", B=1, T=50, D=20, S=20, state=True),
    dict(io="fp32", B=1, T=45, D=34, S=64, state=True),
    dict(io="bf16", B=1, T=37, D=16, S=41, state=True),
    dict(io="fp32", B=2, T=33, D=24, S=16, gate=False, skip=False, bias=False, softplus=False),
    dict(io="bf16", B=2, T=70, D=64, S=16, pad=64),
    dict(io="bf16", B=2, T=70, D=64, S=16, pad=3),
    dict(io="bf16", B=1, D=40, S=16, state=True, lengths=[0, 1, 2, 0, 3, 64, 65, 5, 0]),
    dict(io="fp32", B=1, D=9, S=16, state=True, lengths=[130, 1, 1, 1, 0, 140, 16, 32]),
    dict(io="fp32", B=1, D=33, S=16, lengths=[7, 300, 33]),
    dict(io="fp32", B=1, D=12, S=40, state=True, lengths=[31, 3, 50]),
    dict(io="fp32", B=1, D=16, S=6, state=True, lengths=[17, 16, 1, 200]),
]


def scan_case(kw, seed):
    k = dict(dict(T=0, G=1, state=False, pad=0, gate=True, skip=True, bias=True, softplus=True, lengths=None), **kw)
    g = gen_of(seed)
    starts, cu = starts_of(k["B"], k["T"], k["lengths"])
    T = starts[-1] if cu is not None else k["T"]
    B, D, S, G, dt = k["B"], k["D"], k["S"], k["G"], DT[k["io"]]
    n = len(starts) - 1
    step = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9)
    c = dict(x=torch.randn(B, T, D, generator=g).to(dt),
             dt=(torch.randn(B, T, D, generator=g) * 0.5).to(dt) if k["softplus"]
             else (torch.rand(B, T, D, generator=g) * 0.2).to(dt),
             A_log=torch.log(torch.arange(1, S + 1).float()).repeat(D, 1) + 0.1 * torch.randn(D, S, generator=g),
             b=torch.randn(B, T, G, S, generator=g).to(dt), c=torch.randn(B, T, G, S, generator=g).to(dt),
             d_skip=torch.randn(D, generator=g) if k["skip"] else None,
             z=torch.randn(B, T, D, generator=g).to(dt) if k["gate"] else None,
             dt_bias=step + torch.log(-torch.expm1(-step)) if k["bias"] else None,
             h0=torch.randn(n, D, S, generator=g) if k["state"] else None,
             dy=torch.randn(B, T, D, generator=g).to(dt),
             dht=torch.randn(n, D, S, generator=g) if k["state"] else None)
    f = {name: None if t is None else np64(t).reshape((-1,) + tuple(t.shape[2:]) if name in ("x", "dt", "b", "c", "z", "dy")
                                                     else t.shape) for name, t in c.items()}
    ref = layer.scan(f["x"], f["dt"], f["A_log"], f["b"], f["c"], f["d_skip"], f["z"], f["dt_bias"], f["h0"], starts,
                     k["softplus"], f["dy"], f["dht"])
    gpu = {name: None if t is None else t.cuda() for name, t in c.items()}
    if k["pad"]:
        for name in ("x", "dt", "z"):
            gpu[name] = wide_rows(c[name], k["pad"])
        for name in ("b", "c"):
            gpu[name] = wide_rows(c[name].flatten(2), k["pad"]).unflatten(-1, (G, S))
    return k, gpu, cu, ref


def scan_problem(k, c, cu, save=0, h0="h0"):
    import chunkwise_delta_rule_gb300 as kda
    return kda.make_ssm_problem(c["x"], c["dt"], c["A_log"], c["b"], c["c"], d_skip=c["d_skip"], z=c["z"],
                                dt_bias=c["dt_bias"], dt_softplus=k["softplus"], initial_state=c[h0], cu_seqlens=cu,
                                save_policy=save)


@pytest.mark.parametrize("save", [0, 1])
@pytest.mark.parametrize("kw", SCAN, ids=str)
def test_scan_matches_oracle(kw, save):
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, ref = scan_case(kw, 21)
    p = scan_problem(k, c, cu, save)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, ht, saved = kda.kda_ssm_fwd(p, err=err)
    g = kda.kda_ssm_bwd(p, c["dy"], c["dht"], saved=saved, need_dh0=True)
    assert int(err) == 0
    got = dict(y=y, ht=ht, dx=g.dx, ddt=g.ddt, dA_log=g.dA_log, db=g.db, dc=g.dc, dd_skip=g.dd_skip, dz=g.dz,
               ddt_bias=g.ddt_bias, dh0=g.dh0)
    for name, t in got.items():
        if t is not None:
            check_close(name, np64(t).reshape(ref[name].shape), ref[name], tol(t, True))
    assert (g.dz is None) == (not k["gate"]) and (g.dd_skip is None) == (not k["skip"])


@pytest.mark.parametrize("kw", [SCAN[2], SCAN[4], SCAN[14], SCAN[15]], ids=str)
def test_scan_state_in_place(kw):
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, _ = scan_case(kw, 22)
    p = scan_problem(k, c, cu)
    y1, h1, _ = kda.kda_ssm_fwd(p)
    y2, h2, _ = kda.kda_ssm_fwd(p, ht=c["h0"])
    assert h2.data_ptr() == c["h0"].data_ptr()
    assert torch.equal(y1, y2) and torch.equal(h1, h2)


def test_scan_token_by_token_agrees_with_one_call():
    import chunkwise_delta_rule_gb300 as kda
    k, c, _, ref = scan_case(dict(io="fp32", B=3, T=9, D=40, S=16, state=True), 23)
    state = c["h0"].clone()
    outs = []
    for t in range(9):
        part = {n: v[:, t:t + 1] if n in ("x", "dt", "b", "c", "z") else v for n, v in c.items()}
        part["state"] = state
        outs.append(kda.kda_ssm_fwd(scan_problem(k, part, None, h0="state"), ht=state)[0])
    check_close("y", np64(torch.cat(outs, 1)).reshape(ref["y"].shape), ref["y"], 1e-4)
    check_close("ht", np64(state), ref["ht"], 1e-4)


def test_scan_long_rows_in_pieces_match_oracle():
    """Few channels and long rows: cut into time pieces, joined through their end states; packed boundaries fall
    inside and between pieces."""
    import chunkwise_delta_rule_gb300 as kda
    for kw in (dict(io="fp32", B=1, T=2100, D=8, S=16, state=True),
               dict(io="fp32", B=1, D=8, S=16, state=True, lengths=[300, 1, 1500, 0, 12, 299])):
        k, c, cu, ref = scan_case(kw, 24)
        for save in (0, 1):
            p = scan_problem(k, c, cu, save)
            y, ht, saved = kda.kda_ssm_fwd(p)
            g = kda.kda_ssm_bwd(p, c["dy"], c["dht"], saved=saved)
            for name, t in dict(y=y, ht=ht, dx=g.dx, ddt=g.ddt, dA_log=g.dA_log, db=g.db, dc=g.dc, dd_skip=g.dd_skip,
                                dz=g.dz, ddt_bias=g.ddt_bias, dh0=g.dh0).items():
                check_close(name, np64(t).reshape(ref[name].shape), ref[name], 1e-4)
        state = c["h0"].clone()
        c["state"] = state
        y2, _, _ = kda.kda_ssm_fwd(scan_problem(k, c, cu, h0="state"), ht=state)
        assert torch.equal(y2, y) and torch.equal(state, ht)


def test_scan_is_deterministic_and_policies_agree():
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, _ = scan_case(dict(io="bf16", B=2, T=200, D=96, S=16, state=True), 25)
    runs = []
    for save in (0, 0, 1):
        p = scan_problem(k, c, cu, save)
        y, ht, saved = kda.kda_ssm_fwd(p)
        runs.append((y, ht) + tuple(kda.kda_ssm_bwd(p, c["dy"], c["dht"], saved=saved)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


def test_scan_keeps_a_bad_sequence_to_itself():
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, _ = scan_case(dict(io="fp32", B=1, D=8, S=16, state=True, lengths=[21, 22, 23]), 26)
    for name in ("x", "dt", "z", "b"):
        c[name][0, 21:43] = float("nan")
    c["x"][0, 42] = float("inf")
    c["h0"][1] = float("inf")
    p = scan_problem(k, c, cu)
    y, ht, _ = kda.kda_ssm_fwd(p)
    g = kda.kda_ssm_bwd(p, c["dy"], c["dht"])
    for t in (y, g.dx, g.ddt, g.db, g.dc, g.dz):
        assert torch.isfinite(t[0, :21]).all() and torch.isfinite(t[0, 43:]).all()
    for t in (ht, g.dh0):
        assert torch.isfinite(t[0]).all() and torch.isfinite(t[2]).all()


def test_scan_of_large_steps():
    """Steps far on both sides of the softplus's bend: no overflow, and the decay reaches zero."""
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, _ = scan_case(dict(io="fp32", B=1, T=40, D=8, S=16, bias=False), 27)
    c["dt"] = torch.linspace(-90, 90, 40, device="cuda").view(1, 40, 1).expand(1, 40, 8).contiguous()
    y, ht, _ = kda.kda_ssm_fwd(scan_problem(k, c, cu))
    f = {n: np64(v).reshape((-1,) + tuple(v.shape[2:])) for n, v in c.items() if n in ("x", "dt", "b", "c", "z")}
    ref = layer.scan(f["x"], f["dt"], np64(c["A_log"]), f["b"], f["c"], np64(c["d_skip"]), f["z"], None, None, [0, 40])
    check_close("y", np64(y).reshape(40, 8), ref["y"], 1e-4)
    check_close("ht", np64(ht), ref["ht"], 1e-4)


@pytest.mark.parametrize("B,T,D,S", [(2, 6, 72, 16), (2, 7, 72, 16), (58, 24, 512, 16), (58, 25, 512, 16), (58, 12, 512, 20),
                                     (58, 13, 512, 20)])
def test_scan_of_few_tokens(B, T, D, S):
    """On both sides of the lengths up to which tokens are taken one by one; the states in place."""
    import chunkwise_delta_rule_gb300 as kda
    k, c, cu, ref = scan_case(dict(io="bf16", B=B, T=T, D=D, S=S, state=True), 28)
    h = c["h0"].clone()
    c["h0"] = h
    y, ht, _ = kda.kda_ssm_fwd(scan_problem(k, c, cu), ht=h)
    check_close("y", np64(y).reshape(ref["y"].shape), ref["y"], tol(y, True))
    check_close("ht", np64(ht), ref["ht"], tol(ht, True))


@pytest.mark.parametrize("which", ["conv", "scan"])
def test_inconsistent_offsets_set_the_error_word(which):
    """Decreasing offsets and offsets outside the axis: flagged, and every access stays in bounds (they are clamped)."""
    import chunkwise_delta_rule_gb300 as kda
    for bad in ([0, 9, 4, 12], [0, 4, 99, 12], [3, 4, 8, 12], [0, -5, 8, 11]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        if which == "conv":
            k, c, _, _ = conv_case(dict(io="bf16", B=1, D=16, W=4, state=True, lengths=[4, 4, 4]), 31)
            p = kda.make_conv_problem(c["x"], c["w"], c["bias"], initial_state=c["h0"], cu_seqlens=cu)
            kda.kda_conv_fwd(p, err=err)
            kda.kda_conv_bwd(p, c["dy"], c["df"])
        else:
            k, c, _, _ = scan_case(dict(io="bf16", B=1, D=16, S=16, state=True, lengths=[4, 4, 4]), 31)
            p = scan_problem(k, c, cu)
            kda.kda_ssm_fwd(p, err=err)
            kda.kda_ssm_bwd(p, c["dy"], c["dht"])
        assert int(err) & 1


def test_empty_axis_passes_states_through():
    import chunkwise_delta_rule_gb300 as kda
    h = torch.randn(2, 3, 16, device="cuda").bfloat16()
    x = torch.empty(2, 0, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(16, 4, device="cuda")
    p = kda.make_conv_problem(x, w, initial_state=h)
    assert torch.equal(kda.kda_conv_fwd(p)[1], h)
    dx, dw, _, dinit = kda.kda_conv_bwd(p, x, h)
    assert torch.equal(dinit, h) and not dw.any()
    s = torch.randn(2, 16, 16, device="cuda")
    bc = torch.empty(2, 0, 1, 16, device="cuda", dtype=torch.bfloat16)
    p = kda.make_ssm_problem(x, x, torch.zeros(16, 16, device="cuda"), bc, bc, initial_state=s)
    assert torch.equal(kda.kda_ssm_fwd(p)[1], s)
    g = kda.kda_ssm_bwd(p, x, s)
    assert torch.equal(g.dh0, s) and not g.dA_log.any()


# ------------------------------------------------------------------ norm

NORM = [("bf16", 5, 64), ("bf16", 1, 1), ("bf16", 3, 4096), ("fp32", 4, 257), ("fp32", 700, 40), ("bf16", 2, 5001),
        ("fp32", 2, 8192), ("bf16", 2, 16384), ("fp32", 3, 1000), ("bf16", 33, 2048), ("fp32", 2, 12288)]


def norm_case(io, R, D, seed):
    g = gen_of(seed)
    return tuple(t.cuda() for t in (torch.randn(R, D, generator=g).to(DT[io]), torch.randn(R, D, generator=g).to(DT[io]),
                                    1 + 0.3 * torch.randn(D, generator=g), torch.randn(R, D, generator=g).to(DT[io])))


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("io,R,D", NORM)
def test_norm_matches_oracle(io, R, D, res):
    import chunkwise_delta_rule_gb300 as kda
    x, r, w, dy = norm_case(io, R, D, 41)
    y, scale, h = kda.kda_norm_fwd(kda.make_norm_problem(x, w, residual=r if res else None, eps=1e-5))
    ref = layer.norm(np64(x), np64(w), np64(r) if res else None, 1e-5)
    assert scale is None and (res or h is x)
    check_close("y", np64(y), ref["y"], tol(y))
    check_close("h", np64(h), ref["h"], tol(h))
    dx, dw = kda.kda_norm_bwd(kda.make_norm_problem(h, w, eps=1e-5), dy, r if res else None)
    ref = layer.norm(np64(h), np64(w), None, 1e-5, np64(dy), np64(r) if res else None)
    check_close("dx", np64(dx), ref["dx"], tol(dx))
    check_close("dweight", np64(dw), ref["dweight"], tol(dw))


@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("io,R,D", [("bf16", 4, 4096), ("bf16", 3, 200), ("fp32", 5, 333), ("bf16", 2, 8200),
                                    ("fp32", 2, 31), ("bf16", 2, 16384)])
def test_norm_8bit_output(io, R, D, group):
    import chunkwise_delta_rule_gb300 as kda
    x, r, w, _ = norm_case(io, R, D, 42)
    x[0] *= 1e-3
    q, scale, h = kda.kda_norm_fwd(kda.make_norm_problem(x, w, residual=r, eps=1e-6, out="e4m3", group=group))
    ref = layer.norm(np64(x), np64(w), np64(r), 1e-6)["y"]
    gr = group or D
    ng = -(-D // gr)
    assert q.dtype == torch.float8_e4m3fn and tuple(scale.shape) == (R, ng)
    pad = np.zeros((R, ng * gr))
    pad[:, :D] = np.abs(ref)
    want = pad.reshape(R, ng, gr).max(axis=2) / 448.0
    assert np.max(np.abs(np64(scale) - want) / want) <= 2e-6
    s = np.repeat(np64(scale), gr, axis=1)[:, :D]
    val = np64(q.float()) * s
    assert np.all(np.abs(val - ref) <= np.maximum(np.abs(ref) / 16, s / 1024) * (1 + 1e-4) + s * 448 * 1e-6)
    check_close("h", np64(h), layer.norm(np64(x), np64(w), np64(r), 1e-6)["h"], tol(h))


def test_norm_8bit_zero_tiny_and_bad_rows():
    import chunkwise_delta_rule_gb300 as kda
    x = torch.ones(5, 256, device="cuda")
    x[0] = 0
    x[1, 128:] = 0
    x[2, 3] = float("nan")
    x[3, 200] = float("inf")
    w = torch.ones(256, device="cuda")
    w[:128] = 1e-38
    w[5] = 0
    q, scale, _ = kda.kda_norm_fwd(kda.make_norm_problem(x, w, out="e4m3", group=128))
    v = q.float() * scale.repeat_interleave(128, 1)
    assert not v[0].any() and not scale[0].any()                 # a row of zeros
    assert not v[1, 128:].any() and scale[1, 1] == 0             # a group of zeros
    assert torch.isnan(scale[2]).all()                           # a NaN reaches its whole row through the sum
    assert torch.isnan(scale[3, 1])                              # infinity / infinity
    assert torch.isfinite(v[4]).all() and v[4, 5] == 0           # a group below what 448 / amax can hold
    assert torch.all((q.float()[4, :128] - 448).abs()[torch.arange(128, device="cuda") != 5] <= 16)


def test_norm_updates_the_residual_in_place():
    import chunkwise_delta_rule_gb300 as kda
    x, r, w, _ = norm_case("bf16", 9, 1024, 43)
    y1, _, h1 = kda.kda_norm_fwd(kda.make_norm_problem(x, w, residual=r))
    y2, _, h2 = kda.kda_norm_fwd(kda.make_norm_problem(x, w, residual=r), h=r)
    assert h2.data_ptr() == r.data_ptr() and torch.equal(y1, y2) and torch.equal(h1, h2)


def test_norm_without_rows():
    import chunkwise_delta_rule_gb300 as kda
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert kda.kda_norm_fwd(kda.make_norm_problem(x, w))[0].shape == (0, 64)
    dx, dw = kda.kda_norm_bwd(kda.make_norm_problem(x, w), x)
    assert not dw.any()


# ------------------------------------------------------------------ all of them

def test_gradients_against_differences_on_the_gpu():
    """Central differences along a random direction through the autograd functions, fp32: step 1e-2 leaves a
    truncation of order 1e-4 and a rounding of about 1e-6 / 1e-2 = 1e-4 of the loss's parts: 5e-3 of the derivative's
    natural size (the product of the gradient's and the direction's norms over the root of their length)."""
    import chunkwise_delta_rule_gb300 as kda
    _, c, _, _ = conv_case(dict(io="fp32", B=2, T=40, D=24, W=4, state=True), 51)
    _, s, _, _ = scan_case(dict(io="fp32", B=2, T=40, D=24, S=16, state=True), 52)
    x, r, w, dy = norm_case("fp32", 6, 200, 53)

    def f_conv(x, w, b, h):
        y, f = kda.short_conv(x, w, b, initial_state=h)
        return (y * c["dy"]).double().sum() + (f * c["df"]).double().sum()

    def f_scan(x, dt, A, b, cm, d, z, db, h):
        y, ht = kda.ssm_scan(x, dt, A, b, cm, d_skip=d, z=z, dt_bias=db, initial_state=h)
        return (y * s["dy"]).double().sum() + (ht * s["dht"]).double().sum()

    def f_norm(a, b, g):
        y, h = kda.rms_norm(a, g, residual=b)
        return (y * dy).double().sum() + (h * x).double().sum()

    for f, args in ((f_conv, (c["x"], c["w"], c["bias"], c["h0"])),
                    (f_scan, tuple(s[n] for n in ("x", "dt", "A_log", "b", "c", "d_skip", "z", "dt_bias", "h0"))),
                    (f_norm, (x.clone(), r, w))):
        leaves = [a.clone().requires_grad_(True) for a in args]
        f(*leaves).backward()
        for i in range(len(leaves)):
            v = torch.randn(leaves[i].shape, generator=torch.Generator(device="cuda").manual_seed(60 + i), device="cuda")
            with torch.no_grad():
                up = [a + 1e-2 * v if j == i else a for j, a in enumerate(args)]
                dn = [a - 1e-2 * v if j == i else a for j, a in enumerate(args)]
                num = float(f(*up) - f(*dn)) / 2e-2
            g = leaves[i].grad.double()
            ana = float((g * v.double()).sum())
            assert abs(num - ana) <= 5e-3 * float(g.norm()), (f.__name__, i, num, ana)


def test_operators_run_on_the_current_stream_and_in_a_graph():
    import chunkwise_delta_rule_gb300 as kda
    k, c, _, _ = scan_case(dict(io="bf16", B=4, T=1, D=64, S=16, state=True), 61)
    w, bias = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    cs = torch.randn(4, 3, 64, device="cuda").bfloat16()
    g = torch.ones(64, device="cuda")

    def step(state, conv_state):
        y, _, h = kda.kda_norm_fwd(kda.make_norm_problem(c["x"], g))
        y, _ = kda.kda_conv_fwd(kda.make_conv_problem(y, w, bias, initial_state=conv_state), final_state=conv_state)
        d = dict(c, x=y, state=state)
        return kda.kda_ssm_fwd(scan_problem(k, d, None, h0="state"), ht=state)[0]

    s1, c1 = c["h0"].clone(), cs.clone()
    want = [step(s1, c1).clone() for _ in range(3)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s2, c2 = c["h0"].clone(), cs.clone()
        got = [step(s2, c2).clone() for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and torch.equal(s1, s2)
    s3, c3 = c["h0"].clone(), cs.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s3, c3)
    s3.copy_(c["h0"])
    c3.copy_(cs)
    for a in want:
        graph.replay()
        assert torch.equal(out, a)
    assert torch.equal(s3, s1) and torch.equal(c3, c1)
