"""Cases of the layer operators around the delta rule: the short causal
convolution, the selective state space scan, and the root-mean-square norm with
the residual's addition and an 8-bit output.

``run`` computes a case in its plain form (torch operations in 32 bits, one
rounding at the end) or, with ``own`` true, through the package's entry points;
``exact`` computes it from the definition in 64 bits.

All three work on the packed token axis: sequence n owns the tokens
cu[n] .. cu[n+1]-1 of a [1, total, ...] tensor, or [B, T, ...] with equal lengths.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_E4M3_MAX = 448.0
_EPS = 1e-6


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of each of 64 sequences through the q, k, v convolutions of 32 heads of 128, its state in place
        dict(name="conv_step", op="conv", dir="step", io="bf16", B=64, T=1, D=12288, W=4, silu=True, state=True,
             nseq=0, sliced=False),
        # a packed prefill: ragged prompts (an empty one and one of a single token among them), resumed states
        dict(name="conv_packed", op="conv", dir="fwd", io="bf16", B=1, T=32768, D=4096, W=4, silu=True, state=True,
             nseq=9, sliced=False),
        # training backward; the input is one half of a projection's rows, as a layer has it
        dict(name="conv_back", op="conv", dir="back", io="bf16", B=2, T=8192, D=4096, W=4, silu=True, state=False,
             nseq=0, sliced=True),
        # one token of each of 64 sequences, the states updated in place
        dict(name="ssm_step", op="ssm", dir="step", io="bf16", B=64, T=1, D=4096, N=16, G=1, state=True, nseq=0,
             sliced=True),
        # prompts: two long sequences at full width
        dict(name="ssm_prompt", op="ssm", dir="fwd", io="bf16", B=2, T=8192, D=4096, N=16, G=1, state=False, nseq=0,
             sliced=True),
        # few channels and many tokens (one shard of a wide layer): packed sequences, the time axis is the long one
        dict(name="ssm_long", op="ssm", dir="fwd", io="bf16", B=1, T=32768, D=1024, N=16, G=1, state=True, nseq=3,
             sliced=False),
        # a training step: forward that keeps what its backward reads, and the backward
        dict(name="ssm_train", op="ssm", dir="train", io="bf16", B=4, T=2048, D=2048, N=16, G=1, state=False, nseq=0,
             sliced=True),
        # 32-bit training with odd sizes, two groups, carried states
        dict(name="ssm_odd", op="ssm", dir="train", io="fp32", B=3, T=777, D=250, N=20, G=2, state=True, nseq=0,
             sliced=False),
        # one token of each of 64 sequences: residual added, 8-bit rows for the projection that follows
        dict(name="norm_step", op="norm", dir="fwd", io="bf16", R=64, D=4096, out="e4m3", group=128, res=True),
        # the same for a batch of prompts
        dict(name="norm_prompt", op="norm", dir="fwd", io="bf16", R=16384, D=4096, out="e4m3", group=128, res=True),
        # 32-bit rows of an odd width, output in the input's type
        dict(name="norm_odd", op="norm", dir="fwd", io="fp32", R=777, D=5001, out="io", group=0, res=True),
        # training backward, the residual stream's gradient added
        dict(name="norm_back", op="norm", dir="back", io="bf16", R=16384, D=4096, out="io", group=0, res=True),
    ]


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, v + (v == 3072)))


def draw(rng):
    op = rng.choice(("conv", "ssm", "norm"))
    io = rng.choice(("bf16", "bf16", "fp32"))
    if op == "norm":
        direction = rng.choice(("fwd", "fwd", "back"))
        group = rng.choice((0, 32, 64, 128))
        D = _log(rng, 64, 8192)
        if group and rng.random() < 0.5:
            D = max(group, D // group * group) + (128 if D // group * group == 3072 else 0)
        out = rng.choice(("io", "e4m3")) if direction == "fwd" else "io"
        return dict(op=op, dir=direction, io=io, R=_log(rng, 1, 16384), D=D, out=out,
                    group=group if out == "e4m3" else 0, res=rng.random() < 0.7)
    direction = rng.choice(("fwd", "back", "step") if op == "conv" else ("fwd", "train", "step"))
    packed = direction != "step" and rng.random() < 0.4
    if direction == "step":
        B, T = _log(rng, 1, 256), 1
    elif packed:
        B, T = 1, _log(rng, 16, 32768)
    else:
        B, T = rng.randint(1, 8), _log(rng, 2, 4096)
    case = dict(op=op, dir=direction, io=io, B=B, T=T, D=_log(rng, 16, 8192))
    if rng.random() < 0.6:
        case["D"] = case["D"] // 8 * 8 + (8 if case["D"] // 8 * 8 == 3072 else 0)
    if op == "conv":
        case.update(W=rng.randint(2, 4), silu=rng.random() < 0.8)
        most = 2 * 8192 * 4096 if direction == "back" else 32768 * 4096
        unit = case["D"]
    else:
        G = rng.choice((1, 1, 2))
        case["D"] = case["D"] // G * G
        if case["D"] == 3072:
            case["D"] += 8
        case.update(N=rng.choice((16, 16, 16, _log(rng, 3, 64))), G=G)
        most = 4 * 2048 * 2048 * 16 if direction == "train" else 2 * 8192 * 4096 * 16
        unit = case["D"] * case["N"]
    if case["B"] * case["T"] * unit > most:
        if direction == "step":
            case["B"] = max(1, most // unit)
        else:
            case["T"] = max(2, most // (unit * case["B"]))
            case["T"] += case["T"] == 3072
    case.update(state=direction == "step" or rng.random() < 0.5, nseq=rng.randint(1, 12) if packed else 0,
                sliced=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _uniform(gen, lo, hi, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32) * (hi - lo) + lo


def _slice(t, sliced):
    """The tensor itself, or the same values as the last columns of rows twice as wide (a projection's second half)."""
    if not sliced:
        return t
    wide = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=t.device)
    wide[..., t.shape[-1]:] = t
    return wide[..., t.shape[-1]:]


def _cuts(gen, total, nseq):
    """Offsets of nseq packed sequences: random cuts, an empty sequence and one of a single token where they fit."""
    inner = torch.randint(0, total + 1, (nseq - 1,), generator=gen, device="cuda")
    inner = torch.sort(inner).values
    if nseq >= 4:
        inner[1] = inner[0]
        inner[2] = (inner[1] + 1).clamp(max=total)
        inner = torch.sort(inner).values
    ends = torch.tensor([0, total], device="cuda")
    return torch.cat([ends[:1], inner, ends[1:]]).to(torch.int32)


def prepare(case, seed):
    gen, dt = _gen(seed), _DT[case["io"]]
    s = dict(case)
    if case["op"] == "norm":
        R, D = case["R"], case["D"]
        # a residual stream with a few columns of large values, as trained models have them
        big = torch.where(torch.rand(D, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
        s["x"] = (_randn(gen, R, D) * big).to(dt)
        s["residual"] = (_randn(gen, R, D) * big * 2).to(dt) if case["res"] else None
        s["weight"] = 1 + 0.2 * _randn(gen, D)
        if case["dir"] == "back":
            s["dy"] = _randn(gen, R, D).to(dt)
        return s
    B, T, D = case["B"], case["T"], case["D"]
    s["cu"] = _cuts(gen, B * T, case["nseq"]) if case["nseq"] else None
    n = case["nseq"] or B
    s["x"] = _slice(_randn(gen, B, T, D).to(dt), case["sliced"])
    if case["op"] == "conv":
        W = case["W"]
        s["weight"] = _uniform(gen, -1, 1, D, W) / math.sqrt(W)
        s["bias"] = _uniform(gen, -1, 1, D) / math.sqrt(W)
        s["h0"] = _randn(gen, n, W - 1, D).to(dt) if case["state"] else None
        if case["dir"] == "back":
            s["dy"] = _randn(gen, B, T, D).to(dt)
            s["dfinal"] = _randn(gen, n, W - 1, D).to(dt) if case["state"] else None
        return s
    N, G = case["N"], case["G"]
    # steps of 1e-3 .. 1e-1 around their bias, decay rates 1 .. N, as state space layers start from
    step = torch.exp(_uniform(gen, math.log(1e-3), math.log(1e-1), D))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["dt"] = (0.5 * _randn(gen, B, T, D)).to(dt)
    s["A_log"] = torch.log(torch.arange(1, N + 1, device="cuda", dtype=torch.float32)).repeat(D, 1) \
        + 0.1 * _randn(gen, D, N)
    # b and c: neighbouring columns of one projection's rows
    bc = _randn(gen, B, T, 2 * G * N).to(dt)
    s["b"] = bc[..., :G * N].unflatten(-1, (G, N))
    s["c"] = bc[..., G * N:].unflatten(-1, (G, N))
    if not case["sliced"]:
        s["b"], s["c"] = s["b"].contiguous(), s["c"].contiguous()
    s["d_skip"] = 1 + 0.1 * _randn(gen, D)
    s["z"] = _slice(_randn(gen, B, T, D).to(dt), case["sliced"])
    s["h0"] = 0.5 * _randn(gen, n, D, N) if case["state"] else None
    if case["dir"] == "train":
        s["dy"] = _randn(gen, B, T, D).to(dt)
        s["dht"] = _randn(gen, n, D, N) if case["state"] else None
    return s


# ------------------------------------------------------------------- plain forms

def _axis(s):
    """Per packed token: its sequence, its position in it; per sequence: first token and length."""
    if s["cu"] is not None:
        first, length = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    else:
        first = torch.arange(s["B"], device="cuda") * s["T"]
        length = torch.full_like(first, s["T"])
    total = s["B"] * s["T"]
    seq = torch.repeat_interleave(torch.arange(first.numel(), device="cuda"), length, output_size=total)
    pos = torch.arange(total, device="cuda") - first[seq]
    return seq, pos, first, length


def _taps(s):
    """Rows of [inputs; carried states] that each token's W taps and each final state's W - 1 rows read."""
    seq, pos, first, length = _axis(s)
    W, total = s["W"], s["B"] * s["T"]
    j = torch.arange(W, device="cuda")
    back = pos[:, None] - (W - 1) + j
    tok = torch.where(back >= 0, first[seq][:, None] + back, total + seq[:, None] * (W - 1) + pos[:, None] + j)
    r = torch.arange(W - 1, device="cuda")
    n = torch.arange(first.numel(), device="cuda")
    last = length[:, None] - (W - 1) + r
    fin = torch.where(last >= 0, first[:, None] + last, total + n[:, None] * (W - 1) + length[:, None] + r)
    return tok, fin


def _conv_rows(s):
    x = s["x"].reshape(-1, s["D"]).float()
    n = s["nseq"] or s["B"]
    h0 = x.new_zeros(n * (s["W"] - 1), s["D"]) if s["h0"] is None else s["h0"].reshape(-1, s["D"]).float()
    return torch.cat([x, h0])


def _plain_conv(s):
    rows = _conv_rows(s)
    tok, fin = _taps(s)
    pre = (rows[tok] * s["weight"].t()).sum(1) + s["bias"]
    y = pre * torch.sigmoid(pre) if s["silu"] else pre
    dt = s["x"].dtype
    final = rows[fin].to(dt)
    if s["dir"] == "step":
        final = s["h0"].copy_(final)
    return {"y": y.to(dt).view(s["B"], s["T"], s["D"]), "final": final}


def _plain_conv_back(s):
    rows = _conv_rows(s)
    tok, fin = _taps(s)
    taps = rows[tok]
    pre = (taps * s["weight"].t()).sum(1) + s["bias"]
    d = s["dy"].reshape(-1, s["D"]).float()
    if s["silu"]:
        g = torch.sigmoid(pre)
        d = d * g * (1 + pre * (1 - g))
    drows = torch.zeros_like(rows)
    drows.index_add_(0, tok.reshape(-1), (d[:, None] * s["weight"].t()).reshape(-1, s["D"]))
    if s["dfinal"] is not None:
        drows.index_add_(0, fin.reshape(-1), s["dfinal"].reshape(-1, s["D"]).float())
    total, dt = s["B"] * s["T"], s["x"].dtype
    out = {"dx": drows[:total].to(dt).view(s["B"], s["T"], s["D"]), "dweight": (d[:, None] * taps).sum(0).t(),
           "dbias": d.sum(0)}
    if s["h0"] is not None:
        out["dinit"] = drows[total:].to(dt).view_as(s["h0"])
    return out


def _recur(a, b, reverse=False):
    """h_t = a_t h_{t-1} + b_t along the first axis (or from its end), by doubling; a and b are overwritten."""
    step = 1
    while step < a.shape[0]:
        if reverse:
            b[:-step] += a[:-step] * b[step:]
            a[:-step] = a[:-step] * a[step:]
        else:
            b[step:] += a[step:] * b[:-step]
            a[step:] = a[step:] * a[:-step]
        step *= 2
    return b


def _plain_ssm(s):
    """Forward and, for a training case, the backward; channels as [groups, channels of the group]."""
    seq, pos, first, length = _axis(s)
    B, T, D, N, G = (s[k] for k in ("B", "T", "D", "N", "G"))
    M, total, n, io = D // G, B * T, first.numel(), s["x"].dtype
    tdm = (total, G, M)
    x, z = s["x"].reshape(tdm).float(), s["z"].reshape(tdm).float()
    bm, cm = s["b"].reshape(total, G, 1, N).float(), s["c"].reshape(total, G, 1, N).float()
    raw = s["dt"].reshape(tdm).float() + s["dt_bias"].view(G, M)
    delta = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    A = -torch.exp(s["A_log"]).view(G, M, N)
    h0 = x.new_zeros(n, G, M, N) if s["h0"] is None else s["h0"].view(n, G, M, N)
    some = length > 0
    start, last = first[some], (first + length - 1)[some]
    a = torch.exp(delta[..., None] * A)
    b = (delta * x)[..., None] * bm
    b[start] += a[start] * h0[some]
    k = a.clone() if s["dir"] == "train" else a
    k[start] = 0
    h = _recur(k, b)
    del k
    y0 = (h * cm).sum(-1) + s["d_skip"].view(G, M) * x
    sig = torch.sigmoid(z)
    y = (y0 * z * sig).to(io).view(B, T, D)
    ht = h0.clone()
    ht[some] = h[last]
    ht = ht.view(n, D, N)
    if s["dir"] == "step":
        ht = s["h0"].copy_(ht)
    if s["dir"] != "train":
        return {"y": y, "ht": ht}
    dy = s["dy"].reshape(tdm).float()
    dz = dy * y0 * sig * (1 + z * (1 - sig))
    d0 = dy * z * sig
    g = cm * d0[..., None]
    if s["dht"] is not None:
        g[last] += s["dht"].view(n, G, M, N)[some]
    r = torch.zeros_like(a)
    r[:-1] = a[1:]
    r[last] = 0
    g = _recur(r, g, reverse=True)
    del r
    hp = torch.zeros_like(h)
    hp[1:] = h[:-1]
    hp[start] = h0[some]
    w = g * a * hp
    gb = (g * bm).sum(-1)
    ddelta = (w * A).sum(-1) + x * gb
    draw_ = ddelta * torch.sigmoid(raw)
    out = {"y": y, "ht": ht, "dx": (delta * gb + s["d_skip"].view(G, M) * d0).to(io).view(B, T, D),
           "ddt": draw_.to(io).view(B, T, D), "dz": dz.to(io).view(B, T, D),
           "dA_log": ((w * delta[..., None]).sum(0) * A).view(D, N),
           "db": (g * (delta * x)[..., None]).sum(2).to(io).view(B, T, G, N),
           "dc": (h * d0[..., None]).sum(2).to(io).view(B, T, G, N),
           "dd_skip": (d0 * x).sum(0).view(D), "ddt_bias": draw_.sum(0).view(D)}
    if s["h0"] is not None:
        dh0 = s["dht"].clone().view(n, G, M, N)
        dh0[some] = a[start] * g[start]
        out["dh0"] = dh0.view(n, D, N)
    return out


def _plain_norm(s):
    x = s["x"].float()
    h = x + s["residual"].float() if s["residual"] is not None else x
    D = s["D"]
    y = h * torch.rsqrt((h * h).sum(-1, keepdim=True) / D + _EPS) * s["weight"]
    out = {} if s["residual"] is None else {"h": h.to(s["x"].dtype)}
    if s["out"] == "io":
        return {"y": y.to(s["x"].dtype), **out}
    group = s["group"] or D
    ng = -(-D // group)
    pad = torch.zeros(s["R"], ng * group, device=y.device)
    pad[:, :D] = y
    pad = pad.view(s["R"], ng, group)
    amax = pad.abs().amax(-1)
    inv = torch.where(amax > 0, _E4M3_MAX / amax, 0.0)
    q = (pad * inv[..., None]).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    return {"y": q.view(s["R"], -1)[:, :D], "scale": amax / _E4M3_MAX, **out}


def _plain_norm_back(s):
    h, dy, w = s["x"].float(), s["dy"].float(), s["weight"]
    r = torch.rsqrt((h * h).sum(-1, keepdim=True) / s["D"] + _EPS)
    wd = w * dy
    dx = r * (wd - h * r * r * ((h * wd).sum(-1, keepdim=True) / s["D"]))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h * r).sum(0)}


# ------------------------------------------------------------------- one pass

def _own_conv(s):
    import chunkwise_delta_rule_gb300 as kda
    p = kda.make_conv_problem(s["x"], s["weight"], s["bias"], silu=s["silu"], initial_state=s["h0"],
                              cu_seqlens=s["cu"])
    if s["dir"] == "back":
        dx, dw, db, dinit = kda.kda_conv_bwd(p, s["dy"], s["dfinal"])
        out = {"dx": dx, "dweight": dw, "dbias": db}
        return out if s["h0"] is None else {**out, "dinit": dinit}
    y, final = kda.kda_conv_fwd(p, final_state=s["h0"] if s["dir"] == "step" else None)
    return {"y": y, "final": final}


def _own_ssm(s):
    import chunkwise_delta_rule_gb300 as kda
    train = s["dir"] == "train"
    p = kda.make_ssm_problem(s["x"], s["dt"], s["A_log"], s["b"], s["c"], d_skip=s["d_skip"], z=s["z"],
                             dt_bias=s["dt_bias"], dt_softplus=True, initial_state=s["h0"], cu_seqlens=s["cu"],
                             save_policy=1 if train else 0)
    y, ht, saved = kda.kda_ssm_fwd(p, ht=s["h0"] if s["dir"] == "step" else None)
    if not train:
        return {"y": y, "ht": ht}
    g = kda.kda_ssm_bwd(p, s["dy"], s["dht"], saved=saved)
    out = {"y": y, "ht": ht, "dx": g.dx, "ddt": g.ddt, "dz": g.dz, "dA_log": g.dA_log, "db": g.db, "dc": g.dc,
           "dd_skip": g.dd_skip, "ddt_bias": g.ddt_bias}
    return out if s["h0"] is None else {**out, "dh0": g.dh0}


def _own_norm(s):
    import chunkwise_delta_rule_gb300 as kda
    if s["dir"] == "back":
        p = kda.make_norm_problem(s["x"], s["weight"], eps=_EPS)
        dx, dw = kda.kda_norm_bwd(p, s["dy"], s["residual"])
        return {"dx": dx, "dweight": dw}
    p = kda.make_norm_problem(s["x"], s["weight"], residual=s["residual"], eps=_EPS, out=s["out"], group=s["group"])
    y, scale, h = kda.kda_norm_fwd(p)
    out = {"y": y} if scale is None else {"y": y, "scale": scale}
    return out if s["residual"] is None else {**out, "h": h}


def run(state):
    op, back = state["op"], state["dir"] == "back"
    if own:
        return {"conv": _own_conv, "ssm": _own_ssm, "norm": _own_norm}[op](state)
    if op == "conv":
        return _plain_conv_back(state) if back else _plain_conv(state)
    if op == "ssm":
        return _plain_ssm(state)
    return _plain_norm_back(state) if back else _plain_norm(state)


def work(case):
    io = 2 if case["io"] == "bf16" else 4
    D = case["D"]
    if case["op"] == "norm":
        el = case["R"] * D
        if case["dir"] == "back":
            return {"bytes": el * io * (3 + case["res"]) + 8 * D, "flops": 10 * el}
        out = io if case["out"] == "io" else 1 + 4 / (case["group"] or D)
        return {"bytes": el * (io * (1 + 2 * case["res"]) + out) + 4 * D, "flops": el * (5 + 3 * (case["out"] != "io"))}
    tok, n = case["B"] * case["T"], case["nseq"] or case["B"]
    el = tok * D
    if case["op"] == "conv":
        W = case["W"]
        carried = n * (W - 1) * D * io
        if case["dir"] == "back":
            return {"bytes": 3 * el * io + 8 * D * (W + 1) + 4 * carried * case["state"],
                    "flops": el * (6 * W + 10 * case["silu"] + 1)}
        return {"bytes": 2 * el * io + 4 * D * (W + 1) + carried * (1 + case["state"]),
                "flops": el * (2 * W + 4 * case["silu"])}
    N, G = case["N"], case["G"]
    state = 4 * n * D * N
    params = 4 * D * (N + 2)
    rows = tok * 2 * G * N * io
    data = 4 * el * io + rows + params + state * (1 + case["state"])
    flops = el * (7 * N + 14)
    if case["dir"] == "train":
        data += 7 * el * io + 2 * rows + 2 * params + 3 * state * case["state"]
        flops += el * (19 * N + 40)
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------- 64 bits, token by token

def _spans(s):
    cu = s["cu"].tolist() if s["cu"] is not None else [b * s["T"] for b in range(s["B"] + 1)]
    return list(zip(cu[:-1], cu[1:]))


def _d(t):
    return None if t is None else t.double()


def _exact_conv(s):
    """Sequence by sequence on its extended rows (state rows, then tokens), one shifted copy per tap."""
    D, W, total = s["D"], s["W"], s["B"] * s["T"]
    x, w, bias = _d(s["x"]).reshape(total, D), _d(s["weight"]), _d(s["bias"])
    n = len(_spans(s))
    h0 = torch.zeros(n, W - 1, D, dtype=torch.float64, device=x.device) if s["h0"] is None else _d(s["h0"])
    back = s["dir"] == "back"
    y, final = torch.zeros_like(x), torch.zeros_like(h0)
    dx, dinit, dw, db = torch.zeros_like(x), torch.zeros_like(h0), torch.zeros_like(w), torch.zeros_like(bias)
    for i, (lo, hi) in enumerate(_spans(s)):
        L = hi - lo
        ext = torch.cat([h0[i], x[lo:hi]])
        final[i] = ext[L:]
        pre = bias.expand(L, D).clone()
        for j in range(W):
            pre += w[:, j] * ext[j:j + L]
        sg = 1 / (1 + torch.exp(-pre))
        y[lo:hi] = pre * sg if s["silu"] else pre
        if back:
            d = _d(s["dy"]).reshape(total, D)[lo:hi]
            if s["silu"]:
                d = d * (sg + pre * sg * (1 - sg))
            dext = torch.zeros_like(ext)
            for j in range(W):
                dext[j:j + L] += w[:, j] * d
                dw[:, j] += (d * ext[j:j + L]).sum(0)
            if s["dfinal"] is not None:
                dext[L:] += _d(s["dfinal"][i])
            db += d.sum(0)
            dinit[i], dx[lo:hi] = dext[:W - 1], dext[W - 1:]
    shape = (s["B"], s["T"], D)
    if not back:
        return {"y": y.view(shape), "final": final}
    out = {"dx": dx.view(shape), "dweight": dw, "dbias": db}
    return out if s["h0"] is None else {**out, "dinit": dinit}


def _exact_ssm(s):
    """One token after the other; equal-length sequences side by side, packed ones one by one."""
    B, T, D, N, G = (s[k] for k in ("B", "T", "D", "N", "G"))
    M, train, dev = D // G, s["dir"] == "train", s["x"].device
    spans = _spans(s)
    groups = [(list(range(len(spans))), T)] if s["cu"] is None else [([i], hi - lo) for i, (lo, hi) in enumerate(spans)]
    flat = {k: _d(s[k]).reshape(B * T, -1) for k in ("x", "dt", "z") + (("dy",) if train else ())}
    rows = {k: _d(s[k]).reshape(B * T, G, 1, N) for k in ("b", "c")}
    bias, A, skip = _d(s["dt_bias"]), -torch.exp(_d(s["A_log"])), _d(s["d_skip"])
    f64 = dict(dtype=torch.float64, device=dev)
    h0 = torch.zeros(len(spans), D, N, **f64) if s["h0"] is None else _d(s["h0"])
    dht = torch.zeros_like(h0) if not train or s["dht"] is None else _d(s["dht"])
    res = {k: torch.zeros(B * T, D, **f64) for k in (("y", "dx", "ddt", "dz") if train else ("y",))}
    res.update({k: torch.zeros(B * T, G, N, **f64) for k in (("db", "dc") if train else ())})
    ht, dh0, dA = torch.zeros_like(h0), torch.zeros_like(h0), torch.zeros(D, N, **f64)
    dskip, dbias = torch.zeros(D, **f64), torch.zeros(D, **f64)

    def spread(r):   # [sequences, G, 1, N] -> [sequences, D, N]
        return r.expand(-1, G, M, N).reshape(-1, D, N)

    for ids, L in groups:
        at = torch.tensor([spans[i][0] for i in ids], device=dev)
        h = h0[ids]
        before = torch.zeros(L, *h.shape, **f64) if train else None
        for t in range(L):
            k = at + t
            raw, x, z = flat["dt"][k] + bias, flat["x"][k], flat["z"][k]
            delta = torch.nn.functional.softplus(raw, threshold=1e9)
            if train:
                before[t] = h
            h = torch.exp(delta[..., None] * A) * h + (delta * x)[..., None] * spread(rows["b"][k])
            res["y"][k] = ((h * spread(rows["c"][k])).sum(-1) + skip * x) * z / (1 + torch.exp(-z))
        ht[ids] = h
        if not train:
            continue
        g = dht[ids]
        for t in reversed(range(L)):
            k = at + t
            raw, x, z, dy = flat["dt"][k] + bias, flat["x"][k], flat["z"][k], flat["dy"][k]
            delta = torch.nn.functional.softplus(raw, threshold=1e9)
            bt, ct = spread(rows["b"][k]), spread(rows["c"][k])
            a = torch.exp(delta[..., None] * A)
            h = a * before[t] + (delta * x)[..., None] * bt
            sg = 1 / (1 + torch.exp(-z))
            d0 = dy * z * sg
            res["dz"][k] = dy * ((h * ct).sum(-1) + skip * x) * (sg + z * sg * (1 - sg))
            g = g + d0[..., None] * ct
            res["dc"][k] = (d0[..., None] * h).view(-1, G, M, N).sum(2)
            res["db"][k] = (g * (delta * x)[..., None]).view(-1, G, M, N).sum(2)
            gb = (g * bt).sum(-1)
            res["dx"][k] = gb * delta + skip * d0
            dskip += (d0 * x).sum(0)
            g = g * a
            w = g * before[t]
            dr = (gb * x + (w * A).sum(-1)) * torch.sigmoid(raw)
            res["ddt"][k] = dr
            dbias += dr.sum(0)
            dA += (w * delta[..., None]).sum(0)
        dh0[ids] = g
    out = {k: v.view(B, T, *v.shape[1:]) for k, v in res.items()}
    out["ht"] = ht
    if train:
        out.update(dA_log=dA * A, dd_skip=dskip, ddt_bias=dbias)
        if s["h0"] is not None:
            out["dh0"] = dh0
    return out


def _exact_norm(s):
    h, w, D = _d(s["x"]), _d(s["weight"]), s["D"]
    if s["dir"] == "back":
        dy = _d(s["dy"])
        r = 1 / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + _EPS)
        u = h * r
        v = dy * w
        dx = r * (v - u * (u * v).mean(-1, keepdim=True))
        return {"dx": dx if s["residual"] is None else dx + _d(s["residual"]), "dweight": (dy * u).sum(0)}
    if s["residual"] is not None:
        h = h + _d(s["residual"])
    y = h / torch.sqrt(h.pow(2).mean(-1, keepdim=True) + _EPS) * w
    out = {} if s["residual"] is None else {"h": h}
    if s["out"] == "io":
        return {"y": y, **out}
    group = s["group"] or D
    scale = torch.stack([c.abs().amax(-1) for c in y.split(group, -1)], -1) / _E4M3_MAX
    # the nearest values of 3 bits after the leading one, steps of 2^-9 below 2^-6; ties to even
    v = y / scale.repeat_interleave(group, -1)[:, :D].clamp(min=1e-300)
    quantum = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return {"y": torch.round(v / quantum) * quantum, "scale": scale, **out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "ssm": _exact_ssm, "norm": _exact_norm}[case["op"]](s)
