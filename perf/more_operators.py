"""Cases of linear attention with a decay for each head, of the matrix product of
8-bit values with a scale for each block of 128, and of the rounding to those
8-bit values.

``run`` computes a case in its plain form (torch operations in 32 bits, one
rounding at the end) or, with ``own`` true, through the package's entry points;
``exact`` computes it from the definition in 64 bits.

Linear attention works on [B, T, heads, width] tensors of equal-length sequences,
or on a packed token axis: sequence n owns the tokens cu[n] .. cu[n+1]-1 of a
[1, total, ...] tensor. Values have HV heads, HV / H of which share a head of
queries and keys.
"""

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
_E4M3_MAX = 448.0
_C = 64       # tokens of a chunk of the plain form
_G = 128      # columns of a scale's group


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of each of 64 sequences, the states updated in place
        dict(name="lin_step", op="lin", dir="step", io="bf16", B=64, T=1, H=32, HV=32, K=128, V=128, state=True, nseq=0, sliced=True),
        # prompts: two long sequences, 32 heads; their final states go on to decoding
        dict(name="lin_prompt", op="lin", dir="fwd", io="bf16", B=2, T=8192, H=32, HV=32, K=128, V=128, state=False, nseq=0, sliced=False),
        # a packed prefill of resumed ragged prompts (an empty one and one of a single token among them), two value
        # heads to a key head, queries, keys and values as columns of one projection's rows
        dict(name="lin_packed", op="lin", dir="fwd", io="bf16", B=1, T=32768, H=8, HV=16, K=128, V=128, state=True, nseq=9, sliced=True),
        # few narrow heads and many tokens (one shard of a wide layer): the time axis is the long one
        dict(name="lin_long", op="lin", dir="fwd", io="bf16", B=1, T=32768, H=4, HV=4, K=64, V=64, state=False, nseq=0, sliced=False),
        # a training step's forward and backward
        dict(name="lin_train", op="lin", dir="train", io="bf16", B=4, T=4096, H=16, HV=16, K=128, V=128, state=False, nseq=0, sliced=False),
        # 32-bit training with odd widths and lengths, carried states
        dict(name="lin_odd", op="lin", dir="train", io="fp32", B=3, T=777, H=5, HV=10, K=40, V=72, state=True, nseq=0, sliced=False),
        # the projection of one token of each of 64 sequences: rows as the norm's 8-bit output has them
        dict(name="mm_step", op="mm", M=64, N=4096, K=4096, b="blocks", out="bf16"),
        # the same for a batch of prompts
        dict(name="mm_prompt", op="mm", M=16384, N=4096, K=4096, b="blocks", out="bf16"),
        # a weight's gradient: both sides in rows of 128 tokens
        dict(name="mm_grad", op="mm", M=4096, N=4096, K=16384, b="rows", out="fp32"),
        # sizes that end inside tiles and groups, rows that start on odd addresses
        dict(name="mm_odd", op="mm", M=777, N=1000, K=1111, b="blocks", out="fp32"),
        # a layer's activations for the forward (rows) and for the weight's gradient (the transposed copy)
        dict(name="quant_rows", op="quant", io="bf16", R=16384, D=4096, blocks=False, transposed=True),
        # a weight for the forward and for the input's gradient, once per training step
        dict(name="quant_blocks", op="quant", io="fp32", R=4096, D=4096, blocks=True, transposed=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("lin", "lin", "mm", "quant"))
    if op == "mm":
        case = dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 16, 8192), K=_log(rng, 16, 8192),
                    b=rng.choice(("blocks", "blocks", "rows")), out=rng.choice(("bf16", "fp32")))
        if rng.random() < 0.6:
            case["K"] = max(128, case["K"] // 128 * 128)
            case["N"] = max(16, case["N"] // 16 * 16)
        case["M"] = max(1, min(case["M"], 16384 * 4096 * 4096 // (case["N"] * case["K"])))
        return case
    io = rng.choice(("bf16", "bf16", "fp32"))
    if op == "quant":
        case = dict(op=op, io=io, R=_log(rng, 1, 16384), D=_log(rng, 16, 8192), blocks=rng.random() < 0.4,
                    transposed=rng.random() < 0.6)
        case["R"] = max(1, min(case["R"], 16384 * 4096 // case["D"]))
        return case
    direction = rng.choice(("fwd", "fwd", "train", "step"))
    packed = direction != "step" and rng.random() < 0.4
    if direction == "step":
        B, T = _log(rng, 1, 256), 1
    elif packed:
        B, T = 1, _log(rng, 16, 32768)
    else:
        B, T = rng.randint(1, 8), _log(rng, 2, 8192)
    H, group = _log(rng, 1, 32), rng.choice((1, 1, 2, 4))
    K = rng.choice((64, 128, 128, _log(rng, 8, 128)))
    V = rng.choice((64, 128, 128, _log(rng, 8, 256)))
    if rng.random() < 0.6:
        K, V = K // 8 * 8, V // 8 * 8
    most = 4 * 4096 * 16 * 128 * 128 if direction == "train" else 2 * 8192 * 32 * 128 * 128
    if io == "fp32":
        most //= 4
    unit = H * group * K * V
    if B * T * unit > most:
        if direction == "step":
            B = max(1, most // unit)
        else:
            T = max(2, most // (unit * B))
    return dict(op=op, dir=direction, io=io, B=B, T=T, H=H, HV=H * group, K=K, V=V,
                state=direction == "step" or rng.random() < 0.5, nseq=rng.randint(1, 12) if packed else 0,
                sliced=rng.random() < 0.5)


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _cuts(gen, total, nseq):
    """Offsets of nseq packed sequences: random cuts, an empty sequence and one of a single token where they fit."""
    inner = torch.sort(torch.randint(0, total + 1, (nseq - 1,), generator=gen, device="cuda")).values
    if nseq >= 4:
        inner[1] = inner[0]
        inner[2] = (inner[1] + 1).clamp(max=total)
        inner = torch.sort(inner).values
    ends = torch.tensor([0, total], device="cuda")
    return torch.cat([ends[:1], inner, ends[1:]]).to(torch.int32)


def _outliers(gen, R, D):
    """Activations with a few columns of large values, as trained models have them."""
    return _randn(gen, R, D) * torch.where(torch.rand(D, generator=gen, device="cuda") < 0.01, 16.0, 1.0)


def prepare(case, seed):
    gen = _gen(seed)
    s = dict(case)
    if case["op"] == "quant":
        R, D = case["R"], case["D"]
        s["x"] = (0.02 * _randn(gen, R, D) if case["blocks"] else _outliers(gen, R, D)).to(_DT[case["io"]])
        return s
    if case["op"] == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"], s["sa"] = _round8(_outliers(gen, M, K), 1)
        s["w"], s["sb"] = _round8(0.02 * _randn(gen, N, K), _G if case["b"] == "blocks" else 1)
        return s
    B, T, H, HV, K, V, dt = (case[k] for k in ("B", "T", "H", "HV", "K", "V", "io"))
    dt = _DT[dt]
    widths = (H * K, H * K, HV * V)
    parts = [_randn(gen, B, T, w).to(dt) for w in widths]
    if case["sliced"]:
        parts = list(torch.cat(parts, -1).split(widths, -1))
    s["q"], s["k"] = parts[0].unflatten(-1, (H, K)), parts[1].unflatten(-1, (H, K))
    s["v"] = parts[2].unflatten(-1, (HV, V))
    # the heads' decays as slopes from 2^-1 down to 2^-8 per token
    h = torch.arange(HV, device="cuda", dtype=torch.float32)
    s["decay"] = -torch.exp2(-1 - 7 * h / max(1, HV - 1))
    s["cu"] = _cuts(gen, B * T, case["nseq"]) if case["nseq"] else None
    n = case["nseq"] or B
    s["h0"] = _randn(gen, n, HV, K, V) if case["state"] else None
    if case["dir"] == "train":
        s["do"] = _randn(gen, B, T, HV, V).to(dt)
        s["dht"] = _randn(gen, n, HV, K, V) if case["state"] else None
    return s


# ------------------------------------------------------------------- plain forms

def _round8(x, rows):
    """x in e4m3 with a scale for each group of `rows` rows (1 or 128) and 128 columns: amax / 448."""
    R, D = x.shape
    gr, gd = -(-R // rows), -(-D // _G)
    pad = x.new_zeros(gr * rows, gd * _G)
    pad[:R, :D] = x
    pad = pad.view(gr, rows, gd, _G)
    amax = pad.abs().amax((1, 3), keepdim=True)
    inv = torch.where(amax > 0, _E4M3_MAX / amax, 0.0)
    q = (pad * inv).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(gr * rows, gd * _G)[:R, :D].contiguous(), (amax / _E4M3_MAX).view(gr, gd)


def _plain_quant(s):
    x = s["x"].float()
    rows = _G if s["blocks"] else 1
    q, scale = _round8(x, rows)
    if not s["transposed"]:
        return {"q": q, "scale": scale}
    if s["blocks"]:
        return {"q": q, "scale": scale, "qt": q.t().contiguous(), "scale_t": scale.t().contiguous()}
    qt, scale_t = _round8(x.t(), 1)
    return {"q": q, "scale": scale, "qt": qt, "scale_t": scale_t}


def _plain_mm(s):
    N, K = s["N"], s["K"]
    a = s["a"].float() * s["sa"].repeat_interleave(_G, 1)[:, :K]
    sb = s["sb"].repeat_interleave(_G, 1)[:, :K]
    if s["b"] == "blocks":
        sb = sb.repeat_interleave(_G, 0)[:N]
    return {"y": (a @ (s["w"].float() * sb).t()).to(_DT[s["out"]])}


def _slots(s):
    """Chunks of 64 tokens that start at every sequence's first: each token's place, each chunk's sequence, its place in
    it and its tokens, each sequence's length. Chunks past the last one belong to no sequence (number n)."""
    total, n = s["B"] * s["T"], s["nseq"] or s["B"]
    if s["cu"] is not None:
        first, length = s["cu"][:-1].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    else:
        first = torch.arange(n, device="cuda") * s["T"]
        length = torch.full_like(first, s["T"])
    chunks = (length + _C - 1) // _C
    start = torch.cumsum(chunks, 0) - chunks
    nc = -(-s["T"] // _C) * s["B"] if s["cu"] is None else -(-total // _C) + n
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), length, output_size=total)
    place = start[seq] * _C + torch.arange(total, device="cuda") - first[seq]
    ids = torch.arange(nc, device="cuda")
    owner = torch.searchsorted(torch.cumsum(chunks, 0), ids, right=True)
    at = ids - torch.cat([start, start[-1:]])[owner]
    tokens = (torch.cat([length, length.new_zeros(1)])[owner] - at * _C).clamp(0, _C)
    return place, owner, at, tokens, length, nc


def _plain_lin(s):
    """Chunk by chunk: scores inside a chunk, and the state entering it, a weighted sum of the chunks' own states."""
    B, T, HV, K, V = (s[k] for k in ("B", "T", "HV", "K", "V"))
    place, owner, at, tokens, length, nc = _slots(s)
    n, io, scale, g = length.numel(), s["q"].dtype, K ** -0.5, s["decay"]

    def chunks(x):   # [B, T, heads, width] -> [HV, chunks, 64, width]
        x = x.reshape(B * T, x.shape[2], x.shape[3]).float()
        pad = x.new_zeros(nc * _C, *x.shape[1:])
        pad[place] = x
        return pad.view(nc, _C, *x.shape[1:]).permute(2, 0, 1, 3).repeat_interleave(HV // x.shape[1], 0)

    def tokens_of(x, heads):   # back, the value heads of a key head added up
        x = x.view(heads, HV // heads, nc * _C, x.shape[-1]).sum(1)[:, place]
        return x.permute(1, 0, 2).to(io).view(B, T, heads, x.shape[-1])

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    i = torch.arange(_C, device="cuda")
    gh = g.view(HV, 1, 1)
    away = (i[:, None] - i[None, :])
    mask = torch.where(away >= 0, torch.exp(gh * away.clamp(min=0)), 0.0)[:, None]
    to_end = (tokens[:, None] - 1 - i).clamp(min=0)
    e = torch.exp(gh * to_end)[..., None]                       # [HV, chunks, 64, 1]
    gam = torch.exp(gh * (i + 1))[..., None]                    # [HV, 1, 64, 1]
    c = torch.arange(nc, device="cuda")
    before = (owner[:, None] == owner[None, :]) & (c[None, :] < c[:, None])
    enter = torch.where(before, torch.exp(gh * (_C * (c[:, None] - c[None, :] - 1)).clamp(min=0)), 0.0)
    mine = owner[None, :] == torch.arange(n, device="cuda")[:, None]
    left = (length[:, None] - at[None, :] * _C - tokens[None, :]).clamp(min=0)
    leave = torch.where(mine, torch.exp(gh * left), 0.0)        # [HV, n, chunks]
    carry = torch.exp(gh * (at * _C)[None, None])[:, 0, :, None, None]
    whole = torch.exp(g[None, :] * length[:, None])[..., None, None]
    h0 = q.new_zeros(n, HV, K, V) if s["h0"] is None else s["h0"]
    h0c = torch.cat([h0, h0.new_zeros(1, HV, K, V)])[owner].transpose(0, 1)
    kv = (k * e).transpose(2, 3) @ v
    state = (enter @ kv.view(HV, nc, K * V)).view(HV, nc, K, V) + carry * h0c
    ht = (leave @ kv.view(HV, nc, K * V)).view(HV, n, K, V).transpose(0, 1) + whole * h0
    p = (q @ k.transpose(2, 3)) * mask
    o = scale * (gam * (q @ state) + p @ v)
    if s["dir"] == "step":
        ht = s["h0"].copy_(ht)
    out = {"o": tokens_of(o, HV), "ht": ht.contiguous()}
    if s["dir"] != "train":
        return out
    do = chunks(s["do"])
    dstate = scale * (q * gam).transpose(2, 3) @ do
    dht = q.new_zeros(n, HV, K, V) if s["dht"] is None else s["dht"]
    dkv = (enter.transpose(1, 2) @ dstate.view(HV, nc, K * V)
           + leave.transpose(1, 2) @ dht.transpose(0, 1).reshape(HV, n, K * V)).view(HV, nc, K, V)
    ds = (do @ v.transpose(2, 3)) * mask
    dq = scale * (gam * (do @ state.transpose(2, 3)) + ds @ k)
    dk = scale * (ds.transpose(2, 3) @ q) + e * (v @ dkv.transpose(2, 3))
    dv = scale * (p.transpose(2, 3) @ do) + e * (k @ dkv)
    out.update(dq=tokens_of(dq, s["H"]), dk=tokens_of(dk, s["H"]), dv=tokens_of(dv, HV))
    if s["h0"] is not None:
        part = torch.where(mine, torch.exp(gh * (at * _C)[None, None]), 0.0) @ dstate.view(HV, nc, K * V)
        out["dh0"] = part.view(HV, n, K, V).transpose(0, 1) + whole * dht
    return out


# ------------------------------------------------------------------- one pass

def _own_quant(s):
    import chunkwise_delta_rule_gb300 as kda
    r = kda.kda_quant8(kda.make_quant8_problem(s["x"], blocks=s["blocks"], transposed=s["transposed"]))
    out = {"q": r.q, "scale": r.scale}
    return {**out, "qt": r.qt, "scale_t": r.scale_t} if s["transposed"] else out


def _own_mm(s):
    import chunkwise_delta_rule_gb300 as kda
    return {"y": kda.kda_mm8(kda.make_mm8_problem(s["a"], s["sa"], s["w"], s["sb"], out=s["out"]))}


def _own_lin(s):
    import chunkwise_delta_rule_gb300 as kda
    p = kda.make_lin_problem(s["q"], s["k"], s["v"], s["decay"], initial_state=s["h0"], cu_seqlens=s["cu"])
    o, ht = kda.kda_lin_fwd(p, ht=s["h0"] if s["dir"] == "step" else None)
    out = {"o": o, "ht": ht}
    if s["dir"] != "train":
        return out
    g = kda.kda_lin_bwd(p, s["do"], s["dht"])
    out.update(dq=g.dq, dk=g.dk, dv=g.dv)
    return out if s["h0"] is None else {**out, "dh0": g.dh0}


def run(state):
    if own:
        return {"lin": _own_lin, "mm": _own_mm, "quant": _own_quant}[state["op"]](state)
    return {"lin": _plain_lin, "mm": _plain_mm, "quant": _plain_quant}[state["op"]](state)


def work(case):
    if case["op"] == "quant":
        R, D = case["R"], case["D"]
        copies = 1 + case["transposed"]
        scales = 4 * (R * D / _G / _G if case["blocks"] else R * D / _G)
        return {"bytes": R * D * ((2 if case["io"] == "bf16" else 4) + copies) + copies * scales, "flops": 3 * R * D}
    if case["op"] == "mm":
        M, N, K = case["M"], case["N"], case["K"]
        scales = 4 * (M + (N if case["b"] == "rows" else N / _G)) * K / _G
        return {"bytes": M * K + N * K + scales + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}
    io = 2 if case["io"] == "bf16" else 4
    tok, n = case["B"] * case["T"], case["nseq"] or case["B"]
    row = 2 * case["H"] * case["K"] + case["HV"] * case["V"]
    outs = case["HV"] * case["V"]
    state = 4 * n * case["HV"] * case["K"] * case["V"]
    data = tok * io * (row + outs) + state * (1 + case["state"])
    flops = 4 * tok * case["HV"] * case["K"] * case["V"]
    if case["dir"] == "train":   # the backward reads the inputs and the output's gradient and writes three gradients
        data += tok * io * (2 * row + outs) + 3 * state * case["state"]
        flops += 10 * tok * case["HV"] * case["K"] * case["V"]
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------- 64 bits

def _exact_quant(s):
    """Each value by the nearest of 3 bits after the leading one (steps of 2^-9 below 2^-6; ties to even)."""
    def rounded(x, rows):
        gr, gd = -(-x.shape[0] // rows), -(-x.shape[1] // _G)
        scale = torch.nn.functional.max_pool2d(
            torch.nn.functional.pad(x.abs(), (0, gd * _G - x.shape[1], 0, gr * rows - x.shape[0]))[None], (rows, _G))[0] / _E4M3_MAX
        each = scale.repeat_interleave(rows, 0)[:x.shape[0]].repeat_interleave(_G, 1)[:, :x.shape[1]]
        v = x / each.clamp(min=1e-300)
        quantum = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        return torch.round(v / quantum) * quantum, scale

    x = s["x"].double()
    q, scale = rounded(x, _G if s["blocks"] else 1)
    out = {"q": q, "scale": scale}
    if s["transposed"]:
        out["qt"], out["scale_t"] = rounded(x.t(), _G if s["blocks"] else 1)
    return out


def _exact_mm(s):
    """One group of 128 columns after the other."""
    y = torch.zeros(s["M"], s["N"], dtype=torch.float64, device="cuda")
    for kb, at in enumerate(range(0, s["K"], _G)):
        sb = s["sb"][:, kb].double()
        if s["b"] == "blocks":
            sb = sb.repeat_interleave(_G)[:s["N"]]
        part = s["a"][:, at:at + _G].double() @ s["w"][:, at:at + _G].double().t()
        y += part * s["sa"][:, kb, None].double() * sb
    return {"y": y}


def _exact_lin(s):
    """One token after the other; equal-length sequences side by side, packed ones one by one."""
    B, T, H, HV, K, V = (s[k] for k in ("B", "T", "H", "HV", "K", "V"))
    train, scale = s["dir"] == "train", K ** -0.5
    cu = s["cu"].tolist() if s["cu"] is not None else [b * T for b in range(B + 1)]
    spans = list(zip(cu[:-1], cu[1:]))
    groups = [(list(range(B)), T)] if s["cu"] is None else [([i], hi - lo) for i, (lo, hi) in enumerate(spans)]
    flat = {k: s[k].double().reshape(B * T, s[k].shape[2], -1) for k in ("q", "k", "v") + (("do",) if train else ())}
    for k in ("q", "k"):
        flat[k] = flat[k].repeat_interleave(HV // H, 1)
    a = torch.exp(s["decay"].double()).view(HV, 1, 1)
    f64 = dict(dtype=torch.float64, device="cuda")
    h0 = torch.zeros(len(spans), HV, K, V, **f64) if s["h0"] is None else s["h0"].double()
    dht = torch.zeros_like(h0) if not train or s["dht"] is None else s["dht"].double()
    ht, dh0 = torch.zeros_like(h0), torch.zeros_like(h0)
    names = ("o", "dq", "dk", "dv") if train else ("o",)
    res = {k: torch.zeros(B * T, HV, V if k in ("o", "dv") else K, **f64) for k in names}
    for ids, L in groups:
        at = torch.tensor([spans[i][0] for i in ids], device="cuda")
        h = h0[ids]
        for t in range(L):
            j = at + t
            h = a * h + flat["k"][j][..., None] * flat["v"][j][..., None, :]
            res["o"][j] = scale * (flat["q"][j][..., None, :] @ h)[..., 0, :]
            if train:
                res["dq"][j] = scale * (h @ flat["do"][j][..., None])[..., 0]
        ht[ids] = h
        if not train:
            continue
        r = dht[ids]
        for t in reversed(range(L)):
            j = at + t
            r = r + scale * flat["q"][j][..., None] * flat["do"][j][..., None, :]
            res["dk"][j] = (r @ flat["v"][j][..., None])[..., 0]
            res["dv"][j] = (flat["k"][j][..., None, :] @ r)[..., 0, :]
            r = a * r
        dh0[ids] = r
    for k in ("dq", "dk"):
        if train:
            res[k] = res[k].view(B * T, H, HV // H, K).sum(2)
    out = {k: v.view(B, T, *v.shape[1:]) for k, v in res.items()}
    out["ht"] = ht
    return {**out, "dh0": dh0} if train and s["h0"] is not None else out


def exact(case, seed):
    s = prepare(case, seed)
    return {"lin": _exact_lin, "mm": _exact_mm, "quant": _exact_quant}[case["op"]](s)
