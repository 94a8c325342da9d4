"""A small hybrid language model on this library's operators: layers of the gated
delta rule and of the selective state space scan in turn, each behind a norm that
takes in the residual stream and a short causal convolution.

    python examples/hybrid_stack.py

trains it for some steps on packed sequences (a token repeats after a fixed lag),
then serves it: prompts of several lengths are packed into one row and prefilled,
and every sequence goes on token by token, its states updated in place. Serving
and training run the same weights; the last lines compare the logits of a served
continuation with one pass over the whole sequences.
"""

from __future__ import annotations

import os
import sys

import torch
import torch.nn.functional as F
from torch import nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunkwise_delta_rule_gb300 as kda  # noqa: E402


def _param(*shape, std=1.0):
    return nn.Parameter(torch.randn(*shape) * std)


class Conv(nn.Module):
    """The short convolution with SiLU; `cache` holds a serving state [N, W - 1, D]."""

    def __init__(self, D, W=4):
        super().__init__()
        self.weight, self.bias = _param(D, W, std=W ** -0.5), nn.Parameter(torch.zeros(D))

    def forward(self, x, cu, cache):
        if cache is None:
            return kda.short_conv(x, self.weight, self.bias, cu_seqlens=cu)[0]
        state = cache.get("conv")
        p = kda.make_conv_problem(x, self.weight, self.bias, initial_state=state, cu_seqlens=cu)
        y, cache["conv"] = kda.kda_conv_fwd(p, final_state=state)
        return y


class DeltaLayer(nn.Module):
    """Gated delta rule with a per-channel gate: q, k and v through one convolution."""

    def __init__(self, D, heads, width):
        super().__init__()
        self.heads, self.width, inner = heads, width, heads * width
        self.inp, self.out = _param(4 * inner + heads, D, std=D ** -0.5), _param(D, inner, std=inner ** -0.5)
        self.conv = Conv(3 * inner)
        self.A_log = nn.Parameter(torch.linspace(-1.0, 1.0, heads))
        self.dt_bias = nn.Parameter(torch.full((heads, width), -3.0))

    def forward(self, x, cu, cache):
        H, K, inner = self.heads, self.width, self.heads * self.width
        p = F.linear(x, self.inp.to(x.dtype))
        qkv = self.conv(p[..., :3 * inner], cu, cache)
        q, k, v = (t.reshape(*x.shape[:2], H, K).contiguous() for t in qkv.split(inner, -1))
        g = p[..., 3 * inner:4 * inner].reshape(*x.shape[:2], H, K).float().contiguous()
        beta = torch.sigmoid(p[..., 4 * inner:]).contiguous()
        kw = dict(gate="channel", A_log=self.A_log, dt_bias=self.dt_bias, cu_seqlens=cu)
        if cache is None:
            o, _ = kda.chunk_kda(q, k, v, g, beta, use_qk_l2norm_in_kernel=True, **kw)
        else:
            state = cache.get("state")
            prob = kda.make_problem(q, k, v, g, beta, initial_state=state, qk_l2norm=True, **kw)
            if state is None:
                o, cache["state"], _ = kda.kda_chunk_fwd(prob)
            else:
                o, _ = kda.kda_recurrent_fwd(prob, ht=state)
        return F.linear(o.reshape(*x.shape[:2], inner), self.out.to(x.dtype))


class ScanLayer(nn.Module):
    """Selective state space scan, gated: steps, b and c are projections of its input."""

    def __init__(self, D, inner, states, rank):
        super().__init__()
        self.states, self.rank = states, rank
        self.inp, self.out = _param(2 * inner, D, std=D ** -0.5), _param(D, inner, std=inner ** -0.5)
        self.sel, self.dt = _param(rank + 2 * states, inner, std=inner ** -0.5), _param(inner, rank, std=rank ** -0.5)
        self.conv = Conv(inner)
        self.A_log = nn.Parameter(torch.log(torch.arange(1.0, states + 1)).repeat(inner, 1))
        self.dt_bias, self.d_skip = nn.Parameter(torch.full((inner,), -4.0)), nn.Parameter(torch.ones(inner))

    def forward(self, x, cu, cache):
        u, z = F.linear(x, self.inp.to(x.dtype)).chunk(2, -1)
        u = self.conv(u, cu, cache)
        r, b, c = F.linear(u, self.sel.to(x.dtype)).split([self.rank, self.states, self.states], -1)
        dt = F.linear(r, self.dt.to(x.dtype))
        b, c = b.unsqueeze(2), c.unsqueeze(2)   # one group
        kw = dict(d_skip=self.d_skip, z=z, dt_bias=self.dt_bias, cu_seqlens=cu)
        if cache is None:
            y, _ = kda.ssm_scan(u, dt, self.A_log, b, c, **kw)
        else:
            state = cache.get("state")
            y, cache["state"], _ = kda.kda_ssm_fwd(
                kda.make_ssm_problem(u, dt, self.A_log, b, c, initial_state=state, **kw), ht=state)
        return F.linear(y, self.out.to(x.dtype))


class HybridStack(nn.Module):
    """`forward(tokens, cu)` for training, with `caches` (one dict per layer) for serving."""

    def __init__(self, vocab=64, D=128, layers=4, heads=2, width=64, states=16):
        super().__init__()
        self.embed = _param(vocab, D, std=D ** -0.5)
        self.norms = nn.ParameterList([nn.Parameter(torch.ones(D)) for _ in range(layers + 1)])
        self.layers = nn.ModuleList([DeltaLayer(D, heads, width) if i % 2 == 0 else ScanLayer(D, 2 * D, states, D // 16)
                                     for i in range(layers)])

    def forward(self, tokens, cu=None, caches=None, dtype=torch.bfloat16):
        x, stream = F.embedding(tokens, self.embed).to(dtype), None
        for i, norm in enumerate(self.norms):
            if caches is None:
                x, stream = kda.rms_norm(x, norm, residual=stream)
            else:   # the sum takes the residual stream's own buffer
                x, _, stream = kda.kda_norm_fwd(kda.make_norm_problem(x, norm, residual=stream), h=stream)
            if i < len(self.layers):
                x = self.layers[i](x, cu, None if caches is None else caches[i])
        return F.linear(x, self.embed.to(dtype))


def packed_batch(lengths, vocab, lag, gen, device):
    """Sequences that repeat themselves after `lag` tokens, packed into one row."""
    rows = []
    for n in lengths:
        head = torch.randint(vocab, (lag,), generator=gen)
        rows.append(head.repeat(n // lag + 1)[:n])
    cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=device)
    return torch.cat(rows).unsqueeze(0).to(device), cu


def train(model, steps, lengths=(300, 45, 167), lag=4, vocab=64, seed=0):
    """Some steps of training; returns the losses."""
    device, gen = model.embed.device, torch.Generator().manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        tokens, cu = packed_batch(lengths, vocab, lag, gen, device)
        logits = model(tokens, cu)[0, :-1].float()
        loss_rows = F.cross_entropy(logits, tokens[0, 1:], reduction="none")
        inside = torch.ones_like(loss_rows)
        inside[cu[1:-1].long() - 1] = 0   # the last token of a sequence does not predict the next sequence's first
        loss = (loss_rows * inside).sum() / inside.sum()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def serve(model, prompts, cu, steps, dtype=torch.bfloat16, forced=None):
    """Prefill the packed prompts, then `steps` tokens for every sequence, the likeliest each time (or those
    of `forced` [N, steps]). Returns the tokens [N, steps] and the logits they were taken from."""
    caches = [dict() for _ in model.layers]
    logits = model(prompts, cu, caches, dtype)[0][cu[1:].long() - 1]
    tokens, seen = [], []
    for t in range(steps):
        nxt = logits.argmax(-1) if forced is None else forced[:, t]
        tokens.append(nxt)
        seen.append(logits)
        logits = model(nxt.unsqueeze(1), None, caches, dtype)[:, 0]
    return torch.stack(tokens, 1), torch.stack(seen, 1)


@torch.no_grad()
def agreement(model, lengths=(37, 130, 4), steps=24, dtype=torch.bfloat16, lag=4, vocab=64, seed=1):
    """Normwise difference between the logits of a served continuation and those of one pass over the whole
    sequences, and the share of served tokens that repeat the sequence."""
    gen = torch.Generator().manual_seed(seed)
    whole, cu = packed_batch([n + steps for n in lengths], vocab, lag, gen, model.embed.device)
    rows = [whole[0, a:b] for a, b in zip(cu[:-1].tolist(), cu[1:].tolist())]
    short = torch.cat([r[:n] for r, n in zip(rows, lengths)]).unsqueeze(0)
    cu_short = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device=whole.device)
    forced = torch.stack([r[n:] for r, n in zip(rows, lengths)])
    _, served = serve(model, short, cu_short, steps, dtype, forced)
    full = model(whole, cu, None, dtype)[0]
    want = torch.stack([full[a + n - 1:a + n - 1 + steps] for a, n in zip(cu[:-1].tolist(), lengths)])
    diff = (served.double() - want.double()).norm() / want.double().norm()
    told = torch.tensor([n >= lag for n in lengths], device=whole.device)   # the lag was seen once
    hits = (served.argmax(-1) == forced)[told].float().mean()
    return diff.item(), hits.item()


def main():
    torch.manual_seed(0)
    model = HybridStack().cuda()
    losses = train(model, 300)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    diff, hits = agreement(model)
    print(f"serving: {100 * hits:.1f}% of the served tokens repeat their sequence; "
          f"logits against one pass over the whole sequences: {diff:.1e}")


if __name__ == "__main__":
    main()
