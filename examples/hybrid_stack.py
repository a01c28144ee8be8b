"""A hybrid stack: recurrent blocks with softmax-attention blocks between them, as models mix them, with random weights.

    python examples/hybrid_stack.py

The recurrent blocks are those of examples/token_mixer.py. An attention block is norm -> projection to q, k, v ->
norms of q and k with the position rotation, k and v into a paged cache -> attention over the cache -> gate ->
projection. The script

1. runs packed prompts of several lengths and keeps every block's state: recurrence and convolution states, or the
   pages of the attention blocks' caches (8-bit values with one power of two per row),
2. continues all sequences together token by token, and in one go over several tokens as when drafted tokens are
   verified, and compares with one pass over prompt and continuation,
3. takes gradients of an attention block through the norms' backward call.

The projections, and attention where gradients are taken, are torch; everything else is this library.
"""

from __future__ import annotations

import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path[:0] = [os.path.dirname(HERE), HERE]

import token_mixer as tm  # noqa: E402
from chunkwise_gated_linear_gb300 import (KVCache, block_norm_fwd, paged_attn_step, qk_norm_bwd, qk_norm_fwd,  # noqa: E402
                                          qk_norm_step, rope_frequencies)

DIM, Q_HEADS, KV_HEADS, HEAD, ROTATED, PAGE = tm.DIM, 4, 2, 64, 32, 16
BF, F32 = torch.bfloat16, torch.float32


def attention_weights(g, dev):
    n = lambda *s: (torch.randn(*s, generator=g) * s[0] ** -0.5).to(dev, BF)  # noqa: E731
    ones = lambda k: torch.ones(k, device=dev)  # noqa: E731
    return dict(kind="attn", qkv=n(DIM, (Q_HEADS + 2 * KV_HEADS) * HEAD), gate=n(DIM, Q_HEADS * HEAD), out=n(Q_HEADS * HEAD, DIM),
                q_norm=ones(HEAD) * 1.5, k_norm=ones(HEAD) * 1.5, post=ones(DIM), scale=torch.full((DIM,), 0.5, device=dev),
                next_norm=ones(DIM))


class Pages:
    """What the attention blocks share: a table of pages that covers each sequence's whole length, and the lengths so far."""

    def __init__(self, most, dev, kind):
        need = [-(-n // PAGE) for n in most]
        order = torch.randperm(sum(need), generator=torch.Generator().manual_seed(5)).to(torch.int32)
        self.table = torch.zeros(len(most), max(need), dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.table = self.table.to(dev)
        self.count, self.kind, self.dev = sum(need), kind, dev
        self.lens = torch.zeros(len(most), dtype=torch.int32, device=dev)
        self.freq = rope_frequencies(ROTATED, device=dev)

    def cache(self):
        return KVCache.empty(self.count, KV_HEADS, PAGE, HEAD, self.kind, device=self.dev)


def attend(w, x, cache, pages, cu):
    """An attention block's mixer on the normed stream x [B, T, DIM] (packed prompts with ``cu``); pages.lens
    counts these tokens already."""
    qkv = x @ w["qkv"]
    q, k, v = (t.unflatten(-1, (-1, HEAD)) for t in qkv.split([Q_HEADS * HEAD, KV_HEADS * HEAD, KV_HEADS * HEAD], dim=-1))
    q = qk_norm_step(q, k, v, cache, pages.table, pages.lens, w["q_norm"], w["k_norm"], pages.freq, cu_seqlens=cu)
    if cu is None:
        o = paged_attn_step(q, cache, pages.table, pages.lens)
    else:  # prompts: each sequence's tokens over its own pages
        ends = cu.tolist()
        o = torch.cat([paged_attn_step(q[:, s:e], cache, pages.table[b:b + 1], pages.lens[b:b + 1])
                       for b, (s, e) in enumerate(zip(ends, ends[1:]))], dim=1)
    gate = torch.sigmoid(x @ w["gate"])
    return (o.flatten(2) * gate) @ w["out"]


def forward(blocks, stream, states, pages, cu=None):
    """The residual stream [B, T, DIM] (fp32) through all blocks; returns the last norm's output and the new states."""
    out = []
    x, stream = block_norm_fwd(torch.zeros_like(stream, dtype=BF), stream, torch.ones(DIM, device=stream.device))
    for w, state in zip(blocks, states):
        if w["kind"] == "attn":
            y = attend(w, x, state, pages, cu)
        else:
            y, state = tm.mix(w, x, state, cu)
        out.append(state)
        x, stream = block_norm_fwd(y, stream, w["next_norm"], post_weight=w["post"], scale=w["scale"])
    return x, out


def serve(dev="cuda", lengths=(70, 1, 200, 33), extra=5, seed=0, kind=torch.float8_e4m3fn, at_once=1):
    """Prompts, then ``extra`` more tokens of every sequence, ``at_once`` in a step; returns the largest relative difference
    to one pass over everything."""
    g = torch.Generator().manual_seed(seed)
    blocks = [attention_weights(g, dev) if k == "attn" else tm._weights(g, dev, k) for k in ("kda", "attn", "ssm", "attn")]
    tokens = [torch.randn(n + extra, DIM, generator=g).to(dev) for n in lengths]
    offsets = lambda ns: torch.tensor([0, *torch.tensor(ns).cumsum(0)], dtype=torch.int32, device=dev)  # noqa: E731

    def prompts(ns):
        pages = Pages([n + extra for n in lengths], dev, kind)
        pages.lens += torch.tensor(ns, dtype=torch.int32, device=dev)
        states = [pages.cache() if w["kind"] == "attn" else None for w in blocks]
        x, states = forward(blocks, torch.cat([t[:n] for t, n in zip(tokens, ns)])[None], states, pages, offsets(ns))
        return x, states, pages

    want, _, _ = prompts([n + extra for n in lengths])
    _, states, pages = prompts(list(lengths))
    worst = 0.0
    first = torch.tensor([n + extra for n in lengths]).cumsum(0) - extra
    for k in range(0, extra, at_once):
        new = min(at_once, extra - k)
        pages.lens += new
        got, states = forward(blocks, torch.stack([t[n + k:n + k + new] for t, n in zip(tokens, lengths)]).contiguous(), states, pages)
        for i in range(new):
            ref = want[0, first + k + i].float()
            worst = max(worst, float((got[:, i].float() - ref).norm() / ref.norm()))
    return worst


class _QkNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_norm, k_norm, freq):
        ctx.save_for_backward(q, k, q_norm, k_norm, freq)
        return qk_norm_fwd(q, k, q_norm, k_norm, freq)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, q_norm, k_norm, freq = ctx.saved_tensors
        return *qk_norm_bwd(q, k, q_norm, k_norm, freq, dq.contiguous(), dk.contiguous()), None


def loss(qkv, q_norm, k_norm, target, norm):
    """Causal attention from a projection qkv [B, T, ...] and its distance to a target; ``norm`` is what turns q and k
    (the library's function above, or a plain one)."""
    B, T, _ = qkv.shape
    q, k, v = (t.unflatten(-1, (-1, HEAD)) for t in qkv.split([Q_HEADS * HEAD, KV_HEADS * HEAD, KV_HEADS * HEAD], dim=-1))
    q, k = norm(q, k, q_norm, k_norm)
    k, v = (t.repeat_interleave(Q_HEADS // KV_HEADS, dim=2) for t in (k, v))
    s = torch.einsum("bqhd,bkhd->bhqk", q, k) * HEAD ** -0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=qkv.device).triu(1), float("-inf"))
    return (torch.einsum("bhqk,bkhd->bqhd", torch.softmax(s, -1), v) - target).pow(2).mean()


def gradients(dev="cuda", seed=1):
    """Inputs of :func:`loss` (fp32) and their gradients through the library's calls."""
    g = torch.Generator().manual_seed(seed)
    args = [torch.randn(2, 33, (Q_HEADS + 2 * KV_HEADS) * HEAD, generator=g), 1 + 0.2 * torch.randn(HEAD, generator=g),
            1 + 0.2 * torch.randn(HEAD, generator=g)]
    target = torch.randn(2, 33, Q_HEADS, HEAD, generator=g)
    leaves = [t.to(dev).requires_grad_() for t in args]
    freq = rope_frequencies(ROTATED, device=dev)
    value = loss(*leaves, target.to(dev), lambda q, k, a, b: _QkNorm.apply(q, k, a, b, freq))
    return args, target, torch.autograd.grad(value, leaves)


if __name__ == "__main__":
    print(f"single tokens against one pass: relative difference {serve():.2e} (cache in bf16: {serve(kind=BF):.2e})")
    print(f"several tokens at once: {serve(extra=8, at_once=4):.2e}")
    print("gradients of an attention block:", ", ".join(f"{float(t.norm()):.3e}" for t in gradients()[2]))
