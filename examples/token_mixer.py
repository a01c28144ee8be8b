"""A small stack of blocks that uses the library's operators as a model does, with random weights.

    python examples/token_mixer.py

Each block is norm -> projections -> short causal convolution -> recurrence -> gated norm or gate ->
projection, with the residual update and the next block's norm in one call. The recurrence is
the gated delta rule (``kda`` blocks) or the selective state space scan (``ssm`` blocks). The script

1. runs packed prompts of several lengths and keeps every block's convolution and recurrence states,
2. continues every sequence token by token from those states and compares with one pass over prompt and
   continuation together,
3. takes a few steps of gradient descent on an ssm block through the operators' backward calls.

The projections are torch matrix products; everything else is this library.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from chunkwise_gated_linear_gb300 import (block_norm_bwd, block_norm_fwd, causal_conv_bwd, causal_conv_fwd,  # noqa: E402
                                          causal_conv_step, chunk_kda_fwd, gated_norm_fwd, selective_scan_bwd,
                                          selective_scan_fwd, selective_scan_step)

DIM, HEADS, HEAD, WIDTH = 256, 2, 128, 4        # residual width; heads of the kda blocks; taps
INNER, STATES, RANK = 384, 16, 16               # channels, states and step-size rank of the ssm blocks
BF, F32 = torch.bfloat16, torch.float32


def _weights(g, dev, kind):
    n = lambda *s, std=None, dt=BF: (torch.randn(*s, generator=g) * (std or s[0] ** -0.5)).to(dev, dt)  # noqa: E731
    ones = lambda k: torch.ones(k, device=dev)  # noqa: E731
    if kind == "kda":
        ch = 3 * HEADS * HEAD
        w = dict(inp=n(DIM, ch), gate=n(DIM, HEADS * HEAD), a=n(DIM, HEADS * HEAD), b=n(DIM, HEADS),
                 A_log=torch.zeros(HEADS, device=dev), dt_bias=n(HEADS, HEAD, std=0.1, dt=F32) - 3.0,
                 norm=ones(HEAD), out=n(HEADS * HEAD, DIM))
    else:
        ch = INNER
        w = dict(inp=n(DIM, 2 * INNER), proj=n(INNER, RANK + 2 * STATES), dt=n(RANK, INNER),
                 dt_bias=n(INNER, std=0.5, dt=F32) - 4.0,
                 A=-torch.arange(1, STATES + 1, device=dev, dtype=F32).repeat(INNER, 1).contiguous(), D=ones(INNER),
                 out=n(INNER, DIM))
    return dict(w, kind=kind, conv=n(ch, WIDTH, std=0.5, dt=F32), conv_bias=torch.zeros(ch, device=dev),
                post=ones(DIM), scale=torch.full((DIM,), 0.5, device=dev), next_norm=ones(DIM))


def _convolve(w, x, state, cu):
    """The short convolution: over packed prompts (a new state in the result), or of the next
    tokens with the state updated in place."""
    if state is None:
        return causal_conv_fwd(x, w["conv"], w["conv_bias"], cu_seqlens=cu, output_final_state=True)
    return causal_conv_step(x, state, w["conv"], w["conv_bias"]), state


def mix(w, x, state, cu):
    """One block's mixer on the normed stream x [B, T, DIM]; returns its output and states."""
    conv, rec = state if state is not None else (None, None)
    if w["kind"] == "kda":
        B, T, _ = x.shape
        y, conv = _convolve(w, x @ w["inp"], conv, cu)
        q, k, v = (t.reshape(B, T, HEADS, HEAD).contiguous() for t in y.chunk(3, dim=-1))
        a = (x @ w["a"]).float().reshape(B, T, HEADS, HEAD).contiguous()
        o, rec = chunk_kda_fwd(q, k, v, a, (x @ w["b"]).float().contiguous(), h0=rec, cu_seqlens=cu, recurrent=state is not None,
                               qk_l2norm=True, beta_sigmoid=True, A_log=w["A_log"], dt_bias=w["dt_bias"],
                               ht=rec if state is not None else None)
        z = (x @ w["gate"]).reshape(o.shape)
        return gated_norm_fwd(o, z, w["norm"]).reshape(B, T, -1) @ w["out"], (conv, rec)
    u, z = (x @ w["inp"]).chunk(2, dim=-1)  # slices: read in place
    u, conv = _convolve(w, u, conv, cu)
    low, Bm, Cm = (u @ w["proj"]).split([RANK, STATES, STATES], dim=-1)
    args = (u, low @ w["dt"], w["A"], Bm.unsqueeze(2), Cm.unsqueeze(2))
    if state is None:
        y, rec = selective_scan_fwd(*args, w["D"], z, dt_bias=w["dt_bias"], cu_seqlens=cu)
    else:
        y = selective_scan_step(*args, rec, w["D"], z, dt_bias=w["dt_bias"])
    return y @ w["out"], (conv, rec)


def forward(blocks, stream, states=None, cu=None):
    """The residual stream [B, T, DIM] (fp32) through all blocks; returns the last norm's output
    and the blocks' states."""
    out = []
    x, stream = block_norm_fwd(torch.zeros_like(stream, dtype=BF), stream, torch.ones(DIM, device=stream.device))
    for i, w in enumerate(blocks):
        y, st = mix(w, x, None if states is None else states[i], cu)
        out.append(st)
        x, stream = block_norm_fwd(y, stream, w["next_norm"], post_weight=w["post"], scale=w["scale"])
    return x, out


def serve(dev="cuda", lengths=(70, 1, 200, 33), extra=5, seed=0):
    """Prompts, then ``extra`` single tokens per sequence; returns the largest relative difference to one
    pass over everything."""
    g = torch.Generator().manual_seed(seed)
    blocks = [_weights(g, dev, kind) for kind in ("kda", "ssm", "kda", "ssm")]
    tokens = [torch.randn(n + extra, DIM, generator=g).to(dev) for n in lengths]
    offsets = lambda ns: torch.tensor([0, *torch.tensor(ns).cumsum(0)], dtype=torch.int32, device=dev)  # noqa: E731
    whole = torch.cat(tokens)[None]
    want, _ = forward(blocks, whole, cu=offsets([n + extra for n in lengths]))
    _, states = forward(blocks, torch.cat([t[:n] for t, n in zip(tokens, lengths)])[None], cu=offsets(lengths))
    worst = 0.0
    ends = torch.tensor([n + extra for n in lengths]).cumsum(0) - extra
    for k in range(extra):
        step = torch.stack([t[n + k] for t, n in zip(tokens, lengths)])[:, None]
        got, states = forward(blocks, step.contiguous(), states)
        ref = want[0, ends + k].float()
        worst = max(worst, float((got[:, 0].float() - ref).norm() / ref.norm()))
    return worst


class _Conv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        ctx.save_for_backward(x, weight, bias)
        return causal_conv_fwd(x, weight, bias)[0]

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        return causal_conv_bwd(x, weight, bias, dy.contiguous(), want_ds0=False)[:3]


class _Scan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, z, bias):
        ctx.save_for_backward(u, dt, A, B, C, D, z, bias)
        return selective_scan_fwd(u, dt, A, B, C, D, z, dt_bias=bias, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dy):
        u, dt, A, B, C, D, z, bias = ctx.saved_tensors
        du, ddt, dA, dB, dC, dD, dz, dbias, _ = selective_scan_bwd(u, dt, A, B, C, dy.contiguous(), D, z, dt_bias=bias,
                                                                   want_dh0=False)
        return du, ddt, dA, dB, dC, dD, dz, dbias


class _BlockNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, post, scale):
        ctx.save_for_backward(x, residual, weight, post, scale)
        return block_norm_fwd(x, residual, weight, post_weight=post, scale=scale)

    @staticmethod
    def backward(ctx, dy, dr):
        x, residual, weight, post, scale = ctx.saved_tensors
        dx, dres, dw, dpost, _, dscale = block_norm_bwd(x, residual, weight, dy.contiguous(), dr.contiguous(), post_weight=post,
                                                        scale=scale)
        return dx, dres, dw, dpost, dscale


def train(dev="cuda", steps=8, seed=1):
    """Gradient descent on one ssm block that learns to repeat the token before; returns the losses."""
    g = torch.Generator().manual_seed(seed)
    w = {k: v.requires_grad_() if torch.is_tensor(v) else v for k, v in _weights(g, dev, "ssm").items()}
    params = [v for v in w.values() if torch.is_tensor(v)]
    stream = torch.randn(4, 65, DIM, generator=g).to(dev)
    target = stream.roll(1, 1)[:, 1:]
    opt = torch.optim.Adam(params, lr=2e-3)
    losses = []
    for _ in range(steps):
        x = stream.to(BF)
        u, z = (x @ w["inp"]).chunk(2, dim=-1)
        u = _Conv.apply(u, w["conv"], w["conv_bias"])
        low, Bm, Cm = (u @ w["proj"]).split([RANK, STATES, STATES], dim=-1)
        y = _Scan.apply(u, low @ w["dt"], w["A"], Bm.unsqueeze(2), Cm.unsqueeze(2), w["D"], z, w["dt_bias"])
        normed, _ = _BlockNorm.apply(y @ w["out"], stream, w["next_norm"], w["post"], w["scale"])
        loss = (normed[:, 1:].float() - target).pow(2).mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


if __name__ == "__main__":
    print(f"single tokens against one pass: relative difference {serve():.2e}")
    print("loss:", " ".join(f"{v:.4f}" for v in train()))
