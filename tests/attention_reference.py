"""Plain 64-bit definitions of the attention-layer operators on CPU tensors, written with torch operations that
autograd can differentiate, and helpers for their tests."""

from __future__ import annotations

import math

import torch


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    """x [rows, heads, D], pos [rows] -> the same shape; inv_freq [R / 2] radians per position."""
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    half = len(inv_freq)
    if half == 0:
        return x
    angle = pos.double()[:, None] * inv_freq
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def inv_freq(R, theta=10000.0):
    return theta ** (-torch.arange(R // 2, dtype=torch.float64) * 2.0 / max(R, 1))


def e4m3_round(y):
    """To the nearest e4m3 number, ties to even; |y| <= 448, or not finite."""
    _, e = torch.frexp(y.abs().clamp(min=2.0 ** -6))  # steps are 2^(floor(log2 |y|) - 3), from 2^-9 on
    step = torch.ldexp(torch.ones_like(y), e - 4)
    return torch.where(torch.isfinite(y), torch.round(y / step) * step, y)


def row_unit(x):
    """The power of two of a row x [..., D]: the least 2^e, e >= -126, with max |x| <= 448 2^e."""
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)
    e = torch.where(top == 0, -126, torch.where(m <= 0.875, e - 9, e - 8)).clamp(min=-126)
    e = torch.where(torch.isinf(x).any(-1), torch.full_like(e, 120), e)
    return torch.ldexp(torch.ones_like(top), e)


def positions(cached, news):
    """Per sequence: the positions of its new tokens."""
    return [[n - k + i for i in range(k)] for n, k in zip(cached, news)]


def gather(cache, table, b, n, page):
    """Keys and values of sequence b, positions 0 .. n - 1, in 64 bits: [heads, n, D]."""
    pos = torch.arange(n)
    pages, slots = table[b].long()[pos // page], pos % page
    out = []
    for t, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        if s is None:
            x = t[pages, :, slots].double()
        else:  # torch indexes bytes, not 8-bit floating-point numbers
            x = t.view(torch.uint8)[pages, :, slots].view(t.dtype).double()
            x = x * s.view(torch.uint8)[pages, :, slots].view(s.dtype).double()[..., None]
        out.append(x.transpose(0, 1))
    return out


def attention(q, cache, table, lens, scale):
    """q [B, T, heads, D] -> o, lse in 64 bits; cache on the CPU."""
    B, T, Hq, D = q.shape
    page, heads = cache.k.shape[2], cache.k.shape[1]
    q = q.double()
    o = torch.zeros_like(q)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    for b in range(B):
        k, v = gather(cache, table, b, int(lens[b]), page)
        for t in range(T):
            n = int(lens[b]) - T + t + 1
            if n <= 0:
                continue
            x = torch.einsum("hgd,hnd->hgn", q[b, t].reshape(heads, -1, D), k[:, :n]) * scale
            lse[b, t] = torch.logsumexp(x, -1).reshape(-1)
            o[b, t] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v[:, :n]).reshape(Hq, D)
    return o, lse
