"""Plain 64-bit definitions of the token-mixer operators on CPU tensors, written with torch
operations that autograd can differentiate, and helpers for their tests."""

from __future__ import annotations

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def bounds(lens):
    return [0, *np.cumsum(lens).tolist()]


def cu_of(lens, device="cpu"):
    return torch.tensor(bounds(lens), dtype=torch.int32, device=device)


def act(x, name):
    if name is None:
        return x
    return x * torch.sigmoid(x) if name == "silu" else torch.sigmoid(x)


def conv(x, w, b, s0, lens, activation):
    """x [rows, D], s0 [N, W - 1, D] or None -> y [rows, D], st [N, W - 1, D]."""
    W, D = w.shape[1], x.shape[1]
    ys, sts, at = [], [], 0
    for n, ln in enumerate(lens):
        before = x.new_zeros(W - 1, D) if s0 is None else s0[n]
        ext = torch.cat([before, x[at:at + ln]])
        at += ln
        y = sum(w[:, j] * ext[j:j + ln] for j in range(W))
        ys.append(act(y if b is None else y + b, activation))
        sts.append(ext[ln:])
    return torch.cat(ys), torch.stack(sts)


def scan(u, dt, A, B, C, D, z, bias, softplus, h0, lens):
    """u, dt, z [rows, ch], B, C [rows, G, N], h0 [N, ch, N] -> y [rows, ch], ht."""
    ch, G = A.shape[0], B.shape[1]
    group = torch.arange(ch) // (ch // G)
    s = dt if bias is None else dt + bias
    delta = torch.nn.functional.softplus(s, threshold=50.0) if softplus else s
    ys, hts, at = [], [], 0
    for n, ln in enumerate(lens):
        h = torch.zeros_like(A) if h0 is None else h0[n]
        for t in range(at, at + ln):
            h = torch.exp(delta[t][:, None] * A) * h + (delta[t] * u[t])[:, None] * B[t][group]
            y = (h * C[t][group]).sum(1)
            ys.append(y if D is None else y + D * u[t])
        at += ln
        hts.append(h)
    y = torch.stack(ys) if ys else u.new_zeros(u.shape)
    return (y if z is None else y * act(z, "silu")), torch.stack(hts)


def rms(x, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def gated_norm(x, z, w, eps, activation):
    return rms(x, eps) * w * act(z, activation)


def block_norm(x, r, w, pw, z, scale, eps, activation):
    o = x if pw is None else rms(x, eps) * pw
    if z is not None:
        o = o * act(z, activation)
    if scale is not None:
        o = o * scale
    r = r + o
    return rms(r, eps) * w, r


def leaves(tensors):
    """64-bit CPU copies that require gradients, None kept."""
    return {k: None if t is None else t.detach().double().cpu().requires_grad_() for k, t in tensors.items()}


def grads(outs, cotangents, inputs):
    """Gradients of sum(cotangent * out) for the inputs that are not None; zeros where an input
    has no part in it."""
    loss = sum((o * c.double().cpu().reshape(o.shape)).sum() for o, c in zip(outs, cotangents) if c is not None)
    names = [k for k, v in inputs.items() if v is not None]
    got = torch.autograd.grad(loss, [inputs[k] for k in names], allow_unused=True)
    return {k: torch.zeros_like(inputs[k]) if g is None else g for k, g in zip(names, got)}


def rel(x, ref):
    x, ref = x.detach().double().cpu().reshape(ref.shape), ref.detach()
    assert bool(torch.isfinite(x).all()), "not finite"
    num, den = float((x - ref).norm()), float(ref.norm())
    return num / den if den else num


def check(what, x, ref, dtype, work):
    """The result's own rounding (half a step of its type), plus `work`: the relative error that
    the 32-bit computation may add, derived where it is given."""
    tiny = torch.finfo(dtype).tiny  # values below the type's range come out as zeros
    ref = torch.where(ref.detach().abs() < tiny, 0.0, ref.detach())
    e, tol = rel(x, ref), HALF[dtype] + work
    print(f"{what}: {e:.2e} (tol {tol:.2e})")
    assert x.dtype == dtype, (what, x.dtype)
    assert e <= tol, (what, e, tol)
