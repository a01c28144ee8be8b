"""Cases that measure the token-mixer operators around the recurrence: the short causal
convolution, the selective state space scan, the gated norm of a mixer's output and the
residual update with the norms on both sides of a block.

``run`` computes an operator in elementary torch operations (``own`` false) or calls the
library's entry points (``own`` true) on what ``prepare`` made; ``exact`` computes the same
outputs from the definitions in 64 bits.

Sequences: a case with ``packed`` true has ``seqs`` sequences of random lengths (an empty one
and one of a single token among them where there are five or more) in ``tokens`` rows;
otherwise ``seqs`` sequences of ``tokens`` tokens each.
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one token for 8 sequences, q, k of 16 and v of 32 heads of 128: a small serving step,
        # bound by the latency of a call
        dict(name="conv_step_b8", op="conv", dir="step", dtype="bf16", seqs=8, tokens=1, packed=False,
             channels=8192, width=4, act="silu"),
        # prompts of 16 requests packed along the tokens, the same channels, states kept for decoding
        dict(name="conv_prompt_packed", op="conv", dir="fwd", dtype="bf16", seqs=16, tokens=32761, packed=True,
             channels=8192, width=4, act="silu"),
        # training: q, k, v of 32 heads of 128 over 2 x 8192 tokens
        dict(name="conv_train", op="conv", dir="bwd", dtype="bf16", seqs=2, tokens=8192, packed=False,
             channels=12288, width=4, act="silu"),
        # one token for 256 sequences of 4096 channels: serving, the states in and out of memory
        dict(name="scan_step_b256", op="scan", dir="step", dtype="bf16", seqs=256, tokens=1, packed=False,
             channels=4096, states=16, groups=1),
        # one short prompt in full precision: few channels, an odd length
        dict(name="scan_prompt_short_f32", op="scan", dir="fwd", dtype="f32", seqs=1, tokens=333, packed=False,
             channels=2048, states=16, groups=1),
        # prompts of full length for two sequences, 32 heads of 128
        dict(name="scan_prompt", op="scan", dir="fwd", dtype="bf16", seqs=2, tokens=8192, packed=False,
             channels=4096, states=16, groups=1),
        # seven requests packed, few channels: parallel only along the tokens
        dict(name="scan_long_packed", op="scan", dir="fwd", dtype="bf16", seqs=7, tokens=32771, packed=True,
             channels=2048, states=16, groups=1),
        # training
        dict(name="scan_train", op="scan", dir="bwd", dtype="bf16", seqs=2, tokens=4096, packed=False,
             channels=4096, states=16, groups=1),
        # the recurrence's output, 2 x 8192 tokens of 32 heads of 128, normed per head and gated
        dict(name="gated_norm_prompt", op="gated_norm", dir="fwd", dtype="bf16", rows=524288, channels=128,
             act="silu"),
        # its gradient, 4 x 4096 tokens of 16 heads
        dict(name="gated_norm_train", op="gated_norm", dir="bwd", dtype="bf16", rows=262144, channels=128,
             act="silu"),
        # the end of a block and the start of the next over 2 x 8192 tokens of 4096 channels,
        # residual stream in full precision
        dict(name="block_norm_prompt", op="block_norm", dir="fwd", dtype="bf16", rows=16384, channels=4096,
             act="sigmoid", res="f32", post=True, gate=True, scale=True),
        # training: its gradient
        dict(name="block_norm_train", op="block_norm", dir="bwd", dtype="bf16", rows=8192, channels=4096,
             act="sigmoid", res="f32", post=True, gate=True, scale=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "scan", "scan", "scan", "gated_norm", "block_norm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "conv":
        d = rng.choice(["step", "fwd", "bwd"])
        ch = _log(rng, 256, 12288)
        ch = (ch // 8 | 1) * 8 if rng.random() < 0.8 else ch | 1
        c = dict(op=op, dir=d, dtype=dtype, channels=ch, width=rng.choice([2, 3, 4, 4]), act=rng.choice(["silu", "none"]))
        if d == "step":
            return dict(c, seqs=_log(rng, 1, 512), tokens=1, packed=False)
        rows = int(_log(rng, 64, 32768) * min(1.0, 8192 / ch) / (2 if dtype == "f32" else 1)) | 1
        if rng.random() < 0.5:
            return dict(c, seqs=rng.randint(2, 33), tokens=rows, packed=True)
        n = rng.randint(1, 4)
        return dict(c, seqs=n, tokens=rows // n | 1, packed=False)
    if op == "scan":
        d = rng.choice(["step", "fwd", "fwd", "bwd"])
        g = rng.choice([1, 1, 2])
        ch = _log(rng, 256, 4000) // g
        ch = ((ch // 8 | 1) * 8 if rng.random() < 0.8 else ch | 1) * g
        n = rng.choice([8, 16, 16, 16, 32, 64])
        c = dict(op=op, dir=d, dtype=dtype, channels=ch, states=n, groups=g)
        if d == "step":
            return dict(c, seqs=_log(rng, 1, max(1, min(512, (1 << 24) // (ch * n)))), tokens=1, packed=False)
        most = (8192 if d == "bwd" else 16384) * 4096 * 16 / (ch * n)
        rows = int(math.exp(rng.uniform(math.log(50), math.log(min(most, 16384))))) | 1
        if rng.random() < 0.5:
            return dict(c, seqs=rng.randint(2, 9), tokens=rows, packed=True)
        k = rng.randint(1, 4)
        return dict(c, seqs=k, tokens=rows // k | 1, packed=False)
    d = rng.choice(["fwd", "bwd"])
    if op == "gated_norm":
        ch = rng.choice([64, 128, 128, 256, 512, rng.randint(65, 1500)])
        rows = _log(rng, 16, (1 << 25) // ch) | 1
        return dict(op=op, dir=d, dtype=dtype, rows=rows, channels=ch, act=rng.choice(["silu", "sigmoid"]))
    ch = _log(rng, 512, 8000)
    ch = (ch // 8 | 1) * 8 if rng.random() < 0.8 else ch | 1
    rows = _log(rng, 4, (1 << 24) // ch) | 1
    return dict(op=op, dir=d, dtype=dtype, rows=rows, channels=ch, act=rng.choice(["silu", "sigmoid"]),
                res=rng.choice(["f32", dtype]), post=rng.random() < 0.6, gate=rng.random() < 0.6, scale=rng.random() < 0.6)


def _lengths(case, seed):
    n, t = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [t] * n
    r = random.Random(seed * 7919 + 13)
    cuts = sorted(r.randint(0, t) for _ in range(n - 1))
    ends = cuts + [t]
    lens = [e - s for s, e in zip([0] + cuts, ends)]
    if n >= 5 and t > 2:  # an empty sequence and one of a single token
        i, j, k = r.sample(range(n), 3)
        lens[k] += lens[i] + lens[j]
        lens[i], lens[j] = 0, 0
        if lens[k] > 1:
            lens[k] -= 1
            lens[j] = 1
    return lens


def _shape(case, inner):
    if case["packed"]:
        return (1, case["tokens"], *inner)
    return (case["seqs"], case["tokens"], *inner)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    ch, op, d = case["channels"], case["op"], case["dir"]
    if op in ("conv", "scan"):
        rows = case["tokens"] * (1 if case["packed"] else case["seqs"])
        nseq = case["seqs"]
    if op == "conv":
        w = case["width"]
        par = 4 * ch * (w + 1)
        state = nseq * (w - 1) * ch * e
        act = 5 if case["act"] == "silu" else 0
        if d == "bwd":  # x, dy in, dx out; s0, dst in, ds0 out; weights and their gradients
            return dict(bytes=3 * rows * ch * e + 3 * state + 2 * par, flops=rows * ch * (6 * w + 2 * act + 4))
        return dict(bytes=2 * rows * ch * e + 2 * state + par, flops=rows * ch * (2 * w + act))
    if op == "scan":
        n, g = case["states"], case["groups"]
        par = 4 * ch * (n + 2)
        state = nseq * ch * n * 4
        bc = 2 * rows * g * n * e
        if d == "bwd":  # u, dt, z, dy in and du, ddt, dz out; B, C and their gradients; h0, dht in, dh0 out
            return dict(bytes=7 * rows * ch * e + 2 * bc + 3 * state + 2 * par, flops=rows * ch * (28 * n + 40))
        return dict(bytes=4 * rows * ch * e + bc + 2 * state + par, flops=rows * ch * (7 * n + 20))
    rows = case["rows"]
    if op == "gated_norm":
        if d == "bwd":  # o, z, dy in, do, dz out
            return dict(bytes=5 * rows * ch * e + 8 * ch, flops=rows * ch * 25)
        return dict(bytes=3 * rows * ch * e + 4 * ch, flops=rows * ch * 10)
    r = 4 if case["res"] == "f32" else 2
    par = 4 * ch * (1 + case["post"] + case["scale"])
    gate = case["gate"]
    if d == "bwd":  # x, z, dy and both residual tensors in; dx, dz and the residual's gradient out
        return dict(bytes=rows * ch * (e * (3 + 2 * gate) + 3 * r) + 2 * par, flops=rows * ch * 40)
    return dict(bytes=rows * ch * (e * (2 + gate) + 2 * r) + par, flops=rows * ch * 15)


# ---- inputs ----------------------------------------------------------------------------------

def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    ch = case["channels"]

    def normal(shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    def uniform(shape, lo, hi):
        return torch.rand(shape, generator=g, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = dict(case=dict(case))
    if case["op"] in ("conv", "scan"):
        lens = _lengths(case, seed)
        nseq = len(lens)
        bounds = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
        s["lens"] = lens
        s["bounds"] = torch.from_numpy(bounds).to(dev)
        s["cu"] = torch.from_numpy(bounds.astype(np.int32)).to(dev) if case["packed"] else None
        s["row_seq"] = torch.from_numpy(np.repeat(np.arange(nseq), lens)).to(dev)
    if case["op"] == "conv":
        w = case["width"]
        s["x"] = normal(_shape(case, (ch,)))
        s["weight"] = uniform((ch, w), -1.0, 1.0) * w ** -0.5
        s["bias"] = uniform((ch,), -1.0, 1.0) * w ** -0.5
        s["s0"] = normal((nseq, w - 1, ch))
        if case["dir"] == "bwd":
            s["dy"] = normal(s["x"].shape)
            s["dst"] = normal((nseq, w - 1, ch))
    elif case["op"] == "scan":
        n, grp = case["states"], case["groups"]
        # channels after the convolution's SiLU; step sizes about 1e-3 .. 1e-1 as models start with
        s["u"] = torch.nn.functional.silu(normal(_shape(case, (ch,)), dtype=torch.float32)).to(dt)
        s["dt"] = normal(_shape(case, (ch,)), 0.5)
        step = torch.exp(uniform((ch,), math.log(1e-3), math.log(1e-1)))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        s["A"] = -torch.arange(1, n + 1, device=dev, dtype=torch.float32) * torch.exp(normal((ch, n), 0.1, torch.float32))
        s["A"] = s["A"].contiguous()
        s["B"] = normal(_shape(case, (grp, n)))
        s["C"] = normal(_shape(case, (grp, n)))
        s["D"] = 1.0 + normal((ch,), 0.1, torch.float32)
        s["z"] = normal(_shape(case, (ch,)))
        s["h0"] = normal((nseq, ch, n), 0.3, torch.float32)
        if case["dir"] == "bwd":
            s["dy"] = normal(s["u"].shape)
            s["dht"] = normal((nseq, ch, n), 1.0, torch.float32)
    else:
        rows = case["rows"]
        s["x"] = normal((rows, ch))
        s["weight"] = 1.0 + normal((ch,), 0.1, torch.float32)
        if case["op"] == "gated_norm":
            s["z"] = normal((rows, ch))
        else:
            res = DTYPES[case["res"]]
            s["residual"] = normal((rows, ch), 2.0, res)
            s["post_weight"] = 1.0 + normal((ch,), 0.1, torch.float32) if case["post"] else None
            s["z"] = normal((rows, ch)) if case["gate"] else None
            s["scale"] = 0.5 + normal((ch,), 0.1, torch.float32) if case["scale"] else None
            if case["dir"] == "bwd":
                s["dres"] = normal((rows, ch), 1.0, res)
        if case["dir"] == "bwd":
            s["dy"] = normal((rows, ch))
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    f = _OWN if own else _PLAIN
    return f[c["op"], c["dir"]](s)


def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _gate(x, act):
    return x * _sigmoid(x) if act == "silu" else _sigmoid(x)


def _dgate(x, act):
    p = _sigmoid(x)
    return p * (1.0 + x * (1.0 - p)) if act == "silu" else p * (1.0 - p)


def _conv_rows(s):
    """The row of [x; s0] that each tap of each token reads, [rows, W], and the W - 1 rows of
    each sequence's final state."""
    x, w = s["x"], s["case"]["width"]
    rows = x.shape[0] * x.shape[1]
    seq, start = s["row_seq"], s["bounds"][:-1]
    back = torch.arange(w, device=x.device) - (w - 1)

    def row_of(pos, n):
        before = pos - start[n]
        return torch.where(before >= 0, pos, rows + n * (w - 1) + (w - 1) + before)

    taps = row_of(torch.arange(rows, device=x.device)[:, None] + back, seq[:, None].expand(rows, w))
    n = torch.arange(len(s["lens"]), device=x.device)[:, None].expand(-1, w - 1)
    return taps, row_of(s["bounds"][1:, None] + back[:-1] + 0, n)


def _conv_plain_fwd(s):
    x, s0 = s["x"], s["s0"]
    ch, w = x.shape[-1], s["weight"].shape[1]
    taps, last = _conv_rows(s)
    ext = torch.cat([x.reshape(-1, ch), s0.reshape(-1, ch)]).float()
    pre = (ext[taps] * s["weight"].t()).sum(1) + s["bias"]
    y = pre * _sigmoid(pre) if s["case"]["act"] == "silu" else pre
    return y.to(x.dtype).reshape(x.shape), ext[last].to(x.dtype).reshape(-1, w - 1, ch)


def _conv_plain_step(s):
    y, st = _conv_plain_fwd(s)
    s["s0"].copy_(st)
    return y, s["s0"]


def _conv_plain_bwd(s):
    x, s0 = s["x"], s["s0"]
    ch, w = x.shape[-1], s["weight"].shape[1]
    rows, nseq = x.shape[0] * x.shape[1], len(s["lens"])
    taps, last = _conv_rows(s)
    ext = torch.cat([x.reshape(-1, ch), s0.reshape(-1, ch)]).float()
    read = ext[taps]
    pre = (read * s["weight"].t()).sum(1) + s["bias"]
    g = s["dy"].reshape(-1, ch).float()
    if s["case"]["act"] == "silu":
        g = g * _dgate(pre, "silu")
    dw = (g[:, None] * read).sum(0).t().contiguous()
    db = g.sum(0)
    # what reads a row at position p (a token, or a row of the state before its sequence): the
    # tokens p .. p + W - 1 of the same sequence
    k = torch.arange(w, device=x.device)
    start, end = s["bounds"][:-1], s["bounds"][1:]
    sseq = torch.arange(nseq, device=x.device)[:, None].expand(-1, w - 1).reshape(-1)
    spos = (start[:, None] + k[:-1] - (w - 1)).reshape(-1)
    pos = torch.cat([torch.arange(rows, device=x.device), spos])[:, None] + k
    seq = torch.cat([s["row_seq"], sseq])[:, None]
    inside = (pos >= start[seq]) & (pos < end[seq])
    gz = torch.cat([g, g.new_zeros(1, ch)])
    dext = (gz[torch.where(inside, pos, rows)] * s["weight"].t().flip(0)).sum(1)
    dext[last.reshape(-1)] += s["dst"].reshape(-1, ch).float()  # these rows are distinct
    dx, ds0 = dext[:rows].to(x.dtype).reshape(x.shape), dext[rows:].to(x.dtype).reshape(s0.shape)
    return dx, dw, db, ds0


def _scan_parts(s):
    """Step sizes, decays and the states after every token, as rows [R, G, D / G(, N)]."""
    grp, n = s["case"]["groups"], s["case"]["states"]
    ch = s["case"]["channels"]
    r = s["u"].shape[0] * s["u"].shape[1]
    u = s["u"].reshape(r, grp, ch // grp).float()
    raw = s["dt"].reshape(r, grp, ch // grp).float() + s["dt_bias"].reshape(grp, -1)
    dt = torch.where(raw > 20.0, raw, torch.log1p(torch.exp(torch.clamp(raw, max=20.0))))
    A = s["A"].reshape(grp, -1, n)
    B = s["B"].reshape(r, grp, 1, n).float()
    C = s["C"].reshape(r, grp, 1, n).float()
    a = torch.exp(dt[..., None] * A)
    full = (s["bounds"][1:] > s["bounds"][:-1]).nonzero().reshape(-1)  # sequences that hold tokens
    first, last = s["bounds"][:-1][full], s["bounds"][1:][full] - 1
    h0 = s["h0"].reshape(-1, grp, ch // grp, n)
    h = (dt * u)[..., None] * B
    h[first] += a[first] * h0[full]
    m = a.clone()
    m[first] = 0.0
    _doubling(m, h, max(s["lens"]))
    return dict(u=u, raw=raw, dt=dt, A=A, B=B, C=C, a=a, h=h, h0=h0, full=full, first=first, last=last, r=r)


def _doubling(m, h, longest):
    """h[t] <- h[t] + m[t] h[t-1] for all t at once: spans of twice the length in each turn."""
    k = 1
    while k < longest:
        add = m[k:] * h[:-k]
        h[k:] += add
        torch.mul(m[k:], m[:-k], out=add)
        m[k:] = add
        k *= 2


def _scan_plain_fwd(s):
    p = _scan_parts(s)
    y = (p["h"] * p["C"]).sum(-1) + s["D"].reshape(p["A"].shape[:2]) * p["u"]
    y = y.reshape(s["u"].shape) * _gate(s["z"].float(), "silu")
    ht = s["h0"].clone()
    ht[p["full"]] = p["h"][p["last"]].reshape(-1, *ht.shape[1:])
    return y.to(s["u"].dtype), ht


def _scan_plain_step(s):
    y, ht = _scan_plain_fwd(s)
    s["h0"].copy_(ht)
    return y, s["h0"]


def _scan_plain_bwd(s):
    p = _scan_parts(s)
    u, dt, A, B, C, a, h = (p[k] for k in ("u", "dt", "A", "B", "C", "a", "h"))
    D = s["D"].reshape(A.shape[:2])
    t = s["u"].dtype
    shape = s["u"].shape
    y = (h * C).sum(-1) + D * u
    z, dout = s["z"].reshape(u.shape).float(), s["dy"].reshape(u.shape).float()
    dz = dout * y * _dgate(z, "silu")
    dy = dout * _gate(z, "silu")
    # adjoint of the states, backwards: l[t] = C[t] dy[t] + a[t+1] l[t+1]
    dht = s["dht"].reshape(p["h0"].shape)
    l = dy[..., None] * C
    l[p["last"]] += dht[p["full"]]
    m = torch.cat([a[1:], torch.zeros_like(a[:1])])
    m[p["last"]] = 0.0
    m, l = m.flip(0), l.flip(0)
    _doubling(m, l, max(s["lens"]))
    l = l.flip(0)
    del m
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[p["first"]] = p["h0"][p["full"]]
    q = l * a * before
    del before
    dA = (dt[..., None] * q).sum(0).reshape(s["A"].shape)
    lb = (l * B).sum(-1)
    ddt = ((A * q).sum(-1) + u * lb) * _sigmoid(p["raw"])
    du = D * dy + dt * lb
    dB = (l * (dt * u)[..., None]).sum(2)
    dC = (h * dy[..., None]).sum(2)
    dh0 = s["dht"].clone()
    dh0[p["full"]] = (a[p["first"]] * l[p["first"]]).reshape(-1, *dh0.shape[1:])
    return dict(du=du.to(t).reshape(shape), ddt=ddt.to(t).reshape(shape), dA=dA, dB=dB.to(t).reshape(s["B"].shape),
                dC=dC.to(t).reshape(s["C"].shape), dD=(dy * u).sum(0).reshape(-1), dz=dz.to(t).reshape(shape),
                ddt_bias=ddt.sum(0).reshape(-1), dh0=dh0)


EPS = 1e-6


def _gated_norm_plain_fwd(s):
    x = s["x"].float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return (x * inv * s["weight"] * _gate(s["z"].float(), s["case"]["act"])).to(s["x"].dtype)


def _norm_back(g, x, inv):
    """Gradient of x inv, inv = (mean x^2 + eps)^(-1/2), for the gradient g of the result."""
    xh = x * inv
    return inv * (g - xh * (g * xh).mean(-1, keepdim=True))


def _gated_norm_plain_bwd(s):
    x, z, dy = s["x"].float(), s["z"].float(), s["dy"].float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    gate = _gate(z, s["case"]["act"])
    dx = _norm_back(dy * gate * s["weight"], x, inv)
    dz = dy * x * inv * s["weight"] * _dgate(z, s["case"]["act"])
    return dx.to(s["x"].dtype), dz.to(s["z"].dtype), (dy * gate * x * inv).sum(0)


def _block_parts(s):
    x = s["x"].float()
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) if s["post_weight"] is not None else None
    xn = x if inv is None else x * inv
    b = xn if inv is None else xn * s["post_weight"]
    gate = None if s["z"] is None else _gate(s["z"].float(), s["case"]["act"])
    out = b if gate is None else b * gate
    r = s["residual"].float() + (out if s["scale"] is None else out * s["scale"])
    return x, inv, xn, b, gate, out, r, torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)


def _block_norm_plain_fwd(s):
    *_, r, rinv = _block_parts(s)
    return (r * rinv * s["weight"]).to(s["x"].dtype), r.to(s["residual"].dtype)


def _block_norm_plain_bwd(s):
    x, inv, xn, b, gate, out, r, rinv = _block_parts(s)
    dy = s["dy"].float()
    got = dict(dweight=(dy * r * rinv).sum(0))
    dr = s["dres"].float() + _norm_back(dy * s["weight"], r, rinv)
    got["dresidual"] = dr.to(s["residual"].dtype)
    dout = dr
    if s["scale"] is not None:
        got["dscale"] = (dr * out).sum(0)
        dout = dr * s["scale"]
    db = dout
    if gate is not None:
        got["dz"] = (dout * b * _dgate(s["z"].float(), s["case"]["act"])).to(s["z"].dtype)
        db = dout * gate
    dx = db
    if inv is not None:
        got["dpost_weight"] = (db * xn).sum(0)
        dx = _norm_back(db * s["post_weight"], x, inv)
    got["dx"] = dx.to(s["x"].dtype)
    return got


_PLAIN = {
    ("conv", "fwd"): _conv_plain_fwd, ("conv", "step"): _conv_plain_step, ("conv", "bwd"): _conv_plain_bwd,
    ("scan", "fwd"): _scan_plain_fwd, ("scan", "step"): _scan_plain_step, ("scan", "bwd"): _scan_plain_bwd,
    ("gated_norm", "fwd"): _gated_norm_plain_fwd, ("gated_norm", "bwd"): _gated_norm_plain_bwd,
    ("block_norm", "fwd"): _block_norm_plain_fwd, ("block_norm", "bwd"): _block_norm_plain_bwd,
}


# ---- the library's operators -----------------------------------------------------------------

def _activation(s):
    return None if s["case"]["act"] == "none" else s["case"]["act"]


def _conv_own_fwd(s):
    from chunkwise_gated_linear_gb300 import causal_conv_fwd

    return causal_conv_fwd(s["x"], s["weight"], s["bias"], s0=s["s0"], activation=_activation(s),
                           cu_seqlens=s["cu"], output_final_state=True)


def _conv_own_step(s):
    from chunkwise_gated_linear_gb300 import causal_conv_step

    return causal_conv_step(s["x"], s["s0"], s["weight"], s["bias"], activation=_activation(s)), s["s0"]


def _conv_own_bwd(s):
    from chunkwise_gated_linear_gb300 import causal_conv_bwd

    return causal_conv_bwd(s["x"], s["weight"], s["bias"], s["dy"], s0=s["s0"], dst=s["dst"],
                           activation=_activation(s), cu_seqlens=s["cu"])


def _scan_own_fwd(s):
    from chunkwise_gated_linear_gb300 import selective_scan_fwd

    return selective_scan_fwd(s["u"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], dt_bias=s["dt_bias"],
                              dt_softplus=True, h0=s["h0"], cu_seqlens=s["cu"], output_final_state=True)


def _scan_own_step(s):
    from chunkwise_gated_linear_gb300 import selective_scan_step

    y = selective_scan_step(s["u"], s["dt"], s["A"], s["B"], s["C"], s["h0"], s["D"], s["z"], dt_bias=s["dt_bias"],
                            dt_softplus=True)
    return y, s["h0"]


def _scan_own_bwd(s):
    from chunkwise_gated_linear_gb300 import selective_scan_bwd

    du, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0 = selective_scan_bwd(
        s["u"], s["dt"], s["A"], s["B"], s["C"], s["dy"], s["D"], s["z"], dt_bias=s["dt_bias"], dt_softplus=True,
        h0=s["h0"], dht=s["dht"], cu_seqlens=s["cu"])
    return dict(du=du, ddt=ddt, dA=dA, dB=dB, dC=dC, dD=dD, dz=dz, ddt_bias=ddt_bias, dh0=dh0)


def _gated_norm_own_fwd(s):
    from chunkwise_gated_linear_gb300 import gated_norm_fwd

    return gated_norm_fwd(s["x"], s["z"], s["weight"], eps=EPS, activation=s["case"]["act"])


def _gated_norm_own_bwd(s):
    from chunkwise_gated_linear_gb300 import gated_norm_bwd

    return gated_norm_bwd(s["x"], s["z"], s["weight"], s["dy"], eps=EPS, activation=s["case"]["act"])


def _block_norm_own_fwd(s):
    from chunkwise_gated_linear_gb300 import block_norm_fwd

    return block_norm_fwd(s["x"], s["residual"], s["weight"], post_weight=s["post_weight"], z=s["z"], scale=s["scale"],
                          eps=EPS, activation=s["case"]["act"])


def _block_norm_own_bwd(s):
    from chunkwise_gated_linear_gb300 import block_norm_bwd

    dx, dres, dw, dpw, dz, dscale = block_norm_bwd(
        s["x"], s["residual"], s["weight"], s["dy"], s["dres"], post_weight=s["post_weight"], z=s["z"],
        scale=s["scale"], eps=EPS, activation=s["case"]["act"])
    got = dict(dx=dx, dresidual=dres, dweight=dw, dpost_weight=dpw, dz=dz, dscale=dscale)
    return {k: v for k, v in got.items() if v is not None}


_OWN = {
    ("conv", "fwd"): _conv_own_fwd, ("conv", "step"): _conv_own_step, ("conv", "bwd"): _conv_own_bwd,
    ("scan", "fwd"): _scan_own_fwd, ("scan", "step"): _scan_own_step, ("scan", "bwd"): _scan_own_bwd,
    ("gated_norm", "fwd"): _gated_norm_own_fwd, ("gated_norm", "bwd"): _gated_norm_own_bwd,
    ("block_norm", "fwd"): _block_norm_own_fwd, ("block_norm", "bwd"): _block_norm_own_bwd,
}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    return _EXACT[case["op"]](s, case)


def _act64(x, act):
    """The activation's value and derivative."""
    sg = torch.special.expit(x)
    if act == "silu":
        return x * sg, sg + x * sg * (1 - sg)
    if act == "sigmoid":
        return sg, sg * (1 - sg)
    return x, torch.ones_like(x)


def _conv_exact(s, case):
    """Sequence by sequence: the sequence with its W - 1 rows before it, and W shifted views."""
    w, ch = case["width"], case["channels"]
    x = s["x"].reshape(-1, ch)
    bwd = case["dir"] == "bwd"
    y, st = torch.empty_like(x), torch.empty_like(s["s0"])
    if bwd:
        dx, ds0 = torch.empty_like(x), torch.empty_like(s["s0"])
        dw, db = torch.zeros_like(s["weight"]), torch.zeros_like(s["bias"])
        dy = s["dy"].reshape(-1, ch)
    # sequences of one length go together; packed ones one by one
    at = 0
    same = not case["packed"]
    for n in range(1 if same else len(s["lens"])):
        ln = s["lens"][n]
        pick = slice(None) if same else slice(n, n + 1)
        k = len(s["lens"]) if same else 1
        rows = slice(at, at + k * ln)
        at += k * ln
        long = torch.cat([s["s0"][pick], x[rows].reshape(k, ln, ch)], 1)
        pre = s["bias"].expand(k, ln, ch).clone()
        for j in range(w):
            pre += long[:, j:j + ln] * s["weight"][:, j]
        out, der = _act64(pre, case["act"])
        y[rows] = out.reshape(-1, ch)
        st[pick] = long[:, ln:]
        if bwd:
            gp = dy[rows].reshape(k, ln, ch) * der
            dl = torch.zeros_like(long)
            dl[:, ln:] += s["dst"][pick]
            for j in range(w):
                dl[:, j:j + ln] += gp * s["weight"][:, j]
                dw[:, j] += (gp * long[:, j:j + ln]).sum((0, 1))
            db += gp.sum((0, 1))
            dx[rows] = dl[:, w - 1:].reshape(-1, ch)
            ds0[pick] = dl[:, :w - 1]
    if bwd:
        return dx.reshape(s["x"].shape), dw, db, ds0
    return y.reshape(s["x"].shape), st


def _scan_exact(s, case):
    """Token by token over all sequences at once, shorter ones at rest once they have ended."""
    ch, n, grp = case["channels"], case["states"], case["groups"]
    lens, bwd = s["lens"], case["dir"] == "bwd"
    k, longest = len(lens), max(lens)
    dev = s["u"].device
    if bwd and longest * k * ch * n * 8 > 60e9:
        return None
    flat = {q: s[q].reshape(-1, *s[q].shape[2:]) for q in ("u", "dt", "B", "C", "z") + (("dy",) if bwd else ())}
    start = s["bounds"][:-1]
    ends = torch.tensor(lens, device=dev)
    total = flat["u"].shape[0]
    chan_group = torch.arange(ch, device=dev) // (ch // grp)
    raw = flat["dt"] + s["dt_bias"]
    step = torch.logaddexp(raw, torch.zeros_like(raw))
    y = torch.empty_like(flat["u"])
    h = s["h0"].clone()
    kept = torch.empty((longest + 1, k, ch, n), dtype=torch.float64, device=dev) if bwd else None
    if bwd:
        kept[0] = h
    for t in range(longest):
        rows = torch.clamp(start + t, max=total - 1)
        live = t < ends
        d, uu = step[rows], flat["u"][rows]
        new = torch.exp(d[..., None] * s["A"]) * h + (d * uu)[..., None] * flat["B"][rows][:, chan_group]
        h = torch.where(live[:, None, None], new, h)
        if bwd:
            kept[t + 1] = h
        out = (h * flat["C"][rows][:, chan_group]).sum(-1) + s["D"] * uu
        y[rows[live]] = out[live]
    gate, dgate = _act64(flat["z"], "silu")
    if not bwd:
        return (y * gate).reshape(s["u"].shape), h
    dout = flat["dy"]
    dz = dout * y * dgate
    dy = dout * gate
    lam = s["dht"].clone()  # the adjoint of the state after the last token
    du, draw = torch.empty_like(y), torch.empty_like(y)
    dA, dD, dbias = torch.zeros_like(s["A"]), torch.zeros_like(s["D"]), torch.zeros_like(s["D"])
    dB, dC = torch.zeros_like(flat["B"]), torch.zeros_like(flat["C"])
    for t in range(longest - 1, -1, -1):
        live = (t < ends).nonzero().reshape(-1)
        rows = start[live] + t
        d, uu, g = step[rows], flat["u"][rows], dy[rows]
        Bt, Ct = flat["B"][rows][:, chan_group], flat["C"][rows][:, chan_group]
        a = torch.exp(d[..., None] * s["A"])
        lt = lam[live] + g[..., None] * Ct
        prev = kept[t][live]
        da = lt * prev * a  # with respect to the exponent d A
        dA += (da * d[..., None]).sum(0)
        into = (lt * Bt).sum(-1)
        dd = (da * s["A"]).sum(-1) + into * uu
        dr = dd * torch.special.expit(raw[rows])
        draw[rows] = dr
        du[rows] = into * d + g * s["D"]
        dD += (g * uu).sum(0)
        dbias += dr.sum(0)
        m = len(live)
        dB[rows] = (lt * (d * uu)[..., None]).reshape(m, grp, -1, n).sum(2)
        dC[rows] = (kept[t + 1][live] * g[..., None]).reshape(m, grp, -1, n).sum(2)
        lam[live] = lt * a
    shape = s["u"].shape
    return dict(du=du.reshape(shape), ddt=draw.reshape(shape), dA=dA, dB=dB.reshape(s["B"].shape),
                dC=dC.reshape(s["C"].shape), dD=dD, dz=dz.reshape(shape), ddt_bias=dbias, dh0=lam)


def _rms64(x, g=None):
    """x / rms(x), and the gradient with respect to x for the gradient g of that."""
    rms = torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
    if g is None:
        return x / rms
    return x / rms, g / rms - x * (g * x).mean(-1, keepdim=True) / rms ** 3


def _gated_norm_exact(s, case):
    val, der = _act64(s["z"], case["act"])
    if case["dir"] == "fwd":
        return _rms64(s["x"]) * s["weight"] * val
    xn, dx = _rms64(s["x"], s["dy"] * val * s["weight"])
    return dx, s["dy"] * xn * s["weight"] * der, (s["dy"] * val * xn).sum(0)


def _block_norm_exact(s, case):
    one = torch.ones((), dtype=torch.float64, device=s["x"].device)
    pw = one if s["post_weight"] is None else s["post_weight"]
    sc = one if s["scale"] is None else s["scale"]
    val, der = (one, None) if s["z"] is None else _act64(s["z"], case["act"])
    xn = s["x"] if s["post_weight"] is None else _rms64(s["x"])
    r = s["residual"] + sc * val * pw * xn
    if case["dir"] == "fwd":
        return _rms64(r) * s["weight"], r
    rn, back = _rms64(r, s["dy"] * s["weight"])
    dr = s["dres"] + back
    got = dict(dweight=(s["dy"] * rn).sum(0), dresidual=dr)
    if s["scale"] is not None:
        got["dscale"] = (dr * val * pw * xn).sum(0)
    if s["z"] is not None:
        got["dz"] = dr * sc * pw * xn * der
    into = dr * sc * val
    if s["post_weight"] is not None:
        got["dpost_weight"] = (into * xn).sum(0)
        got["dx"] = _rms64(s["x"], into * pw)[1]
    else:
        got["dx"] = into
    return got


_EXACT = {"conv": _conv_exact, "scan": _scan_exact, "gated_norm": _gated_norm_exact, "block_norm": _block_norm_exact}
