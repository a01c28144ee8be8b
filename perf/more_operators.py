"""Cases that measure the operators of an attention layer beside the recurrent ones: the norms of
queries and keys with the position rotation (and, for single tokens, with the write into the
cache), writing a paged key-value cache and reading it back, and the attention of the next
tokens over that cache.

``run`` computes an operator in elementary torch operations (``own`` false) or calls the
library's entry points (``own`` true) on what ``prepare`` made; ``exact`` computes the same
outputs from the definitions in 64 bits.

A cache holds pages [pages, kv_heads, page, dim]; ``table`` [seqs, pages per sequence] names the
pages of each sequence, ``lens`` [seqs] its length with the new tokens in it. A case with ``kv``
"e4m3" holds 8-bit values and one power of two for each (token, head); otherwise the cache has the
type of the data. Of n new tokens of a sequence, token i stands at position lens - n + i; one at a
negative position is not there (sequences at rest in a batch).
"""

import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6
THETA = 1e6


# ---- cases -----------------------------------------------------------------------------------

def listed():
    return [
        # one token for 8 sequences, 32 query and 8 key heads of 128, into an 8-bit cache: a small
        # serving step, bound by the latency of a call
        dict(name="norm_step_b8", op="norm", dir="step", dtype="bf16", seqs=8, tokens=1, packed=False, q_heads=32,
             kv_heads=8, dim=128, rot=128, layout="halves", norm=True, start=4000, kv="e4m3", page=64),
        # prompts of 2 x 8192 tokens, the same heads
        dict(name="norm_prompt", op="norm", dir="fwd", dtype="bf16", seqs=2, tokens=8192, packed=False, q_heads=32,
             kv_heads=8, dim=128, rot=128, layout="halves", norm=True, start=0),
        # training on 9 packed sequences, 16 query and 2 key heads of 256, a quarter of them rotated
        dict(name="norm_train", op="norm", dir="bwd", dtype="bf16", seqs=9, tokens=8191, packed=True, q_heads=16,
             kv_heads=2, dim=256, rot=64, layout="halves", norm=True, start=0),
        # prompts of 16 requests packed along the tokens, quantised into the cache
        dict(name="cache_write_prompt", op="cache", dir="write", dtype="bf16", seqs=16, tokens=32761, packed=True,
             kv_heads=8, dim=128, page=64, kv="e4m3", start=0),
        # four sequences of 8192 tokens read back (a prefix that a later prompt goes over again)
        dict(name="cache_read_prefix", op="cache", dir="read", dtype="bf16", seqs=4, tokens=8192, packed=False,
             kv_heads=8, dim=128, page=64, kv="e4m3", start=0),
        # the next token of 8 short conversations: bound by latency
        dict(name="attn_step_b8", op="attn", dir="step", dtype="bf16", seqs=8, tokens=700, new=1, q_heads=32, kv_heads=8,
             dim=128, page=64, kv="data", ragged=True, lse=False),
        # one sequence of full length: parallel only along the cache
        dict(name="attn_long_b1", op="attn", dir="step", dtype="bf16", seqs=1, tokens=131071, new=1, q_heads=32, kv_heads=8,
             dim=128, page=64, kv="data", ragged=False, lse=False),
        # a serving batch of very different lengths over an 8-bit cache
        dict(name="attn_ragged_b64", op="attn", dir="step", dtype="bf16", seqs=64, tokens=16384, new=1, q_heads=32, kv_heads=8,
             dim=128, page=64, kv="e4m3", ragged=True, lse=False),
        # wide heads, eight queries to a key head
        dict(name="attn_wide_heads", op="attn", dir="step", dtype="bf16", seqs=32, tokens=8192, new=1, q_heads=16, kv_heads=2,
             dim=256, page=128, kv="data", ragged=True, lse=False),
        # four drafted tokens per sequence at once, small pages, the sums' logarithms for a later join
        dict(name="attn_drafts", op="attn", dir="step", dtype="bf16", seqs=16, tokens=8192, new=4, q_heads=32, kv_heads=4,
             dim=128, page=16, kv="e4m3", ragged=True, lse=True),
        # many short sequences, small heads
        dict(name="attn_many_short", op="attn", dir="step", dtype="bf16", seqs=256, tokens=900, new=1, q_heads=16, kv_heads=8,
             dim=64, page=32, kv="data", ragged=True, lse=False),
        # full precision
        dict(name="attn_f32", op="attn", dir="step", dtype="f32", seqs=3, tokens=4095, new=1, q_heads=16, kv_heads=4,
             dim=128, page=32, kv="data", ragged=False, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "cache", "cache", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16])
    group = rng.choice([1, 2, 3, 4, 4, 5, 8, 8, 16])
    dim = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256])
    page = rng.choice([16, 16, 24, 32, 64, 64, 128])
    kv = rng.choice(["e4m3", "data"])
    c = dict(op=op, dtype=dtype, kv_heads=kv_heads, dim=dim)
    if op == "norm":
        d = rng.choice(["fwd", "bwd", "step"])
        rot = rng.choice([dim, dim, dim // 2, 32, 0])
        c = dict(c, dir=d, q_heads=kv_heads * group, rot=rot, layout=rng.choice(["halves", "halves", "pairs"]),
                 norm=rot == 0 or rng.random() < 0.8)
        if d == "step":
            return dict(c, seqs=_log(rng, 1, 256), tokens=rng.choice([1, 1, 1, 2, 5]), packed=False, start=_log(rng, 16, 100), kv=kv, page=page)
        most = (1 << 25) / (kv_heads * (group + 1) * dim)
        rows = max(8, min(_log(rng, 16, 32768), int(most))) | 1
        start = rng.choice([0, 0, _log(rng, 16, 1000000)])
        if rng.random() < 0.5:
            return dict(c, seqs=rng.randint(2, 33), tokens=rows, packed=True, start=start)
        n = rng.randint(1, 4)
        return dict(c, seqs=n, tokens=rows // n | 1, packed=False, start=start)
    if op == "cache":
        most = (1 << 25) / (kv_heads * dim)
        rows = max(1, min(_log(rng, 1, 65536), int(most)))
        c = dict(c, dir=rng.choice(["write", "read"]), page=page, kv=kv, start=rng.choice([0, 0, 1, _log(rng, 16, 1000)]))
        if rng.random() < 0.5:
            return dict(c, seqs=rng.randint(2, 33), tokens=rows, packed=True)
        n = rng.randint(1, min(64, rows))
        return dict(c, seqs=n, tokens=rows // n, packed=False)
    size = 1 if kv == "e4m3" else BYTES[dtype]
    most = 5e8 / (size * kv_heads * dim)  # tokens of all sequences
    seqs, tokens, ragged = _log(rng, 1, 256), _log(rng, 1, 131072), rng.random() < 0.6
    tokens = max(1, min(tokens, int(most / seqs)))
    new = min(tokens, rng.choice([1, 1, 1, 1, 2, 3, 4, 8]), 64 // group)
    return dict(c, dir="step", seqs=seqs, tokens=tokens, new=new, q_heads=kv_heads * group, page=page, kv=kv, ragged=ragged,
                lse=rng.random() < 0.3)


def _lengths(case):
    """New tokens of each sequence (packed: of random lengths, an empty one and one of a single
    token among them where there are five or more)."""
    n, t = case["seqs"], case["tokens"]
    if not case["packed"]:
        return [t] * n
    r = random.Random(n * 7919 + t)
    cuts = sorted(r.randint(0, t) for _ in range(n - 1))
    lens = [e - s for s, e in zip([0] + cuts, cuts + [t])]
    if n >= 5 and t > 2:
        i, j, k = r.sample(range(n), 3)
        lens[k] += lens[i] + lens[j]
        lens[i], lens[j] = 0, 0
        if lens[k] > 1:
            lens[k] -= 1
            lens[j] = 1
    return lens


def _cached(case):
    """Length of each sequence in the cache, the new tokens among them."""
    if case["op"] != "attn":
        return [n + case["start"] for n in _lengths(case)]
    n, t = case["seqs"], case["tokens"]
    r = random.Random(n * 104729 + t)
    lens = [r.randint(max(1, t // 16), t) if case["ragged"] else t for _ in range(n)]
    if case["ragged"] and n >= 5:  # one at rest and one that begins
        i, j = r.sample(range(n), 2)
        lens[i], lens[j] = 0, case["new"]
    return lens


def work(case):
    e, d = BYTES[case["dtype"]], case["dim"]
    kv = case["kv_heads"]
    row = kv * (d + 1 if case.get("kv") == "e4m3" else d * e)  # of a cache, one of K and V
    if case["op"] == "attn":
        lens, new, hq = _cached(case), case["new"], case["q_heads"]
        seen = sum(max(0, n - new + t + 1) for n in lens for t in range(new))
        return dict(bytes=2 * sum(lens) * row + len(lens) * new * hq * (2 * d * e + 4 * case["lse"]), flops=4 * hq * d * seen)
    rows = sum(_lengths(case))
    if case["op"] == "cache":
        return dict(bytes=2 * rows * (kv * d * e + row), flops=2 * rows * kv * d * 2)
    heads = case["q_heads"] + kv
    each = rows * heads * d
    par = (4 * 2 * d if case["norm"] else 0) + 4 * case["rot"]
    if case["dir"] == "bwd":
        return dict(bytes=3 * each * e + 2 * par, flops=each * 12)
    if case["dir"] == "step":  # q in and out, k and v in, the cache's rows out
        return dict(bytes=rows * (2 * case["q_heads"] * d * e + 2 * kv * d * e + 2 * row) + par, flops=each * 7)
    return dict(bytes=2 * each * e + par, flops=each * 7)


# ---- inputs ----------------------------------------------------------------------------------

def _frequencies(rot):
    """Turns per position of each pair, in units of 2^-64 turns, as 64-bit integers."""
    f = [int(THETA ** (-2.0 * i / rot) / (2.0 * math.pi) * 2.0 ** 64) for i in range(rot // 2)]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in f], dtype=torch.int64)


def _to_e4m3(x):
    """Rows x [..., D] in 32 bits -> 8-bit values and the exponent byte of each row's power of two: the least
    one that leaves the row's largest entry at 448 or below."""
    top = x.abs().amax(-1)
    e = torch.clamp(((top.view(torch.int32) + 0x1FFFFF) >> 23) - 135, min=-126)
    unit = ((127 - e) << 23).view(torch.float32)
    return (x * unit[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _cache(case, normal, page_count, g, dev):
    """Pages with values in all of them (also where no token has been written)."""
    shape = (page_count, case["kv_heads"], case["page"], case["dim"])
    if case["kv"] != "e4m3":
        return dict(k=normal(shape), v=normal(shape))
    k, ks = _to_e4m3(normal(shape, 1.0, torch.float32))
    v, vs = _to_e4m3(normal(shape, 1.0, torch.float32))
    return dict(k=k, v=v, k_scale=ks.view(torch.float8_e8m0fnu), v_scale=vs.view(torch.float8_e8m0fnu))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    d, hk = case["dim"], case["kv_heads"]

    def normal(shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * std).to(dtype)

    s = dict(case=dict(case))
    if case["op"] == "norm" and case["dir"] != "step":
        cached = None
    else:
        cached, page = _cached(case), case["page"]
        need = [-(-n // page) for n in cached]
        s["cache"] = _cache(case, normal, max(1, sum(need)) + 1, g, dev)
        order = torch.randperm(max(1, sum(need)) + 1, generator=g, device=dev).to(torch.int32)
        # pages of a sequence, scattered over the cache; the rest of a row of the table is not read
        at = np.concatenate([[0], np.cumsum(need)])[:-1]
        take = at[:, None] + np.minimum(np.arange(max(1, max(need)))[None], np.maximum(np.array(need) - 1, 0)[:, None])
        s["table"] = order[torch.from_numpy(take).to(dev)].contiguous()
        s["lens"] = torch.tensor(cached, dtype=torch.int32, device=dev)
    if case["op"] == "attn":
        s["q"] = normal((case["seqs"], case["new"], case["q_heads"], d), 1.5)
        return s
    lens = _lengths(case)
    bounds = np.concatenate([[0], np.cumsum(lens)])
    shape = (1, case["tokens"]) if case["packed"] else (case["seqs"], case["tokens"])
    s["cu"] = torch.from_numpy(bounds.astype(np.int32)).to(dev) if case["packed"] else None
    inside = np.arange(sum(lens)) - np.repeat(bounds[:-1], lens)
    pos = inside + case["start"]
    s["pos"] = torch.from_numpy(pos).to(dev)                              # of each row, as the plain form reads it
    s["row_seq"] = torch.from_numpy(np.repeat(np.arange(len(lens)), lens)).to(dev)
    if case["op"] == "cache":
        if case["dir"] == "write":
            s["k"], s["v"] = normal((*shape, hk, d)), normal((*shape, hk, d))
        return s
    hq = case["q_heads"]
    qkv = normal((*shape, (hq + 2 * hk) * d), 1.0)                          # one projection's output, read in slices
    s["q"] = qkv[..., :hq * d].unflatten(-1, (hq, d))
    s["k"] = qkv[..., hq * d:(hq + hk) * d].unflatten(-1, (hk, d))
    s["v"] = qkv[..., (hq + hk) * d:].unflatten(-1, (hk, d))
    s["qw"] = 1.0 + normal((d,), 0.1, torch.float32) if case["norm"] else None
    s["kw"] = 1.0 + normal((d,), 0.1, torch.float32) if case["norm"] else None
    s["freq"] = _frequencies(case["rot"]).to(dev)
    s["positions"] = s["pos"].to(torch.int32).reshape(shape) if case["dir"] != "step" and case["start"] else None
    if case["dir"] == "bwd":
        s["dq"], s["dk"] = normal((*shape, hq, d)), normal((*shape, hk, d))
    return s


# ---- one pass --------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    f = _OWN if own else _PLAIN
    return f[c["op"], c["dir"]](s)


def _turn(x, s, back=False):
    """Rotates the pairs of the first channels of rows x [rows, heads, D], in 32 bits; the angles in 64."""
    c = s["case"]
    half = c["rot"] // 2
    turns = torch.remainder(s["pos"][:, None].double() * (s["freq"].double() * 2.0 ** -64), 1.0) * (2.0 * math.pi)
    cos, sin = torch.cos(turns).float()[:, None], torch.sin(turns).float()[:, None]
    if back:
        sin = -sin
    first, second = (slice(0, half), slice(half, 2 * half)) if c["layout"] == "halves" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    y = x.clone()
    y[..., first] = x[..., first] * cos - x[..., second] * sin
    y[..., second] = x[..., second] * cos + x[..., first] * sin
    return y


def _rows(t):
    return t.reshape(-1, *t.shape[2:])


def _norm_plain(x, w, s):
    x = _rows(x).float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _turn(x, s)


def _norm_plain_fwd(s):
    return tuple(_norm_plain(s[n], s[n + "w"], s).to(s[n].dtype).reshape(s[n].shape) for n in "qk")


def _norm_plain_back(x, w, dy, s):
    t, shape = x.dtype, x.shape
    x, g = _rows(x).float(), _turn(_rows(dy).float(), s, back=True)
    if w is None:
        return g.to(t).reshape(shape), None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    gw = g * w
    dx = r * (gw - x * (r * r * (gw * x).mean(-1, keepdim=True)))
    return dx.to(t).reshape(shape), (g * x * r).sum((0, 1))


def _norm_plain_bwd(s):
    dq, dqw = _norm_plain_back(s["q"], s["qw"], s["dq"], s)
    dk, dkw = _norm_plain_back(s["k"], s["kw"], s["dk"], s)
    return dq, dk, dqw, dkw


def _put(s, name, rows):
    """Rows [rows, heads, D] in 32 bits into the cache, each at its sequence's position."""
    cache, page = s["cache"], s["case"]["page"]
    pages = s["table"][s["row_seq"], s["pos"] // page].long()
    slot = s["pos"] % page
    if s["case"]["kv"] != "e4m3":
        cache[name][pages, :, slot] = rows.to(cache[name].dtype)
        return
    val, e = _to_e4m3(rows)
    cache[name].view(torch.uint8)[pages, :, slot] = val.view(torch.uint8)
    cache[name + "_scale"].view(torch.uint8)[pages, :, slot] = e


def _norm_plain_step(s):
    _put(s, "k", _norm_plain(s["k"], s["kw"], s))
    _put(s, "v", _rows(s["v"]).float())
    return _norm_plain(s["q"], s["qw"], s).to(s["q"].dtype).reshape(s["q"].shape), s["cache"]


def _cache_plain_write(s):
    _put(s, "k", _rows(s["k"]).float())
    _put(s, "v", _rows(s["v"]).float())
    return s["cache"]


def _get(s, name, pages):
    """Pages of the cache in 32 bits."""
    cache = s["cache"]
    if s["case"]["kv"] != "e4m3":
        return cache[name][pages].float()
    scale = cache[name + "_scale"].view(torch.uint8)[pages].int() << 23
    return cache[name].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * scale.view(torch.float32)[..., None]


def _cache_plain_read(s):
    c = s["case"]
    pages = s["table"][s["row_seq"], s["pos"] // c["page"]].long()
    slot = s["pos"] % c["page"]
    got = []
    for name in "kv":
        if c["kv"] == "e4m3":
            val = s["cache"][name].view(torch.uint8)[pages, :, slot].view(torch.float8_e4m3fn).float()
            scale = s["cache"][name + "_scale"].view(torch.uint8)[pages, :, slot].int() << 23
            x = (val * scale.view(torch.float32)[..., None]).to(DTYPES[c["dtype"]])
        else:
            x = s["cache"][name][pages, :, slot]
        got.append(x.reshape(1 if c["packed"] else c["seqs"], -1, c["kv_heads"], c["dim"]))
    return got


def _attn_plain(s):
    c = s["case"]
    hk, d, new, n = c["kv_heads"], c["dim"], c["new"], c["seqs"]
    grp = c["q_heads"] // hk
    pages = s["table"].long()
    q = s["q"].float().reshape(n, new, hk, grp, d).permute(0, 2, 1, 3, 4).reshape(n, 1, hk, new * grp, d)
    score = torch.matmul(q * d ** -0.5, _get(s, "k", pages).transpose(-1, -2))  # [seqs, pages, heads, queries, page]
    at = torch.arange(pages.shape[1] * c["page"], device=q.device).reshape(1, -1, 1, 1, c["page"])
    token = torch.arange(new * grp, device=q.device) // grp
    seen = (s["lens"].long()[:, None] - new + 1 + token).reshape(n, 1, 1, -1, 1)
    score = torch.where(at < seen, score, -math.inf)
    top = torch.clamp(score.amax((1, 4), keepdim=True), min=-1e30)
    p = torch.exp(score - top)
    total = p.sum((1, 4))
    o = torch.matmul(p, _get(s, "v", pages)).sum(1) / torch.clamp(total, min=1e-30)[..., None]
    back = lambda x: x.reshape(n, hk, new, grp, -1).permute(0, 2, 1, 3, 4).reshape(n, new, hk * grp, -1)  # noqa: E731
    o = back(o).to(s["q"].dtype)
    return (o, back((torch.log(total) + top[:, 0, :, :, 0])[..., None])[..., 0]) if c["lse"] else o


_PLAIN = {
    ("norm", "fwd"): _norm_plain_fwd, ("norm", "bwd"): _norm_plain_bwd, ("norm", "step"): _norm_plain_step,
    ("cache", "write"): _cache_plain_write, ("cache", "read"): _cache_plain_read, ("attn", "step"): _attn_plain,
}


# ---- the library's calls ---------------------------------------------------------------------

def _kv(s):
    from chunkwise_gated_linear_gb300 import KVCache

    c = s["cache"]
    return KVCache(c["k"], c["v"], c.get("k_scale"), c.get("v_scale"))


def _norm_own_fwd(s):
    from chunkwise_gated_linear_gb300 import qk_norm_fwd

    return qk_norm_fwd(s["q"], s["k"], s["qw"], s["kw"], s["freq"], positions=s["positions"], cu_seqlens=s["cu"], eps=EPS,
                       interleaved=s["case"]["layout"] == "pairs")


def _norm_own_bwd(s):
    from chunkwise_gated_linear_gb300 import qk_norm_bwd

    return qk_norm_bwd(s["q"], s["k"], s["qw"], s["kw"], s["freq"], s["dq"], s["dk"], positions=s["positions"], cu_seqlens=s["cu"],
                       eps=EPS, interleaved=s["case"]["layout"] == "pairs")


def _norm_own_step(s):
    from chunkwise_gated_linear_gb300 import qk_norm_step

    q = qk_norm_step(s["q"], s["k"], s["v"], _kv(s), s["table"], s["lens"], s["qw"], s["kw"], s["freq"], eps=EPS,
                     interleaved=s["case"]["layout"] == "pairs")
    return q, s["cache"]


def _cache_own_write(s):
    from chunkwise_gated_linear_gb300 import kv_cache_write

    kv_cache_write(s["k"], s["v"], _kv(s), s["table"], s["lens"], cu_seqlens=s["cu"])
    return s["cache"]


def _cache_own_read(s):
    from chunkwise_gated_linear_gb300 import kv_cache_read

    return kv_cache_read(_kv(s), s["table"], s["lens"], s["case"]["tokens"], cu_seqlens=s["cu"], dtype=DTYPES[s["case"]["dtype"]])


def _attn_own(s):
    from chunkwise_gated_linear_gb300 import paged_attn_step

    return paged_attn_step(s["q"], _kv(s), s["table"], s["lens"], want_lse=s["case"]["lse"])


_OWN = {
    ("norm", "fwd"): _norm_own_fwd, ("norm", "bwd"): _norm_own_bwd, ("norm", "step"): _norm_own_step,
    ("cache", "write"): _cache_own_write, ("cache", "read"): _cache_own_read, ("attn", "step"): _attn_own,
}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed), case)


def _places(s, case, lens):
    """(sequence, first row, rows, pages, slots) of the new tokens of each sequence."""
    at, out = 0, []
    for i, n in enumerate(lens):
        pos = torch.arange(n, device=s["lens"].device) + case["start"]
        out.append((i, at, n, s["table"][i].long()[pos // case["page"]], pos % case["page"]))
        at += n
    return out


def _stored(s, case, name, rows):
    """The cache's contents in 64 bits after rows [rows, heads, D] have been written (not rounded to 8 bits)."""
    store = s["cache"][name].double()
    scale = s["cache"][name + "_scale"].double() if case["kv"] == "e4m3" else None
    for _, at, n, pages, slots in _places(s, case, _lengths(case)):
        if n == 0:
            continue
        x = rows[at:at + n]
        if scale is not None:
            m, e = torch.frexp(x.abs().amax(-1))
            e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
            unit = torch.ldexp(torch.ones_like(m), e)
            scale[pages, :, slots] = unit
            x = x / unit[..., None]
        store[pages, :, slots] = x
    return store, scale


def _whole_cache(s, case, k, v):
    (k, ks), (v, vs) = _stored(s, case, "k", k), _stored(s, case, "v", v)
    return dict(k=k, v=v) if ks is None else dict(k=k, v=v, k_scale=ks, v_scale=vs)


def _norm64(x, w, pos, case):
    """Rows through the norm, and the pairs as complex numbers times e^(i angle)."""
    if w is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS) * w
    half = case["rot"] // 2
    if half == 0:
        return x
    per = THETA ** (-torch.arange(half, device=x.device, dtype=torch.float64) * 2.0 / case["rot"])
    angle = pos.double()[:, None] * per
    z = torch.polar(torch.ones_like(angle), angle)[:, None]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if case["layout"] == "halves":
        y = torch.complex(turned[..., :half], turned[..., half:]) * z
        return torch.cat([y.real, y.imag, rest], -1)
    y = torch.complex(turned[..., 0::2], turned[..., 1::2]) * z
    return torch.cat([torch.stack([y.real, y.imag], -1).flatten(-2), rest], -1)


def _norm_exact(s, case):
    pos = torch.cat([torch.arange(n, device=s["q"].device) for n in _lengths(case)]) + case["start"]
    x = {n: s[n].double().flatten(0, 1) for n in "qk"}
    w = {n: None if s[n + "w"] is None else s[n + "w"].double() for n in "qk"}
    if case["dir"] != "bwd":
        y = {n: _norm64(x[n], w[n], pos, case) for n in "qk"}
        if case["dir"] == "fwd":
            return tuple(y[n].reshape(s[n].shape) for n in "qk")
        return y["q"].reshape(s["q"].shape), _whole_cache(s, case, y["k"], s["v"].double().flatten(0, 1))
    dx, dw = [], []
    for n in "qk":
        leaves = [t.requires_grad_() for t in (x[n], w[n]) if t is not None]
        got = torch.autograd.grad(_norm64(x[n], w[n], pos, case), leaves, s["d" + n].double().flatten(0, 1))
        dx.append(got[0].reshape(s[n].shape))
        dw.append(got[1] if len(got) > 1 else None)
    return *dx, *dw


def _loaded(s, case, name, pages, slots):
    x = s["cache"][name].view(torch.uint8 if case["kv"] == "e4m3" else s["cache"][name].dtype)[pages, :, slots]
    if case["kv"] != "e4m3":
        return x.double()
    scale = s["cache"][name + "_scale"].view(torch.uint8)[pages, :, slots].view(torch.float8_e8m0fnu).double()
    return x.view(torch.float8_e4m3fn).double() * scale[..., None]


def _cache_exact(s, case):
    if case["dir"] == "write":
        return _whole_cache(s, case, s["k"].double().flatten(0, 1), s["v"].double().flatten(0, 1))
    shape = (1 if case["packed"] else case["seqs"], -1, case["kv_heads"], case["dim"])
    places = _places(s, case, _lengths(case))
    return [torch.cat([_loaded(s, case, n, p, o) for _, _, _, p, o in places]).reshape(shape) for n in "kv"]


def _attn_exact(s, case):
    """Sequence by sequence and token by token over the keys that the token sees."""
    n, new, hk, d = case["seqs"], case["new"], case["kv_heads"], case["dim"]
    q = s["q"].double().reshape(n, new, hk, -1, d)
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=q.device)
    for i, ln in enumerate(_cached(case)):
        pos = torch.arange(ln, device=q.device)
        where = s["table"][i].long()[pos // case["page"]], pos % case["page"]
        k, v = (_loaded(s, case, x, *where).transpose(0, 1) for x in "kv")  # [heads, ln, D]
        for t in range(new):
            seen = ln - new + t + 1
            if seen <= 0:
                continue
            a = torch.matmul(q[i, t], k[:, :seen].transpose(1, 2)) / math.sqrt(d)
            lse[i, t] = torch.logsumexp(a, -1)
            o[i, t] = torch.matmul(torch.softmax(a, -1), v[:, :seen])
    o = o.reshape(s["q"].shape)
    return (o, lse.reshape(o.shape[:-1])) if case["lse"] else o


_EXACT = {"norm": _norm_exact, "cache": _cache_exact, "attn": _attn_exact}
