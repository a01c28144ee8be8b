"""Caches with scattered pages for the tests of the attention-layer operators."""

from __future__ import annotations

import torch

from chunkwise_gated_linear_gb300 import KVCache

BF, F32, E4M3, E8M0 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float8_e8m0fnu


def tables(g, lens, page, spare=2):
    """A block table over scattered pages and the number of pages; entries beyond a sequence name no page."""
    need = [-(-max(n, 0) // page) for n in lens]
    count = sum(need) + spare
    order = torch.randperm(count, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need)) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, count


def index(t):
    """A tensor that torch can index and assign in, whatever its type."""
    return t.view(torch.uint8) if t.dtype in (E4M3, E8M0) else t


def filled(g, lens, page, heads, D, dtype, std=1.0):
    """A cache on the CPU in which every position of every sequence holds a value, all others NaN, and its table."""
    table, count = tables(g, lens, page)
    shape = (count, heads, page, D)
    if dtype == E4M3:
        k, v = ((torch.randn(shape, generator=g) * 100).clamp(-448, 448).to(E4M3) for _ in "kv")
        ks, vs = (torch.randint(127 - 9, 127 - 5, shape[:3], generator=g).to(torch.uint8).view(E8M0) for _ in "kv")
        c = KVCache(k, v, ks, vs)
        nan = 0x7F
    else:
        c = KVCache(*((torch.randn(shape, generator=g) * std).to(dtype) for _ in "kv"))
        nan = float("nan")
    used = torch.zeros(shape[:3], dtype=torch.bool)
    for b, n in enumerate(lens):
        pos = torch.arange(max(n, 0))
        used[table[b].long()[pos // page], :, pos % page] = True
    for t in (c.k, c.v):
        index(t)[~used] = nan
    if dtype == E4M3:
        for t in (c.k_scale, c.v_scale):
            index(t)[~used] = 0xFF
    return c, table


def to_gpu(c):
    return KVCache(*(None if t is None else t.cuda() for t in c))
