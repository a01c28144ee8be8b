"""Writing the paged key-value cache and reading it back, on the GPU: every value bit for bit as the definition has it
(attention_reference), since a power of two makes every step but the one rounding exact."""

from __future__ import annotations

import pytest
import torch

import attention_reference as aref
import mixer_reference as ref
from attention_cases import BF, E4M3, E8M0, F32, index, tables
from chunkwise_gated_linear_gb300 import KVCache, attention, kda, kv_cache_read, kv_cache_write

pytestmark = pytest.mark.gpu
dev = "cuda"
LENS = [([1], [1], False), ([5, 130, 64, 64], [1, 1, 1, 1], False), ([3, 0, 1, 40], [3, 3, 3, 3], False),
        ([70, 9, 0, 33, 1, 2], [70, 4, 0, 1, 1, 0], True), ([700], [700], False), ([2500, 300], [2300, 300], True)]


def _data(g, cached, news, packed, heads, D, dtype):
    shape = (1, sum(news)) if packed else (len(news), news[0])
    # rows of very different sizes, a row of zeros among them
    size = torch.exp(torch.randn(*shape, heads, 1, generator=g) * 4)
    k, v = ((torch.randn(*shape, heads, D, generator=g) * size).to(dtype) for _ in "kv")
    if k.shape[1] > 2:
        k[0, 1] = 0
    cu = ref.cu_of(news, dev) if packed else None
    return k, v, cu


def _fill(cache, g):
    for t in cache:
        if t is not None:
            index(t).copy_(torch.randint(1, 100, t.shape, generator=g))


def _expect(x, kind):
    """(stored bytes or values, scale bytes) of rows x."""
    if kind != E4M3:
        return x, None
    unit = aref.row_unit(x.double())
    val = aref.e4m3_round(x.double() / unit[..., None])
    return val, unit


def _check_write_and_read(dtype, kind, page, cached, news, packed, D, heads):
    g = torch.Generator().manual_seed(D + page)
    k, v, cu = _data(g, cached, news, packed, heads, D, dtype)
    table, count = tables(g, cached, page)
    cache = KVCache.empty(count, heads, page, D, kind)
    _fill(cache, g)
    old = [None if t is None else t.cpu() for t in cache]
    lens = torch.tensor(cached, dtype=torch.int32, device=dev)
    kv_cache_write(k.to(dev), v.to(dev), cache, table.to(dev), lens, cu_seqlens=cu)
    pos = torch.tensor(sum(aref.positions(cached, news), []), dtype=torch.long)
    seq = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news))
    there = pos >= 0
    pages, slots = table[seq[there], pos[there] // page].long(), pos[there] % page
    back = kv_cache_read(cache, table.to(dev), lens, k.shape[1], cu_seqlens=cu, dtype=dtype)
    for i, x in enumerate((k, v)):
        want, unit = _expect(x.flatten(0, 1)[there], kind)
        now = index(cache[i].cpu())
        got = now[pages, :, slots]
        values = got.view(E4M3).double() if kind == E4M3 else got
        assert torch.equal(values, want)
        read = want if unit is None else want * unit[..., None]
        rows = back[i].cpu().flatten(0, 1)
        assert back[i].dtype == dtype and torch.equal(rows[there].double(), read.double())
        assert torch.equal(rows[~there], torch.zeros_like(rows[~there]))
        now[pages, :, slots] = index(old[i])[pages, :, slots]
        assert torch.equal(now, index(old[i])), "other places were written"
        if unit is not None:
            now = index(cache[2 + i].cpu())
            assert torch.equal(now[pages, :, slots].view(E8M0).double(), unit)
            now[pages, :, slots] = index(old[2 + i])[pages, :, slots]
            assert torch.equal(now, index(old[2 + i]))


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (BF, E4M3), (F32, F32), (F32, E4M3)])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
@pytest.mark.parametrize("cached,news,packed", LENS)
@pytest.mark.parametrize("D", [16, 80, 128, 256])
def test_write_and_read(dtype, kind, page, cached, news, packed, D):
    _check_write_and_read(dtype, kind, page, cached, news, packed, D, 3)


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (BF, E4M3), (F32, F32), (F32, E4M3)])
@pytest.mark.parametrize("D,heads", [(128, 4), (64, 9), (256, 2)])
def test_more_tokens_than_blocks_take_at_once(dtype, kind, D, heads):
    """Several rows of a lane on their way, and more sequences than threads that look for a token's."""
    news = [(7 * i) % 29 for i in range(720)]
    _check_write_and_read(dtype, kind, 16, [n + i % 3 for i, n in enumerate(news)], news, True, D, heads)


def test_rounding_of_every_border():
    """Rows whose largest entry lies at, just below and just above each 448 2^e, and entries at the ties between
    neighbouring e4m3 numbers."""
    top = torch.cat([torch.tensor([448.0, 447.9, 448.1, 449.0, 256.0, 255.0, 224.0, 1.75, 1.7500001, 2.0]) * 2.0 ** e for e in range(-20, 20)])
    x = torch.zeros(1, len(top), 1, 128)
    x[0, :, 0, 0] = top
    lattice = torch.tensor([1.0625, 1.1875, 1.3125, 1.9375, 0.5 * 2.0 ** -9, 1.5 * 2.0 ** -9, 2.0 ** -9, 7.5 * 2.0 ** -9])
    x[0, :, 0, 1:9] = lattice * aref.row_unit(x[0, :, 0].double())[:, None].float()
    x[0, :, 0, 9:17] = -x[0, :, 0, 1:9]
    cache = KVCache.empty(-(-len(top) // 16), 1, 16, 128, E4M3)
    table = torch.arange(len(cache.k), dtype=torch.int32, device=dev)[None]
    lens = torch.tensor([len(top)], dtype=torch.int32, device=dev)
    kv_cache_write(x.to(dev), x.to(dev), cache, table, lens)
    want, unit = _expect(x[0], E4M3)
    k, _ = kv_cache_read(cache, table, lens, len(top), dtype=F32)
    assert torch.equal(k[0].cpu().double(), want * unit[..., None])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_finite_and_extremes(dtype):
    big = float(torch.finfo(dtype).max)
    x = torch.ones(1, 6, 1, 64).to(dtype)
    x[0, 0, 0, 3] = float("nan")
    x[0, 1, 0, 5] = float("inf")
    x[0, 2, 0, 7] = -float("inf")
    x[0, 3, 0, 9] = big / 2
    x[0, 4] = float("nan")
    x[0, 5] = 2.0 ** -131  # below the least power of two: 2^-5 of it, exact
    cache = KVCache.empty(1, 1, 16, 64, E4M3)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.tensor([6], dtype=torch.int32, device=dev)
    kv_cache_write(x.to(dev), x.to(dev), cache, table, lens)
    k, v = kv_cache_read(cache, table, lens, 6, dtype=dtype)
    assert torch.equal(torch.nan_to_num(k, nan=-7.0), torch.nan_to_num(v, nan=-7.0))
    k = k.float().cpu()[0, :, 0]
    ones = torch.ones(64)
    assert bool(torch.isnan(k[0, 3])) and torch.equal(torch.cat([k[0, :3], k[0, 4:]]), ones[1:])
    assert k[1, 5] == float("inf") and k[2, 7] == -float("inf")
    want, unit = _expect(x[0, 3].double(), E4M3)
    assert torch.equal(k[3].double(), (want * unit[..., None])[0])
    assert bool(torch.isnan(k[4]).all()) and torch.equal(k[5], torch.full((64,), 2.0 ** -131))


@pytest.mark.parametrize("kind", [BF, E4M3])
def test_slices(kind):
    """k and v out of one projection, pages of one layer out of a buffer of several, a table's first columns."""
    g = torch.Generator().manual_seed(9)
    alone = KVCache.empty(6, 2, 16, 64, kind)
    wide = [None if t is None else torch.stack([index(t)] * 3, 1).view(t.dtype) for t in alone]
    old = [None if t is None else index(t).clone() for t in wide]
    cache = KVCache(*(None if t is None else t[:, 1] for t in wide))
    qkv = torch.randn(3, 9, 10 * 64, generator=g).to(BF).to(dev)
    k, v = qkv[..., 4 * 64:6 * 64].unflatten(-1, (2, 64)), qkv[..., 8 * 64:].unflatten(-1, (2, 64))
    table = torch.tensor([[0, 3, -1, -1], [1, 4, -1, -1], [5, 2, -1, -1]], dtype=torch.int32, device=dev)
    lens = torch.tensor([20, 9, 32], dtype=torch.int32, device=dev)
    kv_cache_write(k, v, cache, table[:, :2], lens)
    kv_cache_write(k.contiguous(), v.contiguous(), alone, table, lens)
    for a, b in zip(cache, alone):
        if a is not None:
            assert torch.equal(index(a), index(b))
    for t, before in zip(wide, old):
        if t is not None:
            assert torch.equal(index(t)[:, ::2], before[:, ::2])
    a, b = kv_cache_read(cache, table[:, :2], lens, 9), kv_cache_read(alone, table, lens, 9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_bad_pages_and_lengths_are_reported():
    """Pages outside the cache are neither written nor read; lengths outside the table are taken as the nearest."""
    stream = torch.cuda.current_stream().cuda_stream
    kda.kda_get_device_error(stream)
    k = torch.ones(2, 4, 1, 64, dtype=BF, device=dev)
    for pages, cached in (([[0, 7], [1, -3]], [20, 20]), ([[0, 2], [1, 3]], [-1, 4]), ([[0, 2], [1, 3]], [4, 1 << 30])):
        cache = KVCache.empty(4, 1, 16, 64, BF)
        table = torch.tensor(pages, dtype=torch.int32, device=dev)
        lens = torch.tensor(cached, dtype=torch.int32, device=dev)
        kv_cache_write(k, k, cache, table, lens)
        assert kda.kda_get_device_error(stream) == attention.KDA_DEVICE_ERR_CACHE
        a, _ = kv_cache_read(cache, table, lens, 4)
        assert kda.kda_get_device_error(stream) == attention.KDA_DEVICE_ERR_CACHE
        assert bool(torch.isfinite(a).all())
        if cached[0] == 20:
            assert not cache.k.any() and not a.any()
    assert kda.kda_get_device_error(stream) == 0


def test_places_beyond_32_bits():
    """Pages whose offsets pass 2^31 elements and 2^32 bytes."""
    pages = (1 << 32) // (64 * 256) + 3
    cache = KVCache(*(torch.zeros(pages, 1, 64, 256, dtype=BF, device=dev) for _ in "kv"))
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(1, 130, 1, 256, generator=g).to(BF).to(dev) for _ in "kv")
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device=dev)
    lens = torch.tensor([130], dtype=torch.int32, device=dev)
    kv_cache_write(k, v, cache, table, lens)
    assert torch.equal(cache.k[pages - 1, 0], k[0, :64, 0]) and torch.equal(cache.v[pages - 2, 0, :2], v[0, 128:, 0])
    a, b = kv_cache_read(cache, table, lens, 130)
    assert torch.equal(a, k) and torch.equal(b, v)
