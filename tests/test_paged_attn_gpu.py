"""Attention of the next tokens over a paged cache on the GPU against its 64-bit definition (attention_reference). Every
place of the caches that no position of a sequence holds is NaN, and every entry of a table beyond a sequence's
length names no page.

Tolerances: the result is rounded once to its type. fp32: a score is a sum of at most 256 products (below 2^-20 of
|q| |k| scale, at most 20 here), its exponential adds 2^-22, the sums over keys are pairwise over warps and
blocks: 2^-17 together. bf16: scores as in fp32 (products of bf16 numbers are exact in it), each probability rounded
to bf16 once more, off by 2^-8 at most; on values without a common sign those errors add up as the values
themselves do: 2^-8 of the result. lse: the scores' error, absolute.
"""

from __future__ import annotations

import math

import pytest
import torch

import attention_reference as aref
import mixer_reference as ref
from attention_cases import BF, E4M3, F32, filled, index, to_gpu
from chunkwise_gated_linear_gb300 import KVCache, attention, kda, paged_attn_step, qk_norm_step, rope_frequencies

pytestmark = pytest.mark.gpu
dev = "cuda"
WORK = {BF: 2.0 ** -8 + 2.0 ** -17, F32: 2.0 ** -17}
KINDS = [(BF, BF), (BF, E4M3), (F32, F32), (F32, E4M3)]


def _q(g, B, T, Hq, D, dtype, kind):
    # scores of a spread of about 2
    std = 2.0 / (1.5 if kind == E4M3 else 1.0)
    return (torch.randn(B, T, Hq, D, generator=g) * std).to(dtype)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _check(q, cache, table, lens, dtype, scale=None):
    """The call on the GPU against the definition; cache and table on the CPU."""
    D = q.shape[3]
    want, lse_w = aref.attention(q, cache, table, lens, D ** -0.5 if scale is None else scale)
    o, lse = paged_attn_step(q.to(dev), to_gpu(cache), table.to(dev), _int32(lens), scale=scale, want_lse=True)
    ref.check("o", o, want, dtype, WORK[dtype])
    lse = lse.double().cpu()
    empty = torch.isinf(lse_w)
    assert torch.equal(torch.isinf(lse), empty) and bool((lse[empty] < 0).all())
    assert not o.cpu()[empty].any()
    if not bool(empty.all()):
        off = float((lse - lse_w)[~empty].abs().max())
        print(f"lse: {off:.2e}")
        assert off <= 2.0 ** -16
    assert torch.equal(o, paged_attn_step(q.to(dev), to_gpu(cache), table.to(dev), _int32(lens), scale=scale))
    return o


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("D", [16, 64, 80, 128, 192, 256])
@pytest.mark.parametrize("heads,group", [(2, 1), (3, 4), (1, 8), (2, 5), (1, 16), (1, 33), (1, 71)])
def test_head_layouts(dtype, kind, D, heads, group):
    lens = [1, 63, 64, 65, 0, 300]
    g = torch.Generator().manual_seed(D + group)
    cache, table = filled(g, lens, 16, heads, D, kind)
    _check(_q(g, len(lens), 1, heads * group, D, dtype, kind), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 100, 256])
def test_pages(dtype, kind, page):
    lens = [5, 129, 640, 17, 1]
    g = torch.Generator().manual_seed(page)
    cache, table = filled(g, lens, page, 2, 128, kind)
    _check(_q(g, len(lens), 1, 8, 128, dtype, kind), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("T,group", [(2, 1), (4, 8), (3, 5), (8, 4), (17, 2), (70, 1), (5, 16)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_several_tokens(dtype, kind, T, group, D):
    """Each sees the ones before it; sequences shorter than the new tokens have rows that see nothing."""
    lens = [T, T + 1, 200, 2, 0, 64 + T // 2]
    g = torch.Generator().manual_seed(T)
    cache, table = filled(g, lens, 16, 2, D, kind)
    _check(_q(g, len(lens), T, 2 * group, D, dtype, kind), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("lens", [[5000], [0], [1], [40000, 3], [20000] + [1] * 40, list(range(0, 700, 3))])
def test_lengths(dtype, kind, lens):
    """One long sequence over all SMs, uneven batches, more sequences than threads that plan them."""
    g = torch.Generator().manual_seed(len(lens))
    cache, table = filled(g, lens, 32, 2, 64, kind)
    _check(_q(g, len(lens), 1, 8, 64, dtype, kind), cache, table, lens, dtype)


def test_more_sequences_than_a_block_has_threads():
    lens = [(7 * i) % 90 for i in range(1000)]
    g = torch.Generator().manual_seed(1)
    cache, table = filled(g, lens, 16, 1, 64, BF)
    _check(_q(g, len(lens), 1, 2, 64, BF, BF), cache, table, lens, BF)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("size", [0.0, 30.0, -1.0])
def test_sharp_and_flat_scores(dtype, kind, size):
    """Scores that all agree, that leave one key (growing along the sequence, so that the running maximum keeps
    changing), and that fall from the first key on. A score of 300 is off by 2^-24 of it times 16 in 32 bits."""
    lens = [1000, 77]
    g = torch.Generator().manual_seed(2)
    cache, table = filled(g, lens, 16, 1, 64, F32 if kind == E4M3 else kind)
    q = torch.zeros(2, 1, 4, 64)
    q[..., 0] = 8.0 if size else 0.0
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        ramp = torch.arange(n).float() / n * abs(size)
        cache.k[table[b].long()[pos // 16], 0, pos % 16, 0] = (ramp if size > 0 else -ramp).to(cache.k.dtype)
    if kind == E4M3:
        nan = torch.isnan(cache.k)
        made = []
        for t in (cache.k, cache.v):
            x = torch.nan_to_num(t).double()
            unit = aref.row_unit(x)
            made.append(((x / unit[..., None]).float().to(E4M3), torch.log2(unit).add(127).to(torch.uint8).view(torch.float8_e8m0fnu)))
        cache = KVCache(made[0][0], made[1][0], made[0][1], made[1][1])
        index(cache.k)[nan] = 0x7F
        index(cache.v)[nan] = 0x7F
    _check(q.to(dtype), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("D,group", [(64, 2), (64, 1), (128, 5), (64, 8), (256, 3), (256, 6)])
def test_values_without_a_meaning_stay_where_no_row_sees_them(dtype, kind, D, group):
    """NaN and infinities at positions that only later tokens of the call see do not reach earlier ones."""
    lens, T = [70, 9, 200], 5
    g = torch.Generator().manual_seed(3)
    cache, table = filled(g, lens, 16, 2, D, kind)
    q = _q(g, 3, T, 2 * group, D, dtype, kind)
    clean = _check(q, cache, table, lens, dtype)
    bad = KVCache(*(None if t is None else t.clone() for t in cache))
    for b, n in enumerate(lens):
        pos = n - 2  # seen by the last two tokens
        for t, at in ((bad.k, 3), (bad.v, 5)):
            index(t)[table[b, pos // 16].long(), 0, pos % 16, at] = 0x7F if kind == E4M3 else float("nan")
            if kind != E4M3:
                t[table[b, (pos + 1) // 16].long(), 0, (pos + 1) % 16, at] = float("inf")
    o = paged_attn_step(q.to(dev), to_gpu(bad), table.to(dev), _int32(lens))
    assert torch.equal(o[:, :T - 2], clean[:, :T - 2])
    assert torch.equal(o[:, :, group:], clean[:, :, group:])  # the other key head
    assert bool(torch.isnan(o[:, T - 2:, :group]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_finite_are_kept_where_seen(dtype):
    """A NaN value reaches its own channel alone, a NaN key the whole row."""
    lens = [90]
    g = torch.Generator().manual_seed(4)
    cache, table = filled(g, lens, 16, 2, 64, dtype)
    cache.v[table[0, 2].long(), 0, 3, 7] = float("nan")
    cache.k[table[0, 1].long(), 1, 3, 7] = float("nan")
    o = paged_attn_step(_q(g, 1, 1, 4, 64, dtype, dtype).to(dev), to_gpu(cache), table.to(dev), _int32(lens)).cpu()
    bad = torch.isnan(o)
    want = torch.zeros_like(bad)
    want[..., :2, 7] = True
    want[..., 2:, :] = True
    assert torch.equal(bad, want)


def test_scale_and_large_scales_of_rows():
    g = torch.Generator().manual_seed(5)
    lens = [130, 31]
    cache, table = filled(g, lens, 16, 2, 128, BF)
    q = _q(g, 2, 1, 4, 128, BF, BF)
    for scale in (0.0, 0.25, -0.1):
        _check(q, cache, table, lens, BF, scale=scale)
    # rows of an 8-bit cache whose values differ by 2^60 between keys
    cache, table = filled(g, lens, 16, 2, 128, E4M3)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        at = table[b].long()[pos // 16]
        index(cache.v_scale)[at, :, pos % 16] = (90 + 60 * (pos % 2))[:, None].to(torch.uint8)
    _check(q / 2, cache, table, lens, BF)


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_slices(dtype, kind):
    """q out of one projection, pages of one layer out of a buffer of several, a table's first columns."""
    g = torch.Generator().manual_seed(6)
    lens = [100, 33, 1]
    cache, table = filled(g, lens, 16, 2, 64, kind)
    qkv = (torch.randn(3, 2, 12 * 64, generator=g)).to(dtype).to(dev)
    q = qkv[..., 2 * 64:10 * 64].unflatten(-1, (8, 64))
    c = to_gpu(cache)
    wide = KVCache(*(None if t is None else torch.stack([index(t)] * 3, 1).view(t.dtype)[:, 1] for t in c))
    more = torch.full((3, 40), -1, dtype=torch.int32, device=dev)
    more[:, :table.shape[1]] = table.to(dev)
    want = paged_attn_step(q.contiguous(), c, table.to(dev), _int32(lens))
    assert torch.equal(paged_attn_step(q, wide, more[:, :table.shape[1]], _int32(lens)), want)


def test_places_beyond_32_bits():
    """Pages whose offsets pass 2^31 elements and 2^32 bytes."""
    g = torch.Generator().manual_seed(7)
    lens = [200]
    small, table = filled(g, lens, 64, 1, 256, BF)
    pages = (1 << 32) // (64 * 256) + 8
    cache = KVCache(*(torch.zeros(pages, 1, 64, 256, dtype=BF, device=dev) for _ in "kv"))
    far = table.clone()
    for i in range(4):
        far[0, i] = pages - 1 - 2 * i
        for a, b in zip(cache, small):
            if a is not None:
                a[pages - 1 - 2 * i] = b[table[0, i].long()].to(dev)
    q = _q(g, 1, 1, 4, 256, BF, BF)
    want = paged_attn_step(q.to(dev), to_gpu(small), table.to(dev), _int32(lens))
    assert torch.equal(paged_attn_step(q.to(dev), cache, far.to(dev), _int32(lens)), want)


def test_shared_pages_and_joined_caches():
    """Two sequences with one prefix's pages; lse joins the results over a cache cut in two."""
    g = torch.Generator().manual_seed(8)
    cache, table = filled(g, [96], 16, 2, 64, F32)
    q = _q(g, 1, 1, 4, 64, F32, F32).to(dev)
    c, t = to_gpu(cache), table.to(dev)
    both = paged_attn_step(q.expand(2, -1, -1, -1).contiguous(), c, t.expand(2, -1).contiguous(), _int32([96, 96]))
    whole = paged_attn_step(q, c, t, _int32([96]))
    for i in range(2):  # a batch may cut its sequences elsewhere
        ref.check("shared", both[i:i + 1], whole.double().cpu(), F32, WORK[F32])
    o1, l1 = paged_attn_step(q, c, t, _int32([64]), want_lse=True)
    o2, l2 = paged_attn_step(q, c, t[:, 4:].contiguous(), _int32([32]), want_lse=True)
    w = torch.sigmoid(l1 - l2)[..., None]
    ref.check("joined", o1 * w + o2 * (1 - w), whole.double().cpu(), F32, 2 * WORK[F32])


@pytest.mark.parametrize("dtype,kind", KINDS)
def test_bad_pages_and_lengths_are_reported(dtype, kind):
    g = torch.Generator().manual_seed(9)
    stream = torch.cuda.current_stream().cuda_stream
    cache, table = filled(g, [60, 60], 16, 1, 64, kind)
    q = _q(g, 2, 1, 4, 64, dtype, kind).to(dev)
    c = to_gpu(cache)
    kda.kda_get_device_error(stream)
    bad = table.clone()
    bad[1, 2] = cache.k.shape[0]
    o = paged_attn_step(q, c, bad.to(dev), _int32([60, 60]))
    assert kda.kda_get_device_error(stream) == attention.KDA_DEVICE_ERR_CACHE
    assert bool(torch.isfinite(o).all())
    want = paged_attn_step(q, c, table.to(dev), _int32([60, 60]))
    assert kda.kda_get_device_error(stream) == 0 and torch.equal(o[0], want[0])
    short = table[:, :4].contiguous().to(dev)
    o = paged_attn_step(q, c, short, _int32([-3, 60]))
    assert kda.kda_get_device_error(stream) == attention.KDA_DEVICE_ERR_CACHE
    assert not o[0].any() and bool(torch.isfinite(o).all())
    filled_up = to_gpu(filled(g, [64, 64], 16, 1, 64, kind)[0])
    o = paged_attn_step(q, filled_up, short, _int32([64, 1 << 30]))
    assert kda.kda_get_device_error(stream) == attention.KDA_DEVICE_ERR_CACHE


@pytest.mark.parametrize("dtype,kind", [(BF, E4M3), (F32, F32)])
def test_graphs_streams_and_growing_lengths(dtype, kind):
    """Two captured calls, each with scratch of its own, replayed in turn on another stream while the lengths grow in
    place: the plan is made on the device, from the lengths of the moment."""
    g = torch.Generator().manual_seed(10)
    most = [700, 90, 2000]
    cache, table = filled(g, most, 16, 2, 64, kind)
    c, t, lens = to_gpu(cache), table.to(dev), _int32([1, 90, 500])
    qs = [_q(g, 3, 1, 8, 64, dtype, kind).to(dev) for _ in range(2)]
    outs, graphs = [], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for q in qs:
            paged_attn_step(q, c, t, lens)
    torch.cuda.synchronize()
    for q in qs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(paged_attn_step(q, c, t, lens))
        graphs.append(gr)
    for now in ([1, 90, 500], [2, 0, 501], [700, 64, 2000]):
        lens.copy_(_int32(now))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for gr in graphs + graphs:
                gr.replay()
        torch.cuda.synchronize()
        for q, o in zip(qs, outs):
            assert torch.equal(o, paged_attn_step(q, c, t, lens))
            want, _ = aref.attention(q.cpu(), cache, table, now, 64 ** -0.5)
            ref.check("replayed", o, want, dtype, WORK[dtype])


def test_a_captured_serving_step():
    """Norms with the write, attention and the count of the new tokens in one graph, replayed as the sequences grow: the same bits as
    the calls one by one."""
    g = torch.Generator().manual_seed(16)
    B, Hq, H, D, page, start = 3, 8, 2, 64, 16, [0, 15, 300]
    table = torch.arange(B * 21, dtype=torch.int32, device=dev).view(B, 21)
    freq, w = rope_frequencies(D), torch.ones(D, device=dev)
    tokens = [[torch.randn(B, 1, h, D, generator=g).to(BF).to(dev) for h in (Hq, H, H)] for _ in range(20)]
    caches, counts = [KVCache.empty(B * 21, H, page, D, E4M3) for _ in range(2)], [_int32(start) for _ in range(2)]

    def step(q, k, v, cache, lens):
        lens.add_(1)
        return paged_attn_step(qk_norm_step(q, k, v, cache, table, lens, w, w, freq), cache, table, lens)

    want = [step(*x, caches[0], counts[0]) for x in tokens]
    side = [x.clone() for x in tokens[0]]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step(*side, caches[1], counts[1])
    for x, o in zip(tokens, want):
        for a, b in zip(side, x):
            a.copy_(b)
        graph.replay()
        assert torch.equal(got, o)
    assert all(torch.equal(index(a), index(b)) for a, b in zip(*caches)) and counts[1].tolist() == [n + 20 for n in start]


def test_calls_on_two_streams_at_once():
    g = torch.Generator().manual_seed(11)
    cache, table = filled(g, [9000], 64, 4, 128, BF)
    c, t, lens = to_gpu(cache), table.to(dev), _int32([9000])
    qs = [_q(g, 1, 1, 16, 128, BF, BF).to(dev) for _ in range(2)]
    want = [paged_attn_step(q, c, t, lens) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(20):
        got = []
        for s, q in zip(streams, qs):
            with torch.cuda.stream(s):
                got.append(paged_attn_step(q, c, t, lens))
        # and with the library's own scratch, on a stream given by its handle
        got.append(paged_attn_step(qs[0], c, t, lens, o=torch.empty_like(qs[0]), stream=streams[1].cuda_stream))
        torch.cuda.synchronize()
        for o, w in zip(got, want + want[:1]):
            assert torch.equal(o, w)


def test_no_tokens_and_given_outputs():
    g = torch.Generator().manual_seed(12)
    cache, table = filled(g, [20], 16, 1, 64, BF)
    c, t, lens = to_gpu(cache), table.to(dev), _int32([20])
    assert paged_attn_step(torch.empty(1, 0, 4, 64, dtype=BF, device=dev), c, t, lens).shape == (1, 0, 4, 64)
    q = _q(g, 1, 1, 4, 64, BF, BF).to(dev)
    o, lse = torch.empty_like(q), torch.empty(1, 1, 4, device=dev)
    got = paged_attn_step(q, c, t, lens, want_lse=True, o=o, lse=lse)
    assert got[0] is o and got[1] is lse and math.isfinite(float(lse.sum()))
    kept = lse.clone()
    lse.zero_()
    got = paged_attn_step(q, c, t, lens, lse=lse)  # given is wanted
    assert got[1] is lse and torch.equal(lse, kept)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("zeros", ["first", "all", "most"])
def test_rows_of_zeros_in_an_8_bit_cache(dtype, zeros):
    """A row of zeros has the least power of two, 2^-126: it counts in the softmax's sum like any other."""
    g = torch.Generator().manual_seed(13)
    lens = [150, 16, 1]
    cache, table = filled(g, lens, 16, 2, 64, E4M3)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        pos = pos[:40] if zeros == "first" else pos if zeros == "all" else pos[pos % 37 != 5]
        at = table[b].long()[pos // 16]
        index(cache.v)[at, :, pos % 16] = 0
        index(cache.v_scale)[at, :, pos % 16] = 1
    _check(_q(g, 3, 1, 8, 64, dtype, E4M3), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tiny_values_in_an_8_bit_cache(dtype):
    """All values near the least power of two: nothing of them is lost before the result is rounded."""
    g = torch.Generator().manual_seed(14)
    lens = [300, 40]
    cache, table = filled(g, lens, 16, 2, 64, E4M3)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        index(cache.v_scale)[table[b].long()[pos // 16], :, pos % 16] = (5 + 20 * (pos % 2))[:, None].to(torch.uint8)
    _check(_q(g, 2, 1, 8, 64, dtype, E4M3), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 3])
def test_power_of_two_that_is_no_number_stays_in_its_sequence(dtype, T):
    """The byte 255 (NaN) in one sequence's scales: the sequences beside it, worked on after it by the same warps, are as they
    are without it."""
    g = torch.Generator().manual_seed(15)
    lens = [37, 5] * 1000
    cache, table = filled(g, lens, 16, 8, 64, E4M3)
    q = _q(g, len(lens), T, 32, 64, dtype, E4M3)
    call = lambda: paged_attn_step(q.to(dev), to_gpu(cache), table.to(dev), _int32(lens))  # noqa: E731
    want = call()
    for b in range(0, len(lens), 2):
        pos = torch.arange(lens[b])
        index(cache.v_scale)[table[b].long()[pos // 16], :, pos % 16] = 0xFF
    assert bool(torch.isfinite(want).all()) and torch.equal(call()[1::2], want[1::2])


def _places(table, b, pos, page=16):
    """Page, key head 0 and row of a position, as an index."""
    return table[b, pos // page].long(), 0, pos % page


def _infinite_row(t, scale, at, channel):
    """The row of an 8-bit cache at `at` as kv_cache_write leaves it when one channel is infinite: 448 2^120, and zeros."""
    row = torch.zeros(t.shape[3], dtype=torch.uint8)
    row[channel] = 0x7E
    index(t)[at] = row
    index(scale)[at] = 120 + 127


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("part", ["k", "v", "kv"])
@pytest.mark.parametrize("D,group", [(64, 1), (64, 2), (128, 5), (64, 8), (256, 3), (256, 6), (128, 13)])
def test_infinities_of_an_8_bit_cache_stay_where_no_row_sees_them(dtype, part, D, group):
    """The last new token's key or value has an infinity: the tokens before it, and the other key head, are as defined."""
    lens, T = [70, 9, 200, 5], 5
    g = torch.Generator().manual_seed(17)
    cache, table = filled(g, lens, 16, 2, D, E4M3)
    q = _q(g, len(lens), T, 2 * group, D, dtype, E4M3)
    for b, n in enumerate(lens):
        at = _places(table, b, n - 1)
        if "k" in part:
            _infinite_row(cache.k, cache.k_scale, at, 3)
        if "v" in part:
            _infinite_row(cache.v, cache.v_scale, at, 5)
    want, _ = aref.attention(q, cache, table, lens, D ** -0.5)
    o = paged_attn_step(q.to(dev), to_gpu(cache), table.to(dev), _int32(lens))
    ref.check("before", o[:, :T - 1], want[:, :T - 1], dtype, WORK[dtype])
    ref.check("other head", o[:, :, group:], want[:, :, group:], dtype, WORK[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("score,byte", [(-208.0, 143), (-28.0, 143), (-208.0, 200)])
def test_large_values_of_little_weight_after_rows_of_zeros(dtype, T, score, byte):
    """Powers of two 2^142 and more apart: the rows of zeros have nearly all of the weight, the others e^-28 of it or, at
    e^-208, none that 32 bits hold (such a result is 0)."""
    g = torch.Generator().manual_seed(18)
    lens = [100, 41]
    cache, table = filled(g, lens, 16, 1, 64, E4M3)
    q = torch.zeros(2, T, 4, 64)
    q[..., 0] = 8.0  # times 64^-1/2: a key's channel 0 is its score
    index(cache.k_scale)[:] = 127
    for b, n in enumerate(lens):
        for pos in range(n):
            at = _places(table, b, pos)
            row = torch.zeros(64)
            row[0] = score if pos >= 38 else 0.0
            index(cache.k)[at] = row.to(E4M3).view(torch.uint8)
            index(cache.v_scale)[at] = byte if pos >= 38 else 1
            if pos < 38:
                index(cache.v)[at] = 0
    want, _ = aref.attention(q, cache, table, lens, 0.125)
    o = paged_attn_step(q.to(dtype).to(dev), to_gpu(cache), table.to(dev), _int32(lens))
    if score < -200:
        assert not o.any()
    else:
        ref.check("o", o, want, dtype, WORK[dtype])


@pytest.mark.parametrize("dtype,kind", KINDS)
@pytest.mark.parametrize("D,group", [(64, 1), (64, 2), (128, 4), (64, 8), (256, 3), (256, 6), (128, 13)])
@pytest.mark.parametrize("what", ["key", "value", "nan", "infinity"])
def test_results_do_not_depend_on_what_a_row_does_not_see(dtype, kind, D, group, what):
    """With another key or value at the last position the tokens before are the same bit for bit: no rounding of theirs
    follows from what other rows see."""
    lens, T = [25, 40, 70, 9, 200, 6] * 60, 5  # so many that a warp goes through several units of a sequence
    g = torch.Generator().manual_seed(19)
    cache, table = filled(g, lens, 16, 2, D, kind)
    q = _q(g, len(lens), T, 2 * group, D, dtype, kind)
    bad = KVCache(*(None if t is None else t.clone() for t in cache))
    for b, n in enumerate(lens):
        at = _places(table, b, n - 1)
        for t, scale, times in ((bad.k, bad.k_scale, 5 if what == "key" else 0), (bad.v, bad.v_scale, 14 if what == "value" else 0)):
            if what == "nan":
                index(t)[at] = 0x7F if kind == E4M3 else float("nan")
            elif what == "infinity" and kind == E4M3:
                _infinite_row(t, scale, at, 5)
            elif what == "infinity":
                t[(*at, 5)] = float("inf")
            elif kind == E4M3:
                index(scale)[at] += times
            else:
                t[at] *= 2.0 ** times
    call = lambda c: paged_attn_step(q.to(dev), to_gpu(c), table.to(dev), _int32(lens), want_lse=True)  # noqa: E731
    for x, y in zip(call(bad), call(cache)):
        assert torch.equal(x[:, :T - 1], y[:, :T - 1])
        assert torch.equal(x[:, :, group:], y[:, :, group:])  # the other key head


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_of_zero_from_keys_and_queries_of_far_sizes(dtype):
    """Keys with the largest power of two, 2^127, meet entries of 2^20 of a query only in zeros: their scores are 0."""
    g = torch.Generator().manual_seed(20)
    lens = [70, 5]
    cache, table = filled(g, lens, 16, 1, 64, E4M3)
    q = torch.zeros(2, 1, 4, 64)
    q[..., 0] = 2.0 ** 20
    for b, n in enumerate(lens):
        for pos in range(n):
            at = _places(table, b, pos)
            index(cache.k)[(*at, 0)] = 0
            if pos % 2:
                index(cache.k_scale)[at] = 254
    _check(q.to(dtype), cache, table, lens, dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("group", [1, 4, 16])
def test_scores_that_are_all_minus_infinity(dtype, group):
    """Such a row is empty whatever its values are, in one piece or in many."""
    g = torch.Generator().manual_seed(21)
    lens = [5, 300, 20000, 0]
    cache, table = filled(g, lens, 16, 1, 64, dtype)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        at = table[b].long()[pos // 16], 0, pos % 16
        cache.k[(*at, 0)] = -float("inf")
        cache.v[(*at, 7)] = float("nan")
        cache.v[(*at, 9)] = float("inf")
    q = _q(g, len(lens), 2, group, 64, dtype, dtype)
    q[..., 0] = 1.0
    o, lse = paged_attn_step(q.to(dev), to_gpu(cache), table.to(dev), _int32(lens), want_lse=True)
    assert torch.equal(o, torch.zeros_like(o)) and torch.equal(lse, torch.full_like(lse, -math.inf))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("part,q0", [("v", 24.0), ("k", 0.01), ("k", -0.01)])
def test_an_infinity_of_an_8_bit_cache_counts_as_the_number_it_is_held_as(dtype, part, q0):
    """448 2^120, of a value with weight e^-3 beside ones of weight 1, and of a key, which then has all of the weight or none."""
    g = torch.Generator().manual_seed(22)
    lens = [70, 200]
    cache, table = filled(g, lens, 16, 1, 64, E4M3)
    q = torch.zeros(2, 1, 4, 64)
    q[..., 0] = q0
    for b, n in enumerate(lens):
        for pos in range(n):
            at = _places(table, b, pos)
            index(cache.k)[(*at, 0)] = torch.tensor(1.0 if pos != 37 else 0.0).to(E4M3).view(torch.uint8)
            index(cache.k_scale)[at] = 127
        if part == "v":
            _infinite_row(cache.v, cache.v_scale, _places(table, b, 37), 5)
        else:
            _infinite_row(cache.k, cache.k_scale, _places(table, b, 37), 0)
    q = q.to(dtype)
    want, _ = aref.attention(q, cache, table, lens, 0.125)
    o = paged_attn_step(q.to(dev), to_gpu(cache), table.to(dev), _int32(lens))
    ref.check("o", o, want, dtype, WORK[dtype])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("kbyte", [128, 130, 132, 134, 136, 138, 146, 200, 240])
@pytest.mark.parametrize("vbyte", [86, 106, 113, 121, 145])
def test_large_scores_over_an_8_bit_cache(dtype, sign, kbyte, vbyte):
    """Scores of 2^13 to 2^33, of which one key's is far above the others' (they differ by parts of themselves): the result is
    that key's value, however large or small the values are."""
    g = torch.Generator().manual_seed(23)
    lens = [70, 300]
    cache, table = filled(g, lens, 16, 1, 64, E4M3)
    q = torch.zeros(2, 2, 4, 64)
    q[..., 0] = sign * 2.0 ** 13 / 2.0 ** max(0, kbyte - 140)
    for b, n in enumerate(lens):
        for pos in range(n):
            at = _places(table, b, pos)
            x = (448.0 if pos == 37 else 20.0 + pos % 17) if sign > 0 else (20.0 if pos == 37 else 400.0 + 10 * (pos % 3))
            index(cache.k)[(*at, 0)] = torch.tensor(x).to(E4M3).view(torch.uint8)
            index(cache.k_scale)[at] = kbyte
            index(cache.v_scale)[at] = vbyte
    want = aref.attention(q, cache, table, lens, 0.125)[0]
    o = paged_attn_step(q.to(dtype).to(dev), to_gpu(cache), table.to(dev), _int32(lens))
    ref.check("o", o, want, dtype, WORK[dtype])
