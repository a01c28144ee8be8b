"""Norms of queries and keys with the position rotation on the GPU against their 64-bit definition
(attention_reference): forward, gradient, and the form that writes the cache.

Tolerances: a result is rounded once to its type. Before that: a sum of at most 256 squares in 32 bits (8 in a row,
then pairwise: 13 roundings), the root and two products, and the rotation: the angle is off by at most
2^-25 half turns, cosine and sine by two units of 2^-24 each, two products and a sum: below 2^-19 of the row's norm
together. Sums over up to 12,000 rows and heads for the weights' gradients: sqrt(12000) 2^-24 < 2^-17.
"""

from __future__ import annotations

import pytest
import torch

import attention_reference as aref
import mixer_reference as ref
from attention_cases import BF, E4M3, E8M0, F32, index, tables
from chunkwise_gated_linear_gb300 import KVCache, kda, kv_cache_write, qk_norm_bwd, qk_norm_fwd, qk_norm_step, rope_frequencies

pytestmark = pytest.mark.gpu
WORK, SUMS = 2.0 ** -19, 2.0 ** -17
EPS = 1e-6
dev = "cuda"


def _r(g, *s, dt=F32, std=1.0):
    return (torch.randn(*s, generator=g) * std).to(dt).to(dev)


def _case(g, lens, packed, Hq, Hk, D, dtype, parts):
    shape = (1, sum(lens)) if packed else (len(lens), lens[0])
    q, k = _r(g, *shape, Hq, D, dt=dtype, std=2), _r(g, *shape, Hk, D, dt=dtype, std=0.5)
    qw = 1 + _r(g, D, std=0.3) if "q" in parts else None
    kw = 1 + _r(g, D, std=0.3) if "k" in parts else None
    cu = ref.cu_of(lens, dev) if packed else None
    pos = torch.cat([torch.arange(n) for n in lens])
    return q, k, qw, kw, cu, pos


def _check_all(q, k, qw, kw, cu, pos, R, dtype, interleaved, positions=None):
    g = torch.Generator().manual_seed(5)
    freq = rope_frequencies(R) if R else None
    kw_args = dict(positions=positions, cu_seqlens=cu, eps=EPS, interleaved=interleaved)
    v = ref.leaves(dict(q=q, k=k, qw=qw, kw=kw))
    rows = lambda t: t.flatten(0, 1)  # noqa: E731
    yq = aref.norm_rope(rows(v["q"]), v["qw"], pos, aref.inv_freq(R), EPS, interleaved)
    yk = aref.norm_rope(rows(v["k"]), v["kw"], pos, aref.inv_freq(R), EPS, interleaved)
    oq, ok = qk_norm_fwd(q, k, qw, kw, freq, **kw_args)
    ref.check("q", oq, yq.reshape(q.shape), dtype, WORK)
    ref.check("k", ok, yk.reshape(k.shape), dtype, WORK)
    dq, dk = _r(g, *q.shape, dt=dtype), _r(g, *k.shape, dt=dtype)
    want = ref.grads((yq, yk), (rows(dq), rows(dk)), v)
    got = qk_norm_bwd(q, k, qw, kw, freq, dq, dk, **kw_args)
    for name, o, key, dt, tol in zip(("dq", "dk", "dqw", "dkw"), got, ("q", "k", "qw", "kw"), (dtype, dtype, F32, F32),
                                     (WORK, WORK, SUMS, SUMS)):
        if v[key] is None:
            assert o is None
        else:
            ref.check(name, o, want[key], dt, tol)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (64, 64), (256, 64), (96, 48), (80, 40), (192, 192), (128, 0), (256, 256), (48, 32),
                                 (16, 16), (2, 2), (37, 6), (250, 250), (128, 6), (64, 24), (112, 64)])
def test_widths(dtype, interleaved, D, R):
    g = torch.Generator().manual_seed(D + R)
    args = _case(g, [37, 37], False, 6, 2, D, dtype, "qk")
    _check_all(*args, R, dtype, interleaved)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("parts", ["", "q", "k", "qk"])
@pytest.mark.parametrize("lens", [[1], [0, 5, 1, 0, 300, 17], [3000]])
@pytest.mark.parametrize("Hq,Hk", [(4, 1), (1, 1), (5, 3), (33, 3)])
def test_sequences_and_parts(dtype, parts, lens, Hq, Hk):
    if sum(lens) * (Hq + Hk) > 12000:
        Hq, Hk = 3, 1
    g = torch.Generator().manual_seed(Hq)
    args = _case(g, lens, True, Hq, Hk, 64, dtype, parts)
    _check_all(*args, 64, dtype, False)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("R,interleaved", [(64, False), (32, False), (64, True), (0, False)])
def test_more_tokens_than_blocks_take_at_once(dtype, R, interleaved):
    """Blocks go through several shares of the tokens, and look for their first one among more sequences than threads."""
    lens = [(7 * i) % 29 for i in range(720)]
    assert 9728 < sum(lens) < 12000
    args = _case(torch.Generator().manual_seed(11), lens, True, 1, 1, 64, dtype, "qk")
    _check_all(*args, R, dtype, interleaved)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_and_negative_positions(dtype):
    """Angles stay exact at positions where a product in 32 bits would have lost them."""
    g = torch.Generator().manual_seed(1)
    q, k, qw, kw, _, _ = _case(g, [9, 9], False, 2, 1, 128, dtype, "qk")
    pos = torch.randint(-(1 << 24), 1 << 24, (2, 9), generator=g).to(torch.int32)
    pos[0, :4] = torch.tensor([0, 1, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32)
    # the reference's own angles at 2^31 lose 2^31 2^-53 radians: far below WORK
    _check_all(q, k, qw, kw, None, pos.flatten(), 128, dtype, False, positions=pos.to(dev))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [128, 72, 37])
def test_slices_of_one_projection(dtype, D):
    """q and k read in place from [q | k | v] of each token give what contiguous copies give."""
    g = torch.Generator().manual_seed(2)
    qkv = _r(g, 3, 11, 7 * D, dt=dtype)
    q, k = qkv[..., :4 * D].unflatten(-1, (4, D)), qkv[..., 4 * D:6 * D].unflatten(-1, (2, D))
    w, freq = 1 + _r(g, D, std=0.2), rope_frequencies(D // 2 // 2 * 2)
    a = qk_norm_fwd(q, k, w, w, freq)
    b = qk_norm_fwd(q.contiguous(), k.contiguous(), w, w, freq)
    dq, dk = _r(g, *q.shape, dt=dtype), _r(g, *k.shape, dt=dtype)
    a += qk_norm_bwd(q, k, w, w, freq, dq, dk)
    b += qk_norm_bwd(q.contiguous(), k.contiguous(), w, w, freq, dq, dk)
    for x, y in zip(a, b):
        if D % 8:
            assert torch.equal(x, y)
        else:  # the copies may take another path (aligned rows): equal up to the order of the sums
            ref.check("slice", x, y.double().cpu(), x.dtype, WORK)


@pytest.mark.parametrize("D", [128, 40])
def test_in_place_and_given_outputs(D):
    g = torch.Generator().manual_seed(3)
    q, k, w, freq = _r(g, 2, 50, 4, D, dt=BF), _r(g, 2, 50, 2, D, dt=BF), 1 + _r(g, D, std=0.2), rope_frequencies(32)
    want = qk_norm_fwd(q, k, w, w, freq)
    a, b = q.clone(), k.clone()
    got = qk_norm_fwd(a, b, w, w, freq, q_out=a, k_out=b)
    assert got[0] is a and got[1] is b and torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_gradient_in_place_without_weights_gradients():
    from chunkwise_gated_linear_gb300 import attention

    g = torch.Generator().manual_seed(4)
    q, k, w, freq = _r(g, 1, 50, 4, 64, dt=BF), _r(g, 1, 50, 2, 64, dt=BF), 1 + _r(g, 64, std=0.2), rope_frequencies(64)
    dq, dk = _r(g, *q.shape, dt=BF), _r(g, *k.shape, dt=BF)
    want = qk_norm_bwd(q, k, w, w, freq, dq, dk)
    f = attention._norm_check(q, k, w, w, freq, None, None, 1e-6, False, None, None)
    a, b = dq.clone(), dk.clone()
    p = attention.kda_qk_norm_bwd_params(f, a.data_ptr(), b.data_ptr(), a.data_ptr(), b.data_ptr(), None, None, None, 0)
    assert attention.kda_qk_norm_bwd_workspace(p) == 0
    assert attention.kda_qk_norm_bwd(p, torch.cuda.current_stream().cuda_stream) == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_gradient_against_differences():
    """Central differences of the fp32 forward pass along a random direction: second-order error 1e-4 squared times
    curvature, roundings 2^-24 of terms of size 1 over a step of 1e-2 and 2000 terms."""
    g = torch.Generator().manual_seed(6)
    q, k, w, freq = _r(g, 1, 9, 3, 64), _r(g, 1, 9, 1, 64), 1 + _r(g, 64, std=0.2), rope_frequencies(64)
    cq, ck = _r(g, *q.shape), _r(g, *k.shape)
    way = [_r(g, *t.shape) for t in (q, k, w, w)]
    e = 1e-2
    val = lambda s: sum((o.double() * c.double()).sum() for o, c in zip(  # noqa: E731
        qk_norm_fwd(q + s * e * way[0], k + s * e * way[1], w + s * e * way[2], w + s * e * way[3], freq), (cq, ck)))
    diff = float((val(1) - val(-1)) / (2 * e))
    got = qk_norm_bwd(q, k, w, w, freq, cq, ck)
    want = float(sum((a.double() * b.double()).sum() for a, b in zip(got, way)))
    size = sum(float(a.norm() * b.norm()) for a, b in zip(got, way))
    assert abs(diff - want) <= 2e-3 * size


def test_no_tokens():
    q, k = torch.empty(2, 0, 4, 64, dtype=BF, device=dev), torch.empty(2, 0, 1, 64, dtype=BF, device=dev)
    w = torch.ones(64, device=dev)
    oq, ok = qk_norm_fwd(q, k, w, w, rope_frequencies(64))
    assert oq.shape == q.shape and ok.shape == k.shape
    got = qk_norm_bwd(q, k, w, None, rope_frequencies(64), q, k)
    assert got[0].shape == q.shape and torch.equal(got[2], torch.zeros_like(w)) and got[3] is None


def test_malformed_offsets_are_reported():
    q, k = torch.zeros(1, 8, 2, 64, dtype=BF, device=dev), torch.zeros(1, 8, 1, 64, dtype=BF, device=dev)
    stream = torch.cuda.current_stream().cuda_stream
    kda.kda_get_device_error(stream)
    for cu in ([0, 5, 3, 8], [1, 8], [0, 9], [0, -4, 8], [0, 100, 8]):
        qk_norm_fwd(q, k, freq=rope_frequencies(64), cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=dev))
        assert kda.kda_get_device_error(stream) == kda.KDA_DEVICE_ERR_SEQLENS
    assert kda.kda_get_device_error(stream) == 0


@pytest.mark.parametrize("dtype,kind", [(BF, BF), (BF, E4M3), (F32, F32), (F32, E4M3)])
@pytest.mark.parametrize("D,R,interleaved", [(128, 128, False), (64, 32, True), (256, 64, False), (80, 80, False), (16, 6, True)])
@pytest.mark.parametrize("cached,news,packed", [([5, 130, 64], [1, 1, 1], False), ([3, 0, 1, 40], [3, 3, 3, 3], False),
                                                ([70, 9, 0, 33, 1], [70, 4, 0, 1, 1], True)])
def test_step_writes_the_cache(dtype, kind, D, R, interleaved, cached, news, packed):
    """q as by qk_norm_fwd; k and v land at their positions, everything else stays; an 8-bit cache's values are the
    64-bit ones rounded once (half a step, 2^-4 of the value or 2^-10 of the row's power of two)."""
    g = torch.Generator().manual_seed(D)
    page, Hq, Hk = 16, 4, 2
    shape = (1, sum(news)) if packed else (len(news), news[0])
    q, k, v = (_r(g, *shape, h, D, dt=dtype) for h in (Hq, Hk, Hk))
    qw, kw = 1 + _r(g, D, std=0.2), 1 + _r(g, D, std=0.2)
    table, count = tables(g, cached, page)
    cache = KVCache.empty(count, Hk, page, D, kind)
    for t in cache:
        if t is not None:
            index(t).copy_(torch.randint(1, 100, t.shape, generator=g))
    old = [None if t is None else t.clone() for t in cache]
    lens = torch.tensor(cached, dtype=torch.int32, device=dev)
    cu = ref.cu_of(news, dev) if packed else None
    freq = rope_frequencies(R)
    got = qk_norm_step(q, k, v, cache, table.to(dev), lens, qw, kw, freq, cu_seqlens=cu, eps=EPS, interleaved=interleaved)
    pos = torch.tensor(sum(aref.positions(cached, news), []))
    seq = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news))
    d64 = lambda t: t.double().cpu().flatten(0, 1)  # noqa: E731
    ref.check("q", got, aref.norm_rope(d64(q), qw.double().cpu(), pos, aref.inv_freq(R), EPS, interleaved).reshape(q.shape), dtype, WORK)
    there = pos >= 0
    pages, slots = table[seq[there], pos[there] // page].long(), pos[there] % page
    for name, rows in (("k", aref.norm_rope(d64(k), kw.double().cpu(), pos, aref.inv_freq(R), EPS, interleaved)), ("v", d64(v))):
        rows = rows[there]
        store, before = getattr(cache, name).cpu(), old["kv".index(name)].cpu()
        now = index(store)[pages, :, slots]
        if kind != E4M3:
            ref.check(name, now, rows, dtype, WORK)
        else:
            unit = index(cache[2 + "kv".index(name)].cpu())[pages, :, slots].view(E8M0).double()
            top = rows.abs().amax(-1)
            assert bool((top <= 448 * unit * (1 + WORK)).all()) and bool((top > 224 * unit * (1 - WORK)).all())
            off = (now.view(E4M3).double() * unit[..., None] - rows).abs()
            assert bool((off <= 2.0 ** -4 * rows.abs() * (1 + WORK) + (2.0 ** -10 + WORK * 448) * unit[..., None]).all())
        index(store)[pages, :, slots] = index(before)[pages, :, slots]
        assert torch.equal(index(store), index(before)), "other places were written"
    if kind == E4M3:
        for t, before in zip(cache[2:], old[2:]):
            t, before = index(t.cpu()), index(before.cpu())
            t[pages, :, slots] = before[pages, :, slots]
            assert torch.equal(t, before)


@pytest.mark.parametrize("kind", [BF, E4M3])
def test_step_is_forward_and_write(kind):
    """The same bits as qk_norm_fwd followed by kv_cache_write, where k is rounded to its type once in between only for a
    cache of that type."""
    g = torch.Generator().manual_seed(7)
    q, k, v, w = _r(g, 5, 1, 8, 128, dt=BF), _r(g, 5, 1, 2, 128, dt=BF), _r(g, 5, 1, 2, 128, dt=BF), 1 + _r(g, 128, std=0.2)
    cached = [1, 17, 0, 33, 128]
    table, count = tables(g, cached, 32)
    lens, pos = torch.tensor(cached, dtype=torch.int32, device=dev), torch.tensor(cached, dtype=torch.int32, device=dev)[:, None] - 1
    freq = rope_frequencies(128)
    a, b = KVCache.empty(count, 2, 32, 128, kind), KVCache.empty(count, 2, 32, 128, kind)
    qa = qk_norm_step(q, k, v, a, table.to(dev), lens, w, w, freq)
    qb, kb = qk_norm_fwd(q, k, w, w, freq, positions=pos.contiguous())
    kv_cache_write(kb, v, b, table.to(dev), lens)
    assert torch.equal(qa, qb) and torch.equal(index(a.v), index(b.v))
    if kind == BF:
        assert torch.equal(a.k, b.k)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hk", [(5, 1), (3, 2), (8, 4)])
@pytest.mark.parametrize("D", [16, 64, 128, 256, 37])
def test_gradient_without_eps(dtype, D, Hq, Hk):
    """eps 0, with heads that do and do not fill a warp's groups of rows."""
    g = torch.Generator().manual_seed(12)
    q, k, qw, kw, _, pos = _case(g, [7, 7, 7], False, Hq, Hk, D, dtype, "qk")
    R = D // 4 * 2
    v = ref.leaves(dict(q=q, k=k, qw=qw, kw=kw))
    y = [aref.norm_rope(v[x].flatten(0, 1), v[x + "w"], pos, aref.inv_freq(R), 0.0, False) for x in "qk"]
    for name, o, w in zip("qk", qk_norm_fwd(q, k, qw, kw, rope_frequencies(R), eps=0.0), y):
        ref.check(name, o, w.reshape(o.shape), dtype, WORK)
    dq, dk = _r(g, *q.shape, dt=dtype), _r(g, *k.shape, dt=dtype)
    want = ref.grads(y, (dq.flatten(0, 1), dk.flatten(0, 1)), v)
    got = qk_norm_bwd(q, k, qw, kw, rope_frequencies(R), dq, dk, eps=0.0)
    for name, o, key, dt, tol in zip(("dq", "dk", "dqw", "dkw"), got, ("q", "k", "qw", "kw"), (dtype, dtype, F32, F32),
                                     (WORK, WORK, SUMS, SUMS)):
        ref.check(name, o, want[key], dt, tol)
