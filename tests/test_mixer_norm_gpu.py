"""The gated output norm and the block's residual update with its norms, on the GPU against their
64-bit definitions (mixer_reference).

Tolerances: a result is rounded once to its type. A row's sum of squares has up to 8192 terms in
32 bits (added pairwise over threads: below 2^-20), the rest is about ten roundings and an
exponential, and a gradient is a difference of two such terms of at most its own size
on these inputs: 2^-18. Sums over up to 3000 rows: sqrt(3000) 2^-24, below 2^-18.
"""

from __future__ import annotations

import pytest
import torch

import mixer_reference as ref
from chunkwise_gated_linear_gb300 import block_norm_bwd, block_norm_fwd, gated_norm_bwd, gated_norm_fwd

pytestmark = pytest.mark.gpu
WORK = 2.0 ** -18
BF, F32 = torch.bfloat16, torch.float32
dev = "cuda"
EPS = 1e-6


def _r(g, *s, dt=F32, std=1.0):
    return (torch.randn(*s, generator=g) * std).to(dt).to(dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("rows,D", [(1, 64), (33, 64), (100, 128), (7, 200), (50, 256), (3, 1), (5, 37), (9, 1000), (4, 1001),
                                    (6, 1024), (3, 2048), (5, 2047), (3, 4096), (2, 8192), (2, 8191), (3000, 128)])
def test_gated_norm(dtype, act, rows, D):
    g = torch.Generator().manual_seed(D)
    x, z, dy, w = _r(g, rows, D, dt=dtype), _r(g, rows, D, dt=dtype, std=2), _r(g, rows, D, dt=dtype), _r(g, D)
    v = ref.leaves(dict(x=x, z=z, w=w))
    y_r = ref.gated_norm(v["x"], v["z"], v["w"], EPS, act)
    g_r = ref.grads((y_r,), (dy,), v)
    ref.check("y", gated_norm_fwd(x, z, w, eps=EPS, activation=act), y_r, dtype, WORK)
    dx, dz, dw = gated_norm_bwd(x, z, w, dy, eps=EPS, activation=act)
    if D > 1:  # a single channel's norm is its sign: dx is rounding alone
        ref.check("dx", dx, g_r["x"], dtype, WORK)
    ref.check("dz", dz, g_r["z"], dtype, WORK)
    ref.check("dw", dw, g_r["w"], F32, WORK)


@pytest.mark.parametrize("dtype,res", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,D", [(1, 64), (37, 256), (11, 130), (6, 512), (5, 1000), (3, 2048), (3, 4096), (700, 520), (2, 8192),
                                    (2, 8190)])
@pytest.mark.parametrize("parts", ["", "pzs", "p", "z", "s"])
def test_block_norm(dtype, res, rows, D, parts):
    g = torch.Generator().manual_seed(D)
    x, z, r = _r(g, rows, D, dt=dtype), _r(g, rows, D, dt=dtype), _r(g, rows, D, dt=res, std=2)
    w, pw, sc = _r(g, D), _r(g, D), _r(g, D)
    dy, dr = _r(g, rows, D, dt=dtype), _r(g, rows, D, dt=res)
    kw = dict(post_weight=pw if "p" in parts else None, z=z if "z" in parts else None, scale=sc if "s" in parts else None)
    v = ref.leaves(dict(x=x, r=r, w=w, **kw))
    y_r, r_r = ref.block_norm(v["x"], v["r"], v["w"], v["post_weight"], v["z"], v["scale"], EPS, "sigmoid")
    g_r = ref.grads((y_r, r_r), (dy, dr), v)
    y, r2 = block_norm_fwd(x, r, w, eps=EPS, **kw)
    ref.check("y", y, y_r, dtype, WORK)
    ref.check("r", r2, r_r, res, WORK)
    got = block_norm_bwd(x, r, w, dy, dr, eps=EPS, **kw)
    for name, o, key, dt in zip(("dx", "dr", "dw", "dpw", "dz", "dscale"), got, ("x", "r", "w", "post_weight", "z", "scale"),
                                (dtype, res, F32, F32, dtype, F32)):
        if v[key] is None:
            assert o is None
        else:
            ref.check(name, o, g_r[key], dt, WORK)


def test_block_norm_without_gradient_of_the_residual():
    g = torch.Generator().manual_seed(1)
    x, r, w, dy = _r(g, 5, 96), _r(g, 5, 96), _r(g, 96), _r(g, 5, 96)
    a = block_norm_bwd(x, r, w, dy)
    b = block_norm_bwd(x, r, w, dy, torch.zeros_like(r))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF)])
def test_block_norm_in_place(dtype, res):
    g = torch.Generator().manual_seed(2)
    x, r, w = _r(g, 9, 512, dt=dtype), _r(g, 9, 512, dt=res), _r(g, 512)
    y, r2 = block_norm_fwd(x, r, w)
    y3, r3 = block_norm_fwd(x, r, w, new_residual=r)
    assert r3 is r and torch.equal(r, r2) and torch.equal(y, y3)


def test_block_norm_gradient_in_place():
    """kda_block_norm_bwd's dresidual may be dres."""
    from chunkwise_gated_linear_gb300 import kda, mixer

    g = torch.Generator().manual_seed(6)
    x, r, w, dy, dr = _r(g, 9, 320), _r(g, 9, 320), _r(g, 320), _r(g, 9, 320), _r(g, 9, 320)
    want = block_norm_bwd(x, r, w, dy, dr)
    f = mixer._block_norm_params(x, r, w, None, None, None, EPS, "sigmoid", None, None)
    dx, dw, got = torch.empty_like(x), torch.empty_like(w), dr.clone()
    p = mixer.kda_block_norm_bwd_params(f, dy.data_ptr(), got.data_ptr(), dx.data_ptr(), got.data_ptr(), dw.data_ptr(), None, None,
                                        None, None, 0)
    assert mixer.kda_block_norm_bwd(p, torch.cuda.current_stream().cuda_stream) == kda.KDA_OK
    torch.cuda.synchronize()
    assert torch.equal(got, want[1]) and torch.equal(dx, want[0]) and torch.equal(dw, want[2])


def test_rows_of_zeros_and_large_values():
    """A row of zeros (the norm is eps alone) and rows near the type's largest squares stay finite."""
    g = torch.Generator().manual_seed(3)
    x, z, w, dy = _r(g, 6, 128), _r(g, 6, 128), _r(g, 128), _r(g, 6, 128)
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-15
    z[3] = 300.0
    z[4] = -300.0
    v = ref.leaves(dict(x=x, z=z, w=w))
    y_r = ref.gated_norm(v["x"], v["z"], v["w"], EPS, "silu")
    g_r = ref.grads((y_r,), (dy,), v)
    y = gated_norm_fwd(x, z, w)
    dx, dz, dw = gated_norm_bwd(x, z, w, dy)
    for i in range(6):
        ref.check(f"y {i}", y[i], y_r[i], F32, WORK)
        ref.check(f"dz {i}", dz[i], g_r["z"][i], F32, WORK)
    for i in (0, 2, 3):
        ref.check(f"dx {i}", dx[i], g_r["x"][i], F32, WORK)
    assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dw).all())


def test_no_rows():
    w = torch.ones(64, device=dev)
    x = torch.empty(0, 64, device=dev)
    assert gated_norm_fwd(x, x, w).shape == (0, 64)
    dx, dz, dw = gated_norm_bwd(x, x, w, x)
    assert dx.shape == (0, 64) and not dw.any()
    y, r = block_norm_fwd(x, x, w)
    assert y.shape == r.shape == (0, 64)
    assert not block_norm_bwd(x, x, w, x)[2].any()


def test_higher_ranks_and_unaligned_rows():
    g = torch.Generator().manual_seed(4)
    x, z, w = _r(g, 2, 3, 5, 64, dt=BF), _r(g, 2, 3, 5, 64, dt=BF), _r(g, 64)
    y = gated_norm_fwd(x, z, w)
    assert y.shape == x.shape
    # the same rows from memory that starts 2 bytes past a 16-byte boundary
    buf = torch.empty(2 * 3 * 5 * 64 + 1, dtype=BF, device=dev)[1:].view(2, 3, 5, 64)
    buf.copy_(x)
    ref.check("y", gated_norm_fwd(buf, z, w), y.double().cpu(), BF, 2.0 ** -8)


def test_repeats_bitwise_and_in_a_graph():
    g = torch.Generator().manual_seed(5)
    x, z, w, dy = (_r(g, 2000, 128, dt=BF) for _ in range(4))
    w = w[0].float()
    r = _r(g, 300, 2048)
    xb, wb = _r(g, 300, 2048, dt=BF), _r(g, 2048)
    run = lambda **s: (gated_norm_fwd(x, z, w, **s), *gated_norm_bwd(x, z, w, dy, **s), *block_norm_fwd(xb, r, wb, scale=wb, **s),  # noqa: E731
                       *(t for t in block_norm_bwd(xb, r, wb, xb, r, scale=wb, **s) if t is not None))
    first = run()
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for o in got:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a, b)
    got = run(stream=torch.cuda.Stream().cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(first, got):
        assert torch.equal(a, b)


# More rows than one grid covers: a block then takes several row groups, the next one's loads ahead. The
# blocks per SM are at most 4 (gated norm) and 16 (block norm) of 256 threads, of half as many 512. The
# definition runs on the GPU in 64 bits. A block adds at most tens of rows' products to a column, and the
# blocks' sums (below 3000) are added in several lanes: the tolerances above hold.
def _grids(per_sm, D, threads):
    """Rows of two and a half grids, for `threads` per row."""
    blocks = (per_sm if threads <= 256 else (per_sm + 1) // 2) * torch.cuda.get_device_properties(0).multi_processor_count
    return 5 * blocks * max(1, 256 // threads) // 2 + 1


def _on_gpu(seed):
    g = torch.Generator(dev).manual_seed(seed)
    return lambda *s, dt=F32, std=1.0: (torch.randn(*s, generator=g, device=dev) * std).to(dt)


def _gpu_reference(fn, inputs, cotangents):
    v = {k: x.double().requires_grad_() for k, x in inputs.items()}
    outs = fn(v)
    got = torch.autograd.grad(sum((o * c.double()).sum() for o, c in zip(outs, cotangents)), list(v.values()))
    return [o.detach().cpu() for o in outs], {k: x.cpu() for k, x in zip(v, got)}


@pytest.mark.parametrize("dtype,act", [(BF, "silu"), (F32, "sigmoid")])
@pytest.mark.parametrize("D,threads", [(1024, 128), (2048, 256), (1000, 128), (1001, 128), (4096, 512), (6144, 512)])
def test_gated_norm_in_several_turns(dtype, act, D, threads):
    rows, r = _grids(4, D, threads), _on_gpu(D)
    x, z, dy, w = r(rows, D, dt=dtype), r(rows, D, dt=dtype, std=2), r(rows, D, dt=dtype), r(D)
    (y_r,), g_r = _gpu_reference(lambda v: (ref.gated_norm(v["x"], v["z"], v["w"], EPS, act),), dict(x=x, z=z, w=w), (dy,))
    ref.check("y", gated_norm_fwd(x, z, w, eps=EPS, activation=act), y_r, dtype, WORK)
    for name, o, dt in zip("xzw", gated_norm_bwd(x, z, w, dy, eps=EPS, activation=act), (dtype, dtype, F32)):
        ref.check("d" + name, o, g_r[name], dt, WORK)


@pytest.mark.parametrize("dtype,res", [(BF, F32), (BF, BF), (F32, F32)])
@pytest.mark.parametrize("D,threads", [(2048, 256), (2047, 512), (4096, 512), (8192, 512)])
def test_block_norm_in_several_turns(dtype, res, D, threads):
    """In place as well; with a SiLU gate in both passes."""
    rows, rnd = _grids(16, D, threads), _on_gpu(D)
    x, z, r = rnd(rows, D, dt=dtype), rnd(rows, D, dt=dtype), rnd(rows, D, dt=res, std=2)
    w, kw = rnd(D), dict(post_weight=rnd(D), z=z, scale=rnd(D))
    dy, dr = rnd(rows, D, dt=dtype), rnd(rows, D, dt=res)
    (y_r, r_r), g_r = _gpu_reference(
        lambda v: ref.block_norm(v["x"], v["r"], v["w"], v["post_weight"], v["z"], v["scale"], EPS, "silu"),
        dict(x=x, r=r, w=w, **kw), (dy, dr))
    got = block_norm_bwd(x, r, w, dy, dr, eps=EPS, activation="silu", **kw)
    y, r2 = block_norm_fwd(x, r, w, eps=EPS, activation="silu", **kw)
    y3, r3 = block_norm_fwd(x, r, w, eps=EPS, activation="silu", new_residual=r, **kw)
    assert r3 is r and torch.equal(r, r2) and torch.equal(y, y3)
    ref.check("y", y, y_r, dtype, WORK)
    ref.check("r", r2, r_r, res, WORK)
    for name, o, dt in zip(("x", "r", "w", "post_weight", "z", "scale"), got, (dtype, res, F32, F32, dtype, F32)):
        ref.check("d" + name, o, g_r[name], dt, WORK)


@pytest.mark.parametrize("dtype,res", [(BF, F32), (F32, F32)])
@pytest.mark.parametrize("rows,D", [(37, 256), (11, 130), (5, 1000), (3, 4096), (2, 8192), (2, 8190)])
@pytest.mark.parametrize("parts", ["pzs", "z"])
def test_block_norm_with_a_silu_gate(dtype, res, rows, D, parts):
    g = torch.Generator().manual_seed(D + 1)
    x, z, r = _r(g, rows, D, dt=dtype), _r(g, rows, D, dt=dtype, std=2), _r(g, rows, D, dt=res, std=2)
    w, kw = _r(g, D), dict(post_weight=_r(g, D) if "p" in parts else None, scale=_r(g, D) if "s" in parts else None, z=z)
    dy, dr = _r(g, rows, D, dt=dtype), _r(g, rows, D, dt=res)
    v = ref.leaves(dict(x=x, r=r, w=w, **kw))
    y_r, r_r = ref.block_norm(v["x"], v["r"], v["w"], v["post_weight"], v["z"], v["scale"], EPS, "silu")
    g_r = ref.grads((y_r, r_r), (dy, dr), v)
    y, r2 = block_norm_fwd(x, r, w, eps=EPS, activation="silu", **kw)
    ref.check("y", y, y_r, dtype, WORK)
    ref.check("r", r2, r_r, res, WORK)
    got = block_norm_bwd(x, r, w, dy, dr, eps=EPS, activation="silu", **kw)
    for name, o, key, dt in zip(("dx", "dr", "dw", "dpw", "dz", "dscale"), got, ("x", "r", "w", "post_weight", "z", "scale"),
                                (dtype, res, F32, F32, dtype, F32)):
        if v[key] is not None:
            ref.check(name, o, g_r[key], dt, WORK)
