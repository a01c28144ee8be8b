"""The selective state space scan on the GPU against its 64-bit definition (mixer_reference).

Tolerances: a result is rounded once to its type. Before that, one step of the recurrence
rounds its decay's exponent (twice), the exponential (2^-22), the two products and the sum: below
2^-20 relative together, and a step size of bf16 inputs is computed within 2^-20. Such errors
of the steps that a state remembers are independent; the states here remember up to about 1000
steps (delta A as small as 1e-3), but at most the sequence: 2^-20 sqrt(steps) with the sequences'
300 tokens is 2^-16 rounded up, used for all outputs. Gradients pass through two such sums: twice that.
"""

from __future__ import annotations

import pytest
import torch

import mixer_reference as ref
from chunkwise_gated_linear_gb300 import kda, mixer, selective_scan_bwd, selective_scan_fwd, selective_scan_step

pytestmark = pytest.mark.gpu
WORK, WORK_GRAD = 2.0 ** -16, 2.0 ** -15
BF, F32 = torch.bfloat16, torch.float32
dev = "cuda"


def _make(lens, ch, N, G, dtype, seed, D=True, z=True, bias=True, h0=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(dev)  # noqa: E731
    rows, ns = sum(lens), len(lens)
    return dict(u=r(rows, ch), dt=r(rows, ch), A=-(torch.rand(ch, N, generator=g) * 8 + 0.05).to(dev),
                B=r(rows, G, N), C=r(rows, G, N), D=r(ch, dt=F32) if D else None, z=r(rows, ch) if z else None,
                bias=(torch.randn(ch, generator=g) - 3).to(dev) if bias else None,
                h0=r(ns, ch, N, dt=F32) if h0 else None, dy=r(rows, ch), dht=r(ns, ch, N, dt=F32))


def _reference(t, lens, softplus=True):
    v = ref.leaves({k: t[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "bias", "h0")})
    y, ht = ref.scan(*(v[k] for k in ("u", "dt", "A", "B", "C", "D", "z", "bias")), softplus, v["h0"], lens)
    return y, ht, v


def _args(t, lens, packed):
    lead = lambda x: None if x is None else (x.unsqueeze(0) if packed else x.reshape(len(lens), lens[0], *x.shape[1:]))  # noqa: E731
    a = [lead(t["u"]), lead(t["dt"]), t["A"], lead(t["B"]), lead(t["C"])]
    return a, lead(t["dy"]), [t["D"], lead(t["z"])], dict(dt_bias=t["bias"], h0=t["h0"], cu_seqlens=ref.cu_of(lens, dev) if packed else None)


RAGGED = [0, 1, 2, 0, 31, 32, 33, 95, 0, 1, 70, 0]


def _forward(t, lens, packed, dtype, softplus=True):
    y_r, ht_r, _ = _reference(t, lens, softplus)
    a, _, dz, kw = _args(t, lens, packed)
    y, ht = selective_scan_fwd(*a, *dz, dt_softplus=softplus, **kw)
    ref.check("y", y, y_r, dtype, WORK)
    ref.check("ht", ht, ht_r, F32, WORK)
    assert kda.kda_get_device_error(0) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 5, 8, 16, 31, 64])
@pytest.mark.parametrize("ch,G", [(64, 1), (150, 3), (7, 1), (21, 3)])
def test_forward(dtype, N, ch, G):
    for lens, packed in ((RAGGED, True), ([41, 41], False), ([300], False), ([1, 1, 1], False)):
        _forward(_make(lens, ch, N, G, dtype, seed=N + ch), lens, packed, dtype)


def test_forward_many_channels_one_block_per_sequence():
    lens = [70, 70]
    _forward(_make(lens, 5000, 16, 1, BF, 1), lens, False, BF)
    lens = [1, 0, 3, 2, 1, 4, 0]  # a few tokens per sequence: one block each as well
    _forward(_make(lens, 96, 16, 2, BF, 2), lens, True, BF)


@pytest.mark.parametrize("off", [("D",), ("z",), ("bias",), ("h0",), ("D", "z", "bias", "h0")])
def test_optional_arguments(off):
    lens = [70, 3, 90]
    t = _make(lens, 72, 16, 1, F32, 3, **{k: k not in off for k in ("D", "z", "bias", "h0")})
    _forward(t, lens, True, F32)
    _backward(t, lens, True, F32)


def test_without_softplus():
    lens = [50, 60]
    t = _make(lens, 72, 16, 1, F32, 4)
    t["dt"] = t["dt"].abs() * 0.1
    t["bias"] = t["bias"].abs() * 0.01
    _forward(t, lens, True, F32, softplus=False)
    _backward(t, lens, True, F32, softplus=False)


def _backward(t, lens, packed, dtype, softplus=True):
    y_r, ht_r, v = _reference(t, lens, softplus)
    g_r = ref.grads((y_r, ht_r), (t["dy"], t["dht"]), v)
    a, dy, dz, kw = _args(t, lens, packed)
    names = ("u", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    got = dict(zip(names, selective_scan_bwd(*a, dy, *dz, dht=t["dht"], dt_softplus=softplus, **kw)))
    for k in names:
        if t[k] is None:
            assert got[k] is None or k == "h0"
        else:
            ref.check("d" + k, got[k], g_r[k], dtype if k in ("u", "dt", "B", "C", "z") else F32, WORK_GRAD)
    assert kda.kda_get_device_error(0) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [1, 5, 8, 16, 31, 64])
@pytest.mark.parametrize("ch,G", [(64, 1), (150, 3), (7, 1), (21, 3)])
def test_backward(dtype, N, ch, G):
    for lens, packed in ((RAGGED, True), ([41, 41], False), ([200], False), ([1, 1], False)):
        _backward(_make(lens, ch, N, G, dtype, seed=N + ch), lens, packed, dtype)


def test_backward_chunks_of_several_windows():
    """Many channels: fewer chunks than windows, so that a window's state is a local one corrected
    by its chunk's start state."""
    lens = [100, 1, 155, 300]
    _backward(_make(lens, 4096, 4, 1, F32, 6), lens, True, F32)


def test_gradient_against_differences():
    """<gradient, direction> against central differences of the 64-bit forward pass (whose error, 1e-4
    squared times third derivatives of size one, is far below the tolerance)."""
    lens = [40, 0, 37]
    t = _make(lens, 20, 16, 2, F32, 8)
    a, dy, dz, kw = _args(t, lens, True)
    names = ("u", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    got = dict(zip(names, selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)))
    g = torch.Generator().manual_seed(1)
    for k in names:
        way = torch.randn(t[k].shape, generator=g, dtype=torch.float64)

        def loss(eps):
            v = {q: None if t[q] is None else t[q].double().cpu() for q in names}
            v[k] = v[k] + eps * way
            y, ht = ref.scan(*(v[q] for q in names[:8]), True, v["h0"], lens)
            return float((y * t["dy"].double().cpu()).sum() + (ht * t["dht"].double().cpu()).sum())

        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        have = float((got[k].double().cpu().reshape(way.shape) * way).sum())
        size = float(got[k].double().norm() * way.norm())
        assert abs(want - have) <= (WORK_GRAD + 1e-6) * size, (k, want, have)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [3, 16, 40])
def test_steps_continue_a_prompt(dtype, N):
    lens = [9, 9, 9]
    t = _make(lens, 70, N, 2, dtype, 11)
    a, _, (D, z), kw = _args(t, lens, False)
    y_r, ht_r, _ = _reference(t, lens)
    h = t["h0"].clone()
    parts = []
    for i, n in ((0, 1), (1, 1), (2, 5), (7, 1), (8, 1)):
        u, dt, A, B, C = (x if x is t["A"] else x[:, i:i + n].contiguous() for x in a)
        parts.append(selective_scan_step(u, dt, A, B, C, h, D, z[:, i:i + n].contiguous(), dt_bias=t["bias"]))
    ref.check("y", torch.cat(parts, 1), y_r, dtype, WORK)
    ref.check("h", h, ht_r, F32, WORK)


def test_strided_inputs():
    """u, dt, z, B, C as slices of one wide projection, aligned and not."""
    for off in (0, 3):
        lens, ch, N = [45, 45], 48, 16
        t = _make(lens, ch, N, 1, BF, 12)
        a, dy, (D, z), kw = _args(t, lens, False)
        sizes = [ch, ch, ch, N, N]
        wide = torch.full((2, 45, sum(sizes) + 8), float("nan"), dtype=BF, device=dev)
        parts = list(wide[:, :, off:off + sum(sizes)].split(sizes, dim=2))
        for part, x in zip(parts, (a[0], a[1], z, a[3], a[4])):
            part.copy_(x.reshape(part.shape))
        u, dt, zs = parts[:3]
        B, C = parts[3].unflatten(2, (1, N)), parts[4].unflatten(2, (1, N))
        y, ht = selective_scan_fwd(*a, D, z, **kw)
        y2, ht2 = selective_scan_fwd(u, dt, t["A"], B, C, D, zs, **kw)
        assert torch.equal(y, y2) and torch.equal(ht, ht2)
        g1 = selective_scan_bwd(*a, dy, D, z, dht=t["dht"], **kw)
        g2 = selective_scan_bwd(u, dt, t["A"], B, C, dy, D, zs, dht=t["dht"], **kw)
        for p, q in zip(g1, g2):
            assert torch.equal(p, q)


def test_extreme_values():
    """Step sizes of zero and of hundreds, decays that underflow, and A = 0: the states are kept, or
    forgotten at once, without NaN; the last sequence holds an infinity that stays in it."""
    lens = [40, 33, 20]
    t = _make(lens, 64, 16, 1, F32, 13)
    t["A"][0] = 0.0
    t["A"][1] = -1e4
    t["dt"][:, 2] = -200.0   # softplus underflows to zero
    t["dt"][:, 3] = 300.0
    t["z"][:, 4] = -200.0
    t["z"][:, 5] = 200.0
    t["u"][:, 6] = 1e18
    y_r, ht_r, v = _reference(t, lens)
    a, dy, dz, kw = _args(t, lens, True)
    y, ht = selective_scan_fwd(*a, *dz, **kw)
    for c in range(64):  # channel by channel: their sizes differ by 1e18
        ref.check(f"y {c}", y[0, :, c], y_r[:, c], F32, WORK)
        ref.check(f"ht {c}", ht[:, c], ht_r[:, c], F32, WORK)
    t["u"][:, 6] = 1.0
    t["A"][1] = -20.0
    _backward(t, lens, True, F32)
    t["u"][-1, 7] = float("inf")
    a, dy, dz, kw = _args(t, lens, True)
    y, ht = selective_scan_fwd(*a, *dz, **kw)
    assert bool(torch.isfinite(y[0, :73]).all()) and bool(torch.isfinite(ht[:2]).all())
    assert not bool(torch.isfinite(ht[2, 7]).all())
    got = selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)
    assert bool(torch.isfinite(got[0][0, :73]).all()) and bool(torch.isfinite(got[3][0, :73]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_tokens(dtype):
    """Tokens masked by a step size of the type's lowest value or minus infinity: the state passes over
    them unchanged, and their gradients are zero (dD and dz see u and z of the token itself)."""
    lens = [70, 40]
    t = _make(lens, 48, 16, 1, dtype, 18)
    off = torch.zeros(sum(lens), dtype=torch.bool, device=dev)
    off[[0, 1, 33, 34, 35, 69, 75]] = True
    off[90:110] = True  # to the end of the sequence
    t["dt"][off] = torch.finfo(dtype).min
    t["dt"][35] = t["dt"][100] = float("-inf")
    a, dy, dz, kw = _args(t, lens, True)
    y, ht = selective_scan_fwd(*a, *dz, **kw)
    # the same sequences without those tokens
    keep = ~off
    short = {k: (v[keep] if k in ("u", "dt", "B", "C", "z", "dy") else v) for k, v in t.items()}
    l2 = [int(keep[:70].sum()), int(keep[70:].sum())]
    a2, dy2, dz2, kw2 = _args(short, l2, True)
    y2, ht2 = selective_scan_fwd(*a2, *dz2, **kw2)
    ref.check("ht", ht, ht2.double().cpu(), F32, WORK)
    ref.check("y", y[:, keep], y2.double().cpu(), dtype, WORK + 2.0 ** -8 * (dtype == BF))
    t["dy"][off] = 0
    got = selective_scan_bwd(*a, t["dy"][None], *dz, dht=t["dht"], **kw)
    want = selective_scan_bwd(*a2, dy2, *dz2, dht=t["dht"], **kw2)
    for i, (p, q) in enumerate(zip(got, want)):
        if i in (0, 1, 3, 4, 6):
            assert not bool(p[:, off].any())
            p = p[:, keep]
        ref.check(f"gradient {i}", p, q.double().cpu(), p.dtype, WORK_GRAD + ref.HALF[p.dtype])
    # nothing but masked tokens: the states are kept bit for bit, in one pass, in chunks and in steps
    t["dt"].fill_(float("-inf"))
    a, dy, dz, kw = _args(t, lens, True)
    assert torch.equal(selective_scan_fwd(*a, *dz, **kw)[1], t["h0"])
    for n in (1, 2):
        u = t["u"][None, :n]
        h = t["h0"][:1].clone()
        selective_scan_step(u, t["dt"][None, :n], t["A"], t["B"][None, :n], t["C"][None, :n], h, dt_bias=t["bias"])
        assert torch.equal(h, t["h0"][:1])


def test_no_tokens():
    t = _make([0, 0, 0], 24, 16, 1, BF, 14)
    for packed in (False, True):
        a, dy, dz, kw = _args(t, [0, 0, 0], packed)
        y, ht = selective_scan_fwd(*a, *dz, **kw)
        assert y.numel() == 0 and torch.equal(ht, t["h0"])
        got = selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)
        assert torch.equal(got[8], t["dht"]) and not got[2].any() and not got[5].any() and not got[7].any()


@pytest.mark.parametrize("cu", [[0, 90, 40, 120], [0, 40, 90, 400], [-3, 40, 90, 120], [0, 40, 90, 110], [2, 40, 90, 120]])
def test_malformed_offsets_raise_the_error_word(cu):
    t = _make([40, 50, 30], 24, 16, 1, BF, 15)
    a, dy, dz, kw = _args(t, [40, 50, 30], True)
    kw["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    selective_scan_fwd(*a, *dz, **kw)
    assert kda.kda_get_device_error(0) == kda.KDA_DEVICE_ERR_SEQLENS
    selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)
    assert kda.kda_get_device_error(0) == kda.KDA_DEVICE_ERR_SEQLENS
    assert kda.kda_get_device_error(0) == 0


def test_repeats_bitwise_and_in_a_graph_on_another_stream():
    lens = [300, 0, 41, 1, 258]
    t = _make(lens, 264, 16, 1, BF, 16)
    a, dy, dz, kw = _args(t, lens, True)
    run = lambda **s: (*selective_scan_fwd(*a, *dz, **kw, **s), *selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw, **s))  # noqa: E731
    first = run()
    for p, q in zip(first, run()):
        assert torch.equal(p, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for o in got:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for p, q in zip(first, got):
        assert torch.equal(p, q)
    s = torch.cuda.Stream()
    got = run(stream=s.cuda_stream)  # the library's own scratch
    torch.cuda.synchronize()
    for p, q in zip(first, got):
        assert torch.equal(p, q)


def test_workspace_is_what_the_size_says():
    """A given workspace of exactly the stated bytes, bytes past it untouched."""
    lens = [130, 200]
    t = _make(lens, 72, 16, 1, BF, 17)
    a, dy, dz, kw = _args(t, lens, True)
    want = selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)
    f, ns = mixer._scan_params(*a, *dz, t["bias"], True, t["h0"], kw["cu_seqlens"], None, None)
    outs = [torch.empty_like(o) for o in want]
    p = mixer.kda_scan_bwd_params(f, dy.data_ptr(), t["dht"].data_ptr(), *(o.data_ptr() for o in outs), None, 0)
    n = mixer.kda_scan_bwd_workspace(p)
    ws = torch.full((n + 1024,), 0x5A, dtype=torch.uint8, device=dev)
    p.workspace, p.workspace_bytes = ws.data_ptr(), n
    assert mixer.kda_scan_bwd(p, torch.cuda.current_stream().cuda_stream) == kda.KDA_OK
    torch.cuda.synchronize()
    assert bool((ws[n:] == 0x5A).all())
    for x, y in zip(want, outs):
        assert torch.equal(x, y)


def test_agrees_with_the_decay_only_recurrence():
    """With A the same for all channels and one step size per token, the scan is the decay-only
    recurrence of the framework (one gate per head, keys B, queries C, values delta u)."""
    from chunkwise_gated_linear_gb300 import chunk_kda_fwd

    T, ch, N = 150, 64, 64
    g = torch.Generator().manual_seed(20)
    u = torch.randn(1, T, ch, generator=g).to(dev)
    delta = (torch.rand(1, T, 1, generator=g) * 0.05 + 0.01).to(dev)
    A = -torch.ones(ch, N, device=dev)
    B, C = (torch.randn(1, T, 1, N, generator=g).to(dev) for _ in range(2))
    y, ht = selective_scan_fwd(u, delta.expand(1, T, ch).contiguous(), A, B, C, dt_softplus=False)
    o, h = chunk_kda_fwd(C, B, (delta * u).unsqueeze(2).contiguous(), (-delta).contiguous(), None, scale=1.0)
    assert ref.rel(y, o.double().cpu()[:, :, 0]) < 1e-5 and ref.rel(ht, h.double().cpu()[:, 0].transpose(1, 2)) < 1e-5


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("what", ["u", "dt", "B", "C", "z", "dy", "h0", "dht"])
@pytest.mark.parametrize("dtype,N", [(BF, 16), (F32, 5), (F32, 40)])
def test_nonfinite_values_stay_in_their_sequence(dtype, N, what, value):
    """Values that are not finite in one sequence leave the outputs and gradients of the others as
    they are, bit for bit: packed (the sequence before it runs over several chunks and ends in
    the same chunk as the bad one and the start of the next) and in a batch."""
    for lens, packed in (([100, 10, 60, 40], True), ([41, 41, 41], False)):
        t = _make(lens, 64, N, 1, dtype, 21)
        run = lambda: [selective_scan_fwd(*a, *dz, **kw), selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)]  # noqa: E731
        a, dy, dz, kw = _args(t, lens, packed)
        clean = run()
        t = dict(t, **{what: t[what].clone()})
        first, last = lens[0], lens[0] + lens[1]
        t[what][1 if what in ("h0", "dht") else slice(first + 3, first + 5)] = value
        a, dy, dz, kw = _args(t, lens, packed)
        bad = run()
        rows = torch.ones(sum(lens), dtype=torch.bool, device=dev)
        rows[first:last] = False
        seqs = torch.tensor([True, False] + [True] * (len(lens) - 2), device=dev)
        (y, ht), (du, ddt, _, dB, dC, _, dzg, _, dh0) = (tuple(zip(p, q)) for p, q in zip(clean, bad))
        for name, (p, q) in dict(y=y, du=du, ddt=ddt, dB=dB, dC=dC, dz=dzg).items():
            p, q = (x.reshape(sum(lens), -1)[rows] for x in (p, q))
            assert torch.equal(p, q), (name, packed)
        for name, (p, q) in dict(ht=ht, dh0=dh0).items():
            assert torch.equal(p[seqs], q[seqs]), (name, packed)


# The sizes below follow from the GPU's SMs, so that the kernels' loops take more than one turn. Their
# sequences are longer than the 300 tokens of the tolerances above; the states still remember about 1000
# steps, whose independent errors of 2^-20 add up to 2^-15, and to twice that in gradients.
LONG, LONG_GRAD = 2.0 ** -15, 2.0 ** -14


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype,ch,N,G", [(BF, 256, 16, 1), (F32, 256, 16, 1), (BF, 512, 8, 2), (F32, 300, 5, 3), (BF, 256, 32, 1),
                                          (F32, 256, 64, 1), (BF, 90, 40, 2)])
@pytest.mark.parametrize("T", [1, 2])
def test_steps_of_more_sequences_than_blocks(dtype, ch, N, G, T):
    """A block of 256 channels takes several sequences one after another, the next one's states and inputs
    on their way meanwhile: here three, two for the last blocks."""
    per = 2 * _sms() // -(-ch // 256)
    n = 3 * per - per // 2
    t = _make([T] * n, ch, N, G, dtype, 22)
    v = {k: None if x is None else x.double().cpu() for k, x in t.items()}
    ch_of = torch.arange(ch) // (ch // G)
    rows = lambda x: x.reshape(n, T, *x.shape[1:])  # noqa: E731
    h, ys = v["h0"], []
    for i in range(T):  # all sequences at once
        u, dt, B, C, z = (rows(v[k])[:, i] for k in ("u", "dt", "B", "C", "z"))
        delta = torch.nn.functional.softplus(dt + v["bias"], threshold=50.0)
        h = torch.exp(delta[..., None] * v["A"]) * h + (delta * u)[..., None] * B[:, ch_of]
        ys.append(((h * C[:, ch_of]).sum(-1) + v["D"] * u) * ref.act(z, "silu"))
    h_r = t["h0"].clone()
    a = [rows(t["u"]), rows(t["dt"]), t["A"], rows(t["B"]), rows(t["C"])]
    y = selective_scan_step(*a, h_r, t["D"], rows(t["z"]), dt_bias=t["bias"])
    for name, got, want, dt in (("y", y, torch.stack(ys, 1), dtype), ("h", h_r, h, F32)):
        ref.check(name, got, want, dt, WORK)
        for s in (0, per - 1, per, 2 * per - 1, 2 * per, n - 1):  # first and last of each turn
            ref.check(f"{name} {s}", got[s], want[s], dt, WORK)


@pytest.mark.parametrize("dtype,N", [(BF, 16), (F32, 16), (F32, 20)])
def test_forward_one_block_per_sequence(dtype, N):
    """Enough blocks of channels and sequences for three per SM, and more than 64 tokens: no chunks."""
    G = 64  # a block of channels holds one group
    n = -(-3 * _sms() // G)
    _forward(_make([70] * n, 4 * G, N, G, dtype, 23), [70] * n, False, dtype)


def _on_gpu(t, lens):
    """Outputs and gradients of the 64-bit definition, computed on the GPU (many channels and tokens)."""
    names = ("u", "dt", "A", "B", "C", "D", "z", "bias", "h0")
    v = {k: t[k].double().requires_grad_() for k in names}
    y, ht = ref.scan(*(v[k] for k in names[:8]), True, v["h0"], lens)
    g = torch.autograd.grad((y * t["dy"].double()).sum() + (ht * t["dht"].double()).sum(), [v[k] for k in names])
    return y.detach().cpu(), ht.detach().cpu(), {k: x.cpu() for k, x in zip(names, g)}


def _both(t, lens, dtype):
    y_r, ht_r, g_r = _on_gpu(t, lens)
    a, dy, dz, kw = _args(t, lens, True)
    y, ht = selective_scan_fwd(*a, *dz, **kw)
    ref.check("y", y, y_r, dtype, LONG)
    ref.check("ht", ht, ht_r, F32, LONG)
    got = selective_scan_bwd(*a, dy, *dz, dht=t["dht"], **kw)
    for k, o in zip(("u", "dt", "A", "B", "C", "D", "z", "bias", "h0"), got):
        ref.check("d" + k, o, g_r[k], dtype if k in ("u", "dt", "B", "C", "z") else F32, LONG_GRAD)
    assert kda.kda_get_device_error(0) == 0


@pytest.mark.parametrize("dtype,N", [(BF, 10), (F32, 3)])
def test_chunks_of_several_tiles(dtype, N):
    """Chunks of more than 64 rows in both passes, so that B and C come in several tiles of 32 tokens, with
    sequences that start, end and cross inside them."""
    ch = 64 * _sms()
    rows = 70 * 32  # gradient: blocks of 64 channels, 32 chunks; forward: of 256 channels, 16 chunks
    lens = [0, 300, 1, 33, 700, 0, 150]
    _both(_make([*lens, rows - sum(lens)], ch, N, 1, dtype, 24), [*lens, rows - sum(lens)], dtype)


@pytest.mark.parametrize("dtype,N,ch", [(BF, 16, 6), (F32, 2, 5)])
def test_more_than_256_chunks(dtype, N, ch):
    """Few channels: chunks of 16 rows forward and 32 backward, more than 256 of either, so that the carries
    look up where sequences start and end more than once. A sequence crosses each of those places."""
    lens = [4000, 0, 37, 4500, 1, 500]
    t = _make(lens, ch, N, 1, dtype, 25)
    _both(t, lens, dtype)
