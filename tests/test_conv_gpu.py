"""The short causal convolution on the GPU against its 64-bit definition (mixer_reference).

Tolerances: an output is rounded once (half a step of its type); before that, W products and
their sum, bias, and for SiLU an exponential and a reciprocal, each within 2^-21: 2^-18 in all
is allowed. Weight gradients are sums over up to 600 tokens in 32 bits, whose rounding errors
are independent: sqrt(600) 2^-24 of the terms' size, again below 2^-18.
"""

from __future__ import annotations

import pytest
import torch

import mixer_reference as ref
from chunkwise_gated_linear_gb300 import causal_conv_bwd, causal_conv_fwd, causal_conv_step, kda

pytestmark = pytest.mark.gpu
WORK = 2.0 ** -18
BF, F32 = torch.bfloat16, torch.float32
dev = "cuda"


def _make(lens, D, W, dtype, seed, state=True, bias=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g).to(dt).to(dev)  # noqa: E731
    rows, N = sum(lens), len(lens)
    return dict(x=r(rows, D), w=r(D, W, dt=F32), b=r(D, dt=F32) if bias else None, s0=r(N, W - 1, D) if state else None,
                dy=r(rows, D), dst=r(N, W - 1, D))


def _reference(t, lens, act):
    v = ref.leaves({k: t[k] for k in ("x", "w", "b", "s0")})
    y, st = ref.conv(v["x"], v["w"], v["b"], v["s0"], lens, act)
    return y, st, ref.grads((y, st), (t["dy"], t["dst"]), v)


def _lead(t, lens, packed):
    return t.unsqueeze(0) if packed else t.reshape(len(lens), lens[0], -1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("D", [8, 129, 520])
@pytest.mark.parametrize("act", ["silu", None])
def test_forward_and_backward(dtype, W, D, act):
    # packed: sequences shorter than the window, empty ones at both ends, tiles that several share
    for lens, packed in (([0, 1, 2, 3, 0, 4, 5, 70, 0, 1, 33, 131, 0], True), ([37, 37, 37], False), ([1], False)):
        t = _make(lens, D, W, dtype, seed=D + W)
        y_r, st_r, g_r = _reference(t, lens, act)
        cu = ref.cu_of(lens, dev) if packed else None
        x, dy = _lead(t["x"], lens, packed), _lead(t["dy"], lens, packed)
        y, st = causal_conv_fwd(x, t["w"], t["b"], s0=t["s0"], activation=act, cu_seqlens=cu, output_final_state=True)
        ref.check("y", y, y_r, dtype, WORK)
        assert torch.equal(st.double().cpu(), st_r.detach())  # copies of inputs
        dx, dw, db, ds0 = causal_conv_bwd(x, t["w"], t["b"], dy, s0=t["s0"], dst=t["dst"], activation=act, cu_seqlens=cu)
        ref.check("dx", dx, g_r["x"], dtype, WORK)
        ref.check("dw", dw, g_r["w"], F32, WORK)
        ref.check("db", db, g_r["b"], F32, WORK)
        ref.check("ds0", ds0, g_r["s0"], dtype, WORK)
        assert kda.kda_get_device_error(0) == 0


def test_optional_arguments():
    lens = [20, 20]
    t = _make(lens, 48, 4, F32, 3, state=False, bias=False)
    y_r, st_r, g_r = _reference(t, lens, "silu")
    x, dy = _lead(t["x"], lens, False), _lead(t["dy"], lens, False)
    y, st = causal_conv_fwd(x, t["w"])
    assert st is None
    ref.check("y", y, y_r, F32, WORK)
    dx, dw, db, ds0 = causal_conv_bwd(x, t["w"], None, dy, dst=t["dst"], want_ds0=False)
    assert db is None and ds0 is None
    ref.check("dx", dx, g_r["x"], F32, WORK)
    ref.check("dw", dw, g_r["w"], F32, WORK)
    # no gradient of the final state; the gradient at zero states
    t["dst"] = torch.zeros_like(t["dst"])
    t["s0"] = torch.zeros_like(t["dst"])
    g_r = _reference(t, lens, "silu")[2]
    dx, dw, db, ds0 = causal_conv_bwd(x, t["w"], None, dy)
    ref.check("dx", dx, g_r["x"], F32, WORK)
    ref.check("ds0", ds0, g_r["s0"], F32, WORK)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("off,width", [(16, 96), (3, 77)])
def test_strided_input(dtype, off, width):
    """x as a slice of a wider tensor, aligned and not: the same values as its copy, bitwise where
    the same path runs and within a rounding of the products' order (none here) otherwise."""
    lens, D = [19, 19], 32
    t = _make(lens, D, 4, dtype, 5)
    wide = torch.full((2, 19, width), float("nan"), dtype=dtype, device=dev)
    wide[:, :, off:off + D] = _lead(t["x"], lens, False)
    x = wide[:, :, off:off + D]
    y, st = causal_conv_fwd(x, t["w"], t["b"], s0=t["s0"], output_final_state=True)
    y2, st2 = causal_conv_fwd(x.contiguous(), t["w"], t["b"], s0=t["s0"], output_final_state=True)
    assert torch.equal(y, y2) and torch.equal(st, st2)
    dy = _lead(t["dy"], lens, False)
    for a, b in zip(causal_conv_bwd(x, t["w"], t["b"], dy, s0=t["s0"]), causal_conv_bwd(x.contiguous(), t["w"], t["b"], dy, s0=t["s0"])):
        ref.check("grad", a, b.double().cpu(), a.dtype, WORK)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("W", [2, 4])
def test_steps_continue_a_prompt(dtype, W):
    lens, D = [9, 9, 9], 40
    t = _make(lens, D, W, dtype, 7)
    x = _lead(t["x"], lens, False)
    y, st = causal_conv_fwd(x, t["w"], t["b"], s0=t["s0"], output_final_state=True)
    state = t["s0"].clone()
    parts = [causal_conv_step(x[:, i:i + n].contiguous(), state, t["w"], t["b"]) for i, n in ((0, 1), (1, 1), (2, 5), (7, 1), (8, 1))]
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(state, st)
    before = state.clone()
    assert causal_conv_step(x[:, :0], state, t["w"], t["b"]).shape == (3, 0, D)
    assert torch.equal(state, before)


def test_no_tokens():
    w, b, s0 = torch.ones(16, 4, device=dev), torch.ones(16, device=dev), torch.randn(3, 3, 16, device=dev)
    y, st = causal_conv_fwd(torch.empty(3, 0, 16, device=dev), w, b, s0=s0, output_final_state=True)
    assert y.numel() == 0 and torch.equal(st, s0)
    cu = torch.zeros(4, dtype=torch.int32, device=dev)
    x = torch.empty(1, 0, 16, device=dev)
    y, st = causal_conv_fwd(x, w, b, s0=s0, cu_seqlens=cu, output_final_state=True)
    assert torch.equal(st, s0)
    dx, dw, db, ds0 = causal_conv_bwd(x, w, b, x, s0=s0, dst=s0, cu_seqlens=cu)
    assert torch.equal(ds0, s0) and not dw.any() and not db.any()


def test_infinities_stay_in_their_sequence_and_channel():
    lens = [5, 6]
    t = _make(lens, 16, 4, F32, 9)
    clean = causal_conv_fwd(t["x"][None], t["w"], t["b"], s0=t["s0"], cu_seqlens=ref.cu_of(lens, dev))[0]
    t["x"][4, 3] = float("inf")
    t["x"][2, 5] = float("nan")
    y = causal_conv_fwd(t["x"][None], t["w"], t["b"], s0=t["s0"], cu_seqlens=ref.cu_of(lens, dev))[0]
    assert torch.equal(y[:, 5:], clean[:, 5:])
    keep = torch.ones(16, dtype=torch.bool, device=dev)
    keep[3] = keep[5] = False
    assert torch.equal(y[:, :, keep], clean[:, :, keep])


@pytest.mark.parametrize("cu", [[0, 9, 4, 12], [0, 4, 9, 40], [-3, 4, 9, 12], [0, 4, 9, 11], [2, 4, 9, 12]])
def test_malformed_offsets_raise_the_error_word(cu):
    """Every row is still looked up inside the tensors: the call returns, and says so."""
    t = _make([4, 5, 3], 16, 4, BF, 11)
    cu = torch.tensor(cu, dtype=torch.int32, device=dev)
    causal_conv_fwd(t["x"][None], t["w"], t["b"], s0=t["s0"], cu_seqlens=cu, output_final_state=True)
    assert kda.kda_get_device_error(0) == kda.KDA_DEVICE_ERR_SEQLENS
    causal_conv_bwd(t["x"][None], t["w"], t["b"], t["dy"][None], s0=t["s0"], cu_seqlens=cu)
    assert kda.kda_get_device_error(0) == kda.KDA_DEVICE_ERR_SEQLENS
    assert kda.kda_get_device_error(0) == 0


def test_repeats_bitwise_and_in_a_graph_on_another_stream():
    lens = [300, 0, 41, 1, 258]
    t = _make(lens, 264, 4, BF, 13)
    cu = ref.cu_of(lens, dev)
    run = lambda: (*causal_conv_fwd(t["x"][None], t["w"], t["b"], s0=t["s0"], cu_seqlens=cu, output_final_state=True),  # noqa: E731
                   *causal_conv_bwd(t["x"][None], t["w"], t["b"], t["dy"][None], s0=t["s0"], dst=t["dst"], cu_seqlens=cu))
    first = run()
    for a, b in zip(first, run()):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
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
    # a stream given as a handle: the scratch comes from the library's pool
    torch.cuda.synchronize()
    got = causal_conv_bwd(t["x"][None], t["w"], t["b"], t["dy"][None], s0=t["s0"], dst=t["dst"], cu_seqlens=cu, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip(first[2:], got):
        assert torch.equal(a, b)


def test_more_than_2_31_elements():
    rows, D = 263000, 8192
    x = torch.zeros(1, rows, D, dtype=BF, device=dev)
    x[0, -3:] = 1.0
    w = torch.ones(D, 4, device=dev)
    y, st = causal_conv_fwd(x, w, activation=None, output_final_state=True)
    assert rows * D > 2 ** 31
    assert torch.equal(y[0, -4:, ::1000].float().cpu(), torch.tensor([0.0, 1, 2, 3])[:, None].expand(4, 9))
    assert bool((st == 1).all()) and not bool(y[0, :1000].any())
