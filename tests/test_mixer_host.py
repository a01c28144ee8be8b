"""The token-mixer operators on the host: exported symbols, refusals before any CUDA call, the
binding's checks, and the 64-bit definitions against finite differences (no GPU)."""

from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

import chunkwise_gated_linear_gb300 as pkg
from chunkwise_gated_linear_gb300 import kda, mixer
import mixer_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an aligned address that is never dereferenced


def _header():
    text = open(os.path.join(ROOT, "include", "kda_mixer.h"), encoding="utf-8").read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(kda_\w+)\s*\(", _header(), flags=re.M))
    assert names == set(mixer.EXPORTED)
    for name in names:
        assert ctypes.cast(getattr(kda.lib(), name), ctypes.c_void_p).value


def test_structs_match_the_header():
    """Field names in the header's order (their types are by name: pointers, sizes, floats)."""
    for name, body in re.findall(r"typedef struct (\w+) \{(.*?)\}", _header(), flags=re.S):
        fields = []
        for line in body.split(";"):
            line = line.replace("const", " ").replace("*", " ").strip()
            if line:
                first, *rest = line.split(None, 1)
                fields += [f.strip() for f in rest[0].split(",")]
        assert [f for f, _ in getattr(mixer, name)._fields_] == fields, name


def _set(p, **over):
    for k, v in over.items():
        at = p
        if not hasattr(p, k):
            at = p.f
        setattr(at, k, v)
    return p


def _conv(**over):
    return _set(mixer.kda_conv_params(A, A, A, A, A, 2 * A, 0, 2, 5, 64, 4, None, 0, 1), **over)


def _conv_bwd(**over):
    return _set(mixer.kda_conv_bwd_params(A, A, A, A, A, A, A, A, A, A, 0, 2, 5, 64, 4, None, 0, 1, None, 0), **over)


def _scan(**over):
    return _set(mixer.kda_scan_params(A, A, A, A, A, A, A, A, A, A, 2 * A, 0, 0, 0, 0, 0, 2, 5, 64, 16, 2, None, 0, 1, None, 0),
                **over)


def _scan_bwd(**over):
    return _set(mixer.kda_scan_bwd_params(_scan(), A, A, A, A, A, A, A, A, A, A, A, None, 0), **over)


def _gated(**over):
    return _set(mixer.kda_gated_norm_params(A, A, A, A, 7, 128, 1e-6, 0, 1), **over)


def _gated_bwd(**over):
    return _set(mixer.kda_gated_norm_bwd_params(_gated(), A, A, A, A, None, 0), **over)


def _block(**over):
    return _set(mixer.kda_block_norm_params(A, A, A, A, A, A, A, A, 7, 128, 1e-6, 0, 1, 2), **over)


def _block_bwd(**over):
    return _set(mixer.kda_block_norm_bwd_params(_block(), A, A, A, A, A, A, A, A, None, 0), **over)


INV, UNS, ALI = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_ALIGNMENT


@pytest.mark.parametrize("fn,make,over,want", [
    ("conv_fwd", _conv, dict(x=None), INV), ("conv_fwd", _conv, dict(weight=None), INV),
    ("conv_fwd", _conv, dict(y=None), INV), ("conv_fwd", _conv, dict(B=0), INV), ("conv_fwd", _conv, dict(T=-1), INV),
    ("conv_fwd", _conv, dict(D=0), INV), ("conv_fwd", _conv, dict(x_stride=63), INV),
    ("conv_fwd", _conv, dict(x_stride=-64), INV), ("conv_fwd", _conv, dict(W=1), UNS), ("conv_fwd", _conv, dict(W=5), UNS),
    ("conv_fwd", _conv, dict(dtype=2), UNS), ("conv_fwd", _conv, dict(activation=2), UNS),
    ("conv_fwd", _conv, dict(x=A + 1), ALI), ("conv_fwd", _conv, dict(weight=A + 2), ALI),
    ("conv_fwd", _conv, dict(st=A + 1), ALI), ("conv_fwd", _conv, dict(B=1 << 20, T=1 << 20), UNS),
    ("conv_fwd", _conv, dict(st=A), INV), ("scan_fwd", _scan, dict(ht=A), INV),  # states in place: the step calls only
    ("conv_step", _conv, dict(s0=None), INV), ("conv_step", _conv, dict(st=None), INV),
    ("conv_step", _conv, dict(cu_seqlens=A), INV),
    ("conv_bwd", _conv_bwd, dict(dy=None), INV), ("conv_bwd", _conv_bwd, dict(dx=None), INV),
    ("conv_bwd", _conv_bwd, dict(dweight=None), INV), ("conv_bwd", _conv_bwd, dict(W=9), UNS),
    ("conv_bwd", _conv_bwd, dict(ds0=A + 1), ALI), ("conv_bwd", _conv_bwd, dict(workspace=A, workspace_bytes=16), INV),
    ("scan_fwd", _scan, dict(u=None), INV), ("scan_fwd", _scan, dict(A=None), INV), ("scan_fwd", _scan, dict(y=None), INV),
    ("scan_fwd", _scan, dict(G=3), INV), ("scan_fwd", _scan, dict(G=0), INV), ("scan_fwd", _scan, dict(N=0), INV),
    ("scan_fwd", _scan, dict(N=65), UNS), ("scan_fwd", _scan, dict(dtype=5), UNS), ("scan_fwd", _scan, dict(B_stride=31), INV),
    ("scan_fwd", _scan, dict(z_stride=8), INV), ("scan_fwd", _scan, dict(u=A + 1), ALI), ("scan_fwd", _scan, dict(h0=A + 2), ALI),
    ("scan_fwd", _scan, dict(batch=1 << 16, T=1 << 16), UNS), ("scan_fwd", _scan, dict(channels=1 << 28), UNS),
    ("scan_step", _scan, dict(h0=None), INV), ("scan_step", _scan, dict(ht=None), INV), ("scan_step", _scan, dict(cu_seqlens=A), INV),
    ("scan_bwd", _scan_bwd, dict(dy=None), INV), ("scan_bwd", _scan_bwd, dict(dA=None), INV), ("scan_bwd", _scan_bwd, dict(dB=None), INV),
    ("scan_bwd", _scan_bwd, dict(D=None), INV), ("scan_bwd", _scan_bwd, dict(z=None), INV), ("scan_bwd", _scan_bwd, dict(N=100), UNS),
    ("scan_bwd", _scan_bwd, dict(du=A + 1), ALI), ("scan_bwd", _scan_bwd, dict(workspace=A, workspace_bytes=64), INV),
    ("gated_norm_fwd", _gated, dict(x=None), INV), ("gated_norm_fwd", _gated, dict(z=None), INV),
    ("gated_norm_fwd", _gated, dict(D=8193), UNS), ("gated_norm_fwd", _gated, dict(D=0), INV), ("gated_norm_fwd", _gated, dict(rows=-1), INV),
    ("gated_norm_fwd", _gated, dict(eps=-1.0), INV), ("gated_norm_fwd", _gated, dict(eps=float("nan")), INV),
    ("gated_norm_fwd", _gated, dict(activation=0), UNS), ("gated_norm_fwd", _gated, dict(y=A + 1), ALI),
    ("gated_norm_bwd", _gated_bwd, dict(dweight=None), INV), ("gated_norm_bwd", _gated_bwd, dict(dz=None), INV),
    ("gated_norm_bwd", _gated_bwd, dict(workspace=A, workspace_bytes=4), INV),
    ("block_norm_fwd", _block, dict(residual=None), INV), ("block_norm_fwd", _block, dict(weight=None), INV),
    ("block_norm_fwd", _block, dict(dtype=1, res_dtype=0), UNS), ("block_norm_fwd", _block, dict(activation=0), UNS),
    ("block_norm_fwd", _block, dict(new_residual=A + 2), ALI), ("block_norm_fwd", _block, dict(D=9000), UNS),
    ("block_norm_bwd", _block_bwd, dict(dresidual=None), INV), ("block_norm_bwd", _block_bwd, dict(z=None), INV),
    ("block_norm_bwd", _block_bwd, dict(scale=None), INV), ("block_norm_bwd", _block_bwd, dict(post_weight=None), INV),
    ("block_norm_bwd", _block_bwd, dict(dres=A + 2), ALI),
])
def test_bad_arguments_are_rejected(fn, make, over, want):
    assert getattr(mixer, "kda_" + fn)(make(**over), 0) == want


def test_null_params():
    for name in mixer.EXPORTED:
        got = mixer._fn(name)(None) if name.endswith("_workspace") else mixer._fn(name)(None, None)
        assert got == (0 if name.endswith("_workspace") else INV)


def test_workspace_sizes_of_rejected_calls_are_zero():
    assert mixer.kda_conv_bwd_workspace(_conv_bwd(W=7)) == 0
    assert mixer.kda_scan_bwd_workspace(_scan_bwd(N=65)) == 0
    assert mixer.kda_scan_fwd_workspace(_scan(N=65)) == 0
    assert mixer.kda_gated_norm_bwd_workspace(_gated_bwd(D=0)) == 0
    assert mixer.kda_block_norm_bwd_workspace(_block_bwd(D=0)) == 0


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


F = torch.float32


@pytest.mark.parametrize("what,error", [
    ("x_dim", ValueError), ("x_dtype", TypeError), ("w_shape", ValueError), ("w_dtype", TypeError), ("bias", ValueError),
    ("s0", ValueError), ("s0_dtype", TypeError), ("act", ValueError), ("cu_batch", ValueError), ("cu_dtype", TypeError),
    ("y", ValueError), ("st", ValueError), ("stride", ValueError)])
def test_conv_binding_rejects(what, error):
    x, w, b, kw = _t(2, 5, 16), _t(16, 4, dtype=F), _t(16, dtype=F), {}
    if what == "x_dim":
        x = _t(5, 16)
    elif what == "x_dtype":
        x = _t(2, 5, 16, dtype=torch.float16)
    elif what == "w_shape":
        w = _t(16, 5, dtype=F)
    elif what == "w_dtype":
        w = _t(16, 4)
    elif what == "bias":
        b = _t(15, dtype=F)
    elif what == "s0":
        kw["s0"] = _t(2, 4, 16)
    elif what == "s0_dtype":
        kw["s0"] = _t(2, 3, 16, dtype=F)
    elif what == "act":
        kw["activation"] = "sigmoid"
    elif what == "cu_batch":
        kw["cu_seqlens"] = torch.tensor([0, 5], dtype=torch.int32)
    elif what == "cu_dtype":
        x, kw["cu_seqlens"] = _t(1, 5, 16), torch.tensor([0, 5])
    elif what == "y":
        kw["y"] = _t(2, 5, 15)
    elif what == "st":
        kw.update(st=_t(1, 3, 16), output_final_state=True)
    else:
        x = _t(2, 5, 32)[:, :, ::2]
    with pytest.raises(error) as ei:
        pkg.causal_conv_fwd(x, w, b, **kw)
    assert "CUDA" not in str(ei.value)


def _scan_args(**over):
    a = dict(u=_t(2, 5, 12), dt=_t(2, 5, 12), A=_t(12, 7, dtype=F), B=_t(2, 5, 3, 7), C=_t(2, 5, 3, 7), D=_t(12, dtype=F),
             z=_t(2, 5, 12))
    a.update(over)
    return a


@pytest.mark.parametrize("over,error", [
    (dict(u=_t(5, 12)), ValueError), (dict(dt=_t(2, 5, 11)), ValueError), (dict(dt=_t(2, 5, 12, dtype=F)), TypeError),
    (dict(A=_t(12, 65, dtype=F)), ValueError), (dict(A=_t(12, 7)), TypeError), (dict(B=_t(2, 5, 5, 7)), ValueError),
    (dict(C=_t(2, 5, 3, 8)), ValueError), (dict(D=_t(12)), TypeError), (dict(z=_t(2, 4, 12)), ValueError)])
def test_scan_binding_rejects(over, error):
    for fn, more in ((pkg.selective_scan_fwd, {}), (pkg.selective_scan_step, dict(h=_t(2, 12, 7, dtype=F))),
                     (pkg.selective_scan_bwd, dict(dy=_t(2, 5, 12)))):
        with pytest.raises((ValueError, TypeError)) as ei:
            fn(**{**_scan_args(**over), **more})
        assert "CUDA" not in str(ei.value)
        if fn is pkg.selective_scan_fwd:
            assert isinstance(ei.value, error)


def test_well_formed_arguments_reach_the_device_check():
    x = _t(2, 5, 16)
    w = _t(16, 4, dtype=F)
    v = _t(16, dtype=F)
    calls = [lambda: pkg.causal_conv_fwd(x, w, v), lambda: pkg.causal_conv_bwd(x, w, v, x),
             lambda: pkg.causal_conv_step(x, _t(2, 3, 16), w, v),
             lambda: pkg.causal_conv_fwd(_t(2, 5, 48)[:, :, 16:32], w, v),
             lambda: pkg.selective_scan_fwd(**_scan_args()), lambda: pkg.selective_scan_bwd(**_scan_args(), dy=_t(2, 5, 12)),
             lambda: pkg.selective_scan_step(**_scan_args(), h=_t(2, 12, 7, dtype=F)),
             lambda: pkg.gated_norm_fwd(x, x, v), lambda: pkg.gated_norm_bwd(x, x, v, x),
             lambda: pkg.block_norm_fwd(x, _t(2, 5, 16, dtype=F), v), lambda: pkg.block_norm_bwd(x, x, v, x)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


@pytest.mark.parametrize("call,error", [
    (lambda x, v: pkg.gated_norm_fwd(x, x, _t(15, dtype=F)), ValueError),
    (lambda x, v: pkg.gated_norm_fwd(x, x.float(), v), TypeError),
    (lambda x, v: pkg.gated_norm_fwd(x, x, v, activation=None), ValueError),
    (lambda x, v: pkg.gated_norm_bwd(x, x, v, x[:1]), ValueError),
    (lambda x, v: pkg.block_norm_fwd(x.float(), x, v), TypeError),
    (lambda x, v: pkg.block_norm_fwd(x, x, v, scale=v.to(torch.bfloat16)), TypeError),
    (lambda x, v: pkg.block_norm_fwd(x, x, v, z=x[:1]), ValueError),
    (lambda x, v: pkg.block_norm_bwd(x, x, v, x, x.float()), TypeError),
    (lambda x, v: pkg.gated_norm_fwd(_t(1, 8200), _t(1, 8200), _t(8200, dtype=F)), ValueError)])
def test_norm_binding_rejects(call, error):
    with pytest.raises(error) as ei:
        call(_t(2, 5, 16), _t(16, dtype=F))
    assert "CUDA" not in str(ei.value)


def test_token_strides():
    wide = _t(3, 7, 40)
    assert mixer._token_stride(wide, "x") == 0
    assert mixer._token_stride(wide[:, :, 8:24], "x") == 40
    assert mixer._token_stride(_t(3, 1, 40)[:, :, :8], "x") == 40          # one token each: the batch's spacing
    assert mixer._token_stride(_t(1, 7, 40)[:, ::2], "x") == 80
    assert mixer._token_stride(_t(2, 5, 2, 3, 16)[:, :, 1], "B") == 96      # [B, T, G, N] inside something wider
    for bad in (wide[:, 1:], wide[:, :, ::2], wide.transpose(0, 1), wide[:, :1].expand(3, 7, 40)):
        with pytest.raises(ValueError):
            mixer._token_stride(bad, "x")


def test_reference_gradients_against_differences():
    """autograd through the 64-bit definitions, which the GPU tests compare with, against central
    differences along a random direction (error of second order: 1e-6 squared times curvature)."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    lens = [3, 0, 4]
    cases = [
        (lambda x, w, b, s0: ref.conv(x, w, b, s0, lens, "silu"), (r(7, 5), r(5, 3), r(5), r(3, 2, 5))),
        (lambda u, dt, A, B, C, D, z, b, h: ref.scan(u, dt, A, B, C, D, z, b, True, h, lens),
         (r(7, 4), r(7, 4), -r(4, 3).exp(), r(7, 2, 3), r(7, 2, 3), r(4), r(7, 4), r(4), r(3, 4, 3))),
        (lambda x, z, w: (ref.gated_norm(x, z, w, 1e-6, "silu"),), (r(3, 6), r(3, 6), r(6))),
        (lambda x, q, w, p, z, s: ref.block_norm(x, q, w, p, z, s, 1e-6, "sigmoid"), (r(3, 6), r(3, 6), r(6), r(6), r(3, 6), r(6))),
    ]
    for fn, args in cases:
        args = [a.clone().requires_grad_() for a in args]
        outs = fn(*args)
        cot = [r(*o.shape) for o in outs]
        got = torch.autograd.grad(sum((o * c).sum() for o, c in zip(outs, cot)), args)
        way = [r(*a.shape) for a in args]
        eps = 1e-6
        value = lambda e: sum((o * c).sum() for o, c in zip(fn(*[a.detach() + e * w for a, w in zip(args, way)]), cot))  # noqa: E731
        diff = float((value(eps) - value(-eps)) / (2 * eps))
        want = float(sum((a * w).sum() for a, w in zip(got, way)))
        assert abs(diff - want) <= 1e-7 * (1 + abs(want))


class _OnGpu(torch.Tensor):
    """A host tensor that says it lies on the GPU ``gpu``: what the binding's checks see of a device."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.gpu


def _on(gpu, *shape, dtype=torch.bfloat16):
    t = _t(*shape, dtype=dtype).as_subclass(_OnGpu)
    t.gpu = gpu
    return t


def _device_calls():
    """Every call of the binding with all its tensor arguments: (function, {name: (shape, dtype)}, other arguments)."""
    bf, i32 = torch.bfloat16, torch.int32
    conv = dict(x=((1, 5, 16), bf), weight=((16, 4), F), bias=((16,), F), s0=((2, 3, 16), bf), cu_seqlens=((3,), i32))
    scan = dict(u=((1, 5, 12), bf), dt=((1, 5, 12), bf), A=((12, 7), F), B=((1, 5, 3, 7), bf), C=((1, 5, 3, 7), bf), D=((12,), F),
                z=((1, 5, 12), bf), dt_bias=((12,), F))
    packed = dict(scan, h0=((2, 12, 7), F), cu_seqlens=((3,), i32))
    gated = dict(x=((5, 16), bf), z=((5, 16), bf), weight=((16,), F))
    block = dict(x=((5, 16), bf), residual=((5, 16), F), weight=((16,), F), post_weight=((16,), F), z=((5, 16), bf), scale=((16,), F))
    return [
        (pkg.causal_conv_fwd, dict(conv, y=((1, 5, 16), bf), st=((2, 3, 16), bf)), dict(output_final_state=True)),
        (pkg.causal_conv_step, dict(x=((2, 1, 16), bf), state=((2, 3, 16), bf), weight=((16, 4), F), bias=((16,), F), y=((2, 1, 16), bf)), {}),
        (pkg.causal_conv_bwd, dict(conv, dy=((1, 5, 16), bf), dst=((2, 3, 16), bf)), {}),
        (pkg.selective_scan_fwd, dict(packed, y=((1, 5, 12), bf), ht=((2, 12, 7), F)), {}),
        (pkg.selective_scan_step, dict(scan, h=((1, 12, 7), F), y=((1, 5, 12), bf)), {}),
        (pkg.selective_scan_bwd, dict(packed, dy=((1, 5, 12), bf), dht=((2, 12, 7), F)), {}),
        (pkg.gated_norm_fwd, dict(gated, y=((5, 16), bf)), {}),
        (pkg.gated_norm_bwd, dict(gated, dy=((5, 16), bf)), {}),
        (pkg.block_norm_fwd, dict(block, y=((5, 16), bf), new_residual=((5, 16), F)), {}),
        (pkg.block_norm_bwd, dict(block, dy=((5, 16), bf), dresidual=((5, 16), F)), {}),
    ]


@pytest.fixture
def on_gpus(monkeypatch):
    """Device 0 is current; the library's calls are recorded with the device that is current then."""
    current, calls = [0], []

    class device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            current.append(self.d)

        def __exit__(self, *a):
            current.pop()

    def fn(name):
        def call(p, *stream):
            calls.append((name, current[-1]))
            return 0
        return call

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(mixer, "_current_device", lambda: current[-1])
    monkeypatch.setattr(mixer, "_fn", fn)
    monkeypatch.setattr(mixer, "_stream", lambda device: 0)
    return calls


@pytest.mark.parametrize("fn,tensors,more", _device_calls(), ids=lambda v: getattr(v, "__name__", ""))
def test_tensors_of_two_devices_are_rejected(on_gpus, fn, tensors, more):
    make = lambda other: {k: _on(1 if k == other else 0, *s, dtype=d) for k, (s, d) in tensors.items()}  # noqa: E731
    fn(**make(None), **more)
    assert [d for _, d in on_gpus] == [0] * len(on_gpus) and on_gpus
    on_gpus.clear()
    for other in tensors:
        with pytest.raises(ValueError, match="one CUDA device"):
            fn(**make(other), **more)
    assert not on_gpus


@pytest.mark.parametrize("fn,tensors,more", _device_calls(), ids=lambda v: getattr(v, "__name__", ""))
def test_calls_run_on_the_tensors_device(on_gpus, fn, tensors, more):
    """Workspace query and call with the tensors' device current, also where a stream is given."""
    for kw in ({}, dict(stream=7)):
        fn(**{k: _on(1, *s, dtype=d) for k, (s, d) in tensors.items()}, **more, **kw)
    assert [d for _, d in on_gpus] == [1] * len(on_gpus)
    assert len([n for n, _ in on_gpus if not n.endswith("_workspace")]) == 2
