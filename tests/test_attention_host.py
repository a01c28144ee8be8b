"""The attention-layer operators on the host: exported symbols, refusals before any CUDA call, the binding's
checks, frequencies, and the 64-bit definitions against each other (no GPU)."""

from __future__ import annotations

import ctypes
import math
import os
import re

import pytest
import torch

import attention_reference as aref
import chunkwise_gated_linear_gb300 as pkg
from attention_cases import BF, E4M3, E8M0, filled
from chunkwise_gated_linear_gb300 import KVCache, attention, kda, mixer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # an aligned address that is never dereferenced
F, I32 = torch.float32, torch.int32
INV, UNS, ALI = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_ALIGNMENT


def _header():
    text = open(os.path.join(ROOT, "include", "kda_attention.h"), encoding="utf-8").read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(kda_\w+)\s*\(", _header(), flags=re.M))
    assert names == set(attention.EXPORTED)
    for name in names:
        assert ctypes.cast(getattr(kda.lib(), name), ctypes.c_void_p).value


def test_structs_match_the_header():
    for name, body in re.findall(r"typedef struct (\w+) \{(.*?)\}", _header(), flags=re.S):
        fields = []
        for line in body.split(";"):
            line = line.replace("const", " ").replace("*", " ").strip()
            if line:
                first, *rest = line.split(None, 1)
                fields += [f.strip() for f in rest[0].split(",")]
        assert [f for f, _ in getattr(attention, name)._fields_] == fields, name


def _set(p, **over):
    """Fields of a struct or, by name, of the structs in it; `c_` in front: of its cache."""
    for k, v in over.items():
        at = p
        if k.startswith("c_"):
            at, k = p.cache, k[2:]
        elif not hasattr(p, k):
            at = p.f
        setattr(at, k, v)
    return p


def _cache():
    return attention.kda_kv_cache(A, A, None, None, 0, 0, 10, 2, 16, 64, 0, A, 4, 0, A)


def _fwd(**over):
    return _set(attention.kda_qk_norm_params(A, A, A, A, A, A, 2 * A, 2 * A, 0, 0, 2, 5, 4, 2, 64, 64, None, 1e-6, 0, 0), **over)


def _bwd(**over):
    return _set(attention.kda_qk_norm_bwd_params(_fwd(), A, A, A, A, A, A, None, 0), **over)


def _step(**over):
    return _set(attention.kda_qk_norm_step_params(_fwd(), A, 0, _cache()), **over)


def _write(**over):
    return _set(attention.kda_kv_cache_write_params(A, A, 0, 0, 2, 5, None, 0, _cache()), **over)


def _read(**over):
    return _set(attention.kda_kv_cache_read_params(A, A, 2, 5, None, 0, _cache()), **over)


def _attn(**over):
    return _set(attention.kda_attn_step_params(A, A, A, 0, 2, 1, 8, 0.125, 0, _cache(), None, 0), **over)


CACHE = [(dict(c_k=None), INV), (dict(c_v=None), INV), (dict(c_block_table=None), INV), (dict(c_lens=None), INV), (dict(c_pages=0), INV),
         (dict(c_page_size=0), INV), (dict(c_max_pages=0), INV), (dict(c_dtype=3), UNS), (dict(c_dtype=1), UNS), (dict(c_dtype=2), INV),
         (dict(c_k_scale=A), INV), (dict(c_page_stride=2 * 16 * 64 - 64), INV), (dict(c_page_stride=2 * 16 * 64 + 1), INV),
         (dict(c_dtype=2, c_k_scale=A, c_v_scale=A, c_scale_stride=31), INV), (dict(c_table_stride=3), INV), (dict(c_k=A + 8), ALI),
         (dict(c_v=A + 2), ALI), (dict(c_lens=A + 2), ALI), (dict(c_block_table=A + 1), ALI), (dict(c_pages=1 << 30), UNS)]


@pytest.mark.parametrize("fn,make,over,want", [
    ("qk_norm_fwd", _fwd, dict(q=None), INV), ("qk_norm_fwd", _fwd, dict(k_out=None), INV), ("qk_norm_fwd", _fwd, dict(B=0), INV),
    ("qk_norm_fwd", _fwd, dict(T=-1), INV), ("qk_norm_fwd", _fwd, dict(q_heads=0), INV), ("qk_norm_fwd", _fwd, dict(D=0), INV),
    ("qk_norm_fwd", _fwd, dict(D=257, R=64), UNS), ("qk_norm_fwd", _fwd, dict(R=66), INV), ("qk_norm_fwd", _fwd, dict(R=63), INV),
    ("qk_norm_fwd", _fwd, dict(R=-2), INV), ("qk_norm_fwd", _fwd, dict(freq=None), INV), ("qk_norm_fwd", _fwd, dict(eps=-1.0), INV),
    ("qk_norm_fwd", _fwd, dict(eps=float("nan")), INV), ("qk_norm_fwd", _fwd, dict(dtype=2), UNS),
    ("qk_norm_fwd", _fwd, dict(q_stride=255), INV), ("qk_norm_fwd", _fwd, dict(k_stride=-128), INV), ("qk_norm_fwd", _fwd, dict(q=A + 1), ALI),
    ("qk_norm_fwd", _fwd, dict(q_weight=A + 2), ALI), ("qk_norm_fwd", _fwd, dict(freq=A + 4), ALI),
    ("qk_norm_fwd", _fwd, dict(positions=A + 1), ALI), ("qk_norm_fwd", _fwd, dict(cu_seqlens=A + 2), ALI),
    ("qk_norm_fwd", _fwd, dict(B=1 << 15, T=1 << 15), UNS), ("qk_norm_fwd", _fwd, dict(q_heads=4, k_heads=(1 << 31) - 1), UNS),
    ("qk_norm_fwd", _fwd, dict(B=1, T=1 << 28, q_heads=4, k_heads=2), UNS), ("qk_norm_bwd", _bwd, dict(k_heads=(1 << 31) - 1), UNS),
    ("kv_cache_write", _write, dict(c_heads=(1 << 30) + 2), UNS), ("kv_cache_read", _read, dict(c_heads=(1 << 31) - 1), UNS),
    ("qk_norm_fwd", _fwd, dict(q_out=A, q_stride=512), INV), ("qk_norm_fwd", _fwd, dict(k_out=A, k_stride=512), INV),  # in place: contiguous
    ("qk_norm_bwd", _bwd, dict(dq_out=None), INV), ("qk_norm_bwd", _bwd, dict(dk=None), INV), ("qk_norm_bwd", _bwd, dict(q_weight=None), INV),
    ("qk_norm_bwd", _bwd, dict(k_weight=None), INV), ("qk_norm_bwd", _bwd, dict(dq=A + 1), ALI), ("qk_norm_bwd", _bwd, dict(dk_weight=A + 1), ALI),
    ("qk_norm_bwd", _bwd, dict(D=300), UNS),
    ("qk_norm_step", _step, dict(v=None), INV), ("qk_norm_step", _step, dict(v_stride=64), INV), ("qk_norm_step", _step, dict(v=A + 1), ALI),
    ("qk_norm_step", _step, dict(c_heads=1), INV), ("qk_norm_step", _step, dict(c_D=32), INV), ("qk_norm_step", _step, dict(q_out=None), INV),
    ("kv_cache_write", _write, dict(k=None), INV), ("kv_cache_write", _write, dict(v=None), INV), ("kv_cache_write", _write, dict(B=0), INV),
    ("kv_cache_write", _write, dict(dtype=2), UNS), ("kv_cache_write", _write, dict(k_stride=127), INV), ("kv_cache_write", _write, dict(v=A + 1), ALI),
    ("kv_cache_read", _read, dict(k=None), INV), ("kv_cache_read", _read, dict(T=-1), INV), ("kv_cache_read", _read, dict(v=A + 1), ALI),
    ("kv_cache_read", _read, dict(dtype=2), UNS),
    ("attn_step", _attn, dict(q=None), INV), ("attn_step", _attn, dict(o=None), INV), ("attn_step", _attn, dict(q_heads=7), INV),
    ("attn_step", _attn, dict(q_heads=0), INV), ("attn_step", _attn, dict(B=0), INV), ("attn_step", _attn, dict(T=-1), INV),
    ("attn_step", _attn, dict(scale=float("inf")), INV), ("attn_step", _attn, dict(scale=float("nan")), INV), ("attn_step", _attn, dict(dtype=2), UNS),
    ("attn_step", _attn, dict(q_stride=500), INV), ("attn_step", _attn, dict(q_stride=513), ALI), ("attn_step", _attn, dict(q=A + 8), ALI),
    ("attn_step", _attn, dict(o=A + 2), ALI), ("attn_step", _attn, dict(lse=A + 2), ALI), ("attn_step", _attn, dict(T=1 << 28), UNS),
    ("attn_step", _attn, dict(q_heads=514), UNS), ("attn_step", _attn, dict(B=4, T=1 << 20, c_max_pages=1 << 20), UNS),  # counts of units
    ("attn_step", _attn, dict(B=1 << 20, T=1, c_max_pages=1 << 20, dtype=1, c_dtype=1), UNS),
] + [(fn, make, over, want) for over, want in CACHE
     for fn, make in (("qk_norm_step", _step), ("kv_cache_write", _write), ("kv_cache_read", _read), ("attn_step", _attn))])
def test_bad_arguments_are_rejected(fn, make, over, want):
    assert getattr(attention, "kda_" + fn)(make(**over), 0) == want


def test_step_with_keys_in_place():
    """Keys that are also written beside the cache may be written in place only where they are contiguous, as in the forward call."""
    assert attention.kda_qk_norm_step(_step(k_out=A, k_stride=512), 0) == INV
    assert attention.kda_qk_norm_step(_step(q_out=A, q_stride=512), 0) == INV


@pytest.mark.parametrize("over", [dict(c_heads=1 << 29, c_page_size=1 << 30, c_D=32), dict(c_heads=(1 << 30) - (1 << 16), c_page_size=(1 << 31) - 1, c_D=256),
                                  dict(c_heads=1 << 20, c_page_size=1 << 20, c_D=64), dict(c_heads=1, c_page_size=(1 << 31) - 1, c_pages=3)])
def test_caches_of_more_rows_than_are_counted(over):
    """Sizes whose products pass 63 bits are refused like all that pass the limit of rows."""
    sizes = {"B": 1, "T": 1, "c_pages": 1, **over}
    assert attention.kda_kv_cache_write(_write(**sizes), 0) == UNS
    assert attention.kda_kv_cache_read(_read(**sizes), 0) == UNS


@pytest.mark.parametrize("D", [8, 24, 272])
def test_widths_that_a_cache_does_not_hold(D):
    assert attention.kda_kv_cache_write(_write(c_D=D), 0) == UNS
    assert attention.kda_attn_step(_attn(c_D=D), 0) == UNS


def test_null_params():
    for name in attention.EXPORTED:
        got = mixer._fn(name)(None) if name.endswith("_workspace") else mixer._fn(name)(None, None)
        assert got == (0 if name.endswith("_workspace") else INV)


def test_workspace_sizes_of_rejected_calls_are_zero():
    assert attention.kda_qk_norm_bwd_workspace(_bwd(D=0)) == 0
    assert attention.kda_attn_step_workspace(_attn(c_D=8)) == 0
    assert attention.kda_attn_step_workspace(_attn(T=0)) == 0
    assert attention.kda_attn_step_workspace(_attn(B=4, T=1 << 20, c_max_pages=1 << 20)) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="a host without a device")
def test_well_formed_calls_report_a_missing_device():
    for fn, make in (("qk_norm_fwd", _fwd), ("qk_norm_bwd", _bwd), ("qk_norm_step", _step), ("kv_cache_write", _write), ("kv_cache_read", _read),
                     ("attn_step", _attn)):
        for over in (dict(), dict(D=24, R=24)) if fn.startswith("qk_norm") and fn != "qk_norm_step" else (dict(),):
            assert getattr(attention, "kda_" + fn)(make(**over), 0) == kda.KDA_ERR_CUDA, (fn, over)
    attention.kda_qk_norm_bwd_workspace(_bwd())
    attention.kda_attn_step_workspace(_attn())


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=torch.uint8).view(dtype) if dtype in (E4M3, E8M0) else torch.zeros(*shape, dtype=dtype)


def _pages(dtype=BF, heads=2, D=64):
    c = (_t(10, heads, 16, D, dtype=dtype), _t(10, heads, 16, D, dtype=dtype))
    return KVCache(*c, *((_t(10, heads, 16, dtype=E8M0), _t(10, heads, 16, dtype=E8M0)) if dtype == E4M3 else ()))


def _calls(**over):
    """Every call with well-formed arguments (of which `over` replaces some) as (function, arguments by name)."""
    a = dict(q=_t(3, 5, 8, 64), k=_t(3, 5, 2, 64), v=_t(3, 5, 2, 64), q_weight=_t(64, dtype=F), k_weight=_t(64, dtype=F),
             freq=_t(32, dtype=torch.int64), cache=_pages(), block_table=_t(3, 4, dtype=I32), lens=_t(3, dtype=I32),
             dq_out=_t(3, 5, 8, 64), dk_out=_t(3, 5, 2, 64), tokens=5)
    a.update(over)
    pick = lambda *names: {n: a[n] for n in names + tuple(k for k in over if k in ("positions", "cu_seqlens", "q_out"))}  # noqa: E731
    return {"fwd": (pkg.qk_norm_fwd, pick("q", "k", "q_weight", "k_weight", "freq")),
            "bwd": (pkg.qk_norm_bwd, {n: v for n, v in pick("q", "k", "q_weight", "k_weight", "freq", "dq_out", "dk_out").items() if n != "q_out"}),
            "step": (pkg.qk_norm_step, pick("q", "k", "v", "cache", "block_table", "lens", "q_weight", "k_weight", "freq")),
            "write": (pkg.kv_cache_write, {n: a[n] for n in ("k", "v", "cache", "block_table", "lens")}),
            "read": (pkg.kv_cache_read, {n: a[n] for n in ("cache", "block_table", "lens", "tokens")}),
            "attn": (pkg.paged_attn_step, {n: a[n] for n in ("q", "cache", "block_table", "lens")})}


@pytest.mark.parametrize("over,names,error", [
    (dict(q=_t(3, 5, 64)), "fwd bwd step attn", ValueError), (dict(q=_t(3, 5, 8, 64, dtype=torch.float16)), "fwd bwd step attn", TypeError),
    (dict(k=_t(3, 4, 2, 64)), "fwd bwd step write", ValueError), (dict(k=_t(3, 5, 2, 64, dtype=F)), "fwd bwd step write", TypeError),
    (dict(q=_t(3, 5, 8, 128)[..., ::2]), "fwd step attn", ValueError), (dict(q=_t(3, 6, 8, 64)[:, 1:]), "fwd step attn", ValueError),
    (dict(q_weight=_t(63, dtype=F)), "fwd bwd step", ValueError), (dict(k_weight=_t(64)), "fwd bwd step", TypeError),
    (dict(freq=_t(33, dtype=torch.int64)), "fwd bwd step", ValueError), (dict(freq=_t(32, dtype=F)), "fwd bwd step", TypeError),
    (dict(positions=_t(3, 4, dtype=I32)), "fwd bwd step", ValueError), (dict(positions=_t(3, 5, dtype=torch.int64)), "fwd bwd step", TypeError),
    (dict(cu_seqlens=_t(3, dtype=I32)), "fwd bwd step", ValueError), (dict(q_out=_t(3, 5, 8, 32)), "fwd step", ValueError),
    (dict(dq_out=_t(3, 5, 8, 32)), "bwd", ValueError), (dict(dk_out=_t(3, 5, 2, 64, dtype=F)), "bwd", TypeError),
    (dict(v=_t(3, 5, 1, 64)), "step write", ValueError), (dict(v=_t(3, 5, 2, 64, dtype=F)), "step write", TypeError),
    (dict(cache=_pages(heads=3)), "step write attn", ValueError), (dict(cache=_pages(D=32)), "step write attn", ValueError),
    (dict(cache=_pages(F)), "step write attn", TypeError), (dict(cache=_pages(D=24)), "step write read attn", ValueError),
    (dict(cache=_pages(E4M3)._replace(k_scale=None)), "step write read attn", ValueError),
    (dict(cache=_pages(E4M3)._replace(v_scale=_t(10, 2, 15, dtype=E8M0))), "step write read attn", ValueError),
    (dict(cache=_pages(E4M3)._replace(v_scale=_t(10, 2, 16, dtype=torch.uint8))), "step write read attn", TypeError),
    (dict(cache=_pages()._replace(k_scale=_t(10, 2, 16, dtype=E8M0))), "step write read attn", ValueError),
    (dict(cache=_pages()._replace(v=_t(9, 2, 16, 64))), "step write read attn", ValueError),
    (dict(cache=_pages()._replace(v=_t(10, 2, 2, 16, 64)[:, 1])), "step write read attn", ValueError),
    (dict(cache=KVCache(*(_t(10, 2, 64, 16).transpose(2, 3) for _ in "kv"))), "step write read attn", ValueError),
    (dict(block_table=_t(2, 4, dtype=I32)), "step write read attn", ValueError), (dict(block_table=_t(3, 4)), "step write read attn", TypeError),
    (dict(block_table=_t(4, 3, dtype=I32).t()), "step write read attn", ValueError),
    (dict(lens=_t(2, dtype=I32)), "step write read attn", ValueError), (dict(lens=_t(3, dtype=torch.int64)), "step write read attn", TypeError),
    (dict(lens=_t(6, dtype=I32)[::2]), "step write read attn", ValueError), (dict(q=_t(3, 5, 7, 64)), "attn", ValueError),
    (dict(tokens=-1), "read", ValueError)])
def test_binding_rejects(over, names, error):
    calls = _calls(**over)
    for name in names.split():
        fn, args = calls[name]
        with pytest.raises(error) as ei:
            fn(**args)
        assert "CUDA" not in str(ei.value), name


def test_well_formed_arguments_reach_the_device_check():
    for over in ({}, dict(cache=_pages(E4M3)), dict(q_weight=None, freq=None)):
        for fn, args in _calls(**over).values():
            with pytest.raises(ValueError, match="CUDA tensor"):
                fn(**args)


class _OnGpu(torch.Tensor):
    """A host tensor that says it lies on the GPU ``gpu``: what the binding's checks see of a device."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.gpu


def _on(gpu, t):
    if isinstance(t, KVCache):
        return KVCache(*(None if x is None else _on(gpu, x) for x in t))
    if not torch.is_tensor(t):
        return t
    t = t.as_subclass(_OnGpu)
    t.gpu = gpu
    return t


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

    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(mixer, "_current_device", lambda: current[-1])
    monkeypatch.setattr(mixer, "_fn", fn)
    monkeypatch.setattr(mixer, "_stream", lambda device: 0)
    return calls


@pytest.mark.parametrize("name", ["fwd", "bwd", "step", "write", "read", "attn"])
def test_devices(on_gpus, name):
    fn, args = _calls(cache=_pages(E4M3))[name]
    for gpu in (0, 1):
        fn(**{k: _on(gpu, v) for k, v in args.items()})
        fn(**{k: _on(gpu, v) for k, v in args.items()}, stream=7)
        assert on_gpus and all(d == gpu for _, d in on_gpus)
        assert len([n for n, _ in on_gpus if not n.endswith("_workspace")]) == 2
        on_gpus.clear()
    for other in args:
        if isinstance(args[other], KVCache):
            for i in range(4):
                mixed = {k: _on(0, v) for k, v in args.items()}
                mixed["cache"] = KVCache(*(_on(1 if i == j else 0, t) for j, t in enumerate(args["cache"])))
                with pytest.raises(ValueError, match="one CUDA device"):
                    fn(**mixed)
        elif torch.is_tensor(args[other]):
            with pytest.raises(ValueError, match="one CUDA device"):
                fn(**{k: _on(1 if k == other else 0, v) for k, v in args.items()})
    assert not on_gpus


def test_frequencies():
    """Fractions of a turn: a double's few last bits of each, and one unit of the table, 2^-64 (it is cut off there)."""
    for R, theta in ((128, 1e4), (64, 1e6), (2, 1e4)):
        f = pkg.rope_frequencies(R, theta, device="cpu")
        want = aref.inv_freq(R, theta) / (2 * math.pi)
        assert f.dtype == torch.int64 and f.shape == (R // 2,)
        assert bool(((f.double() * 2.0 ** -64 - want).abs() <= 2.0 ** -51 * want + 2.0 ** -64).all())
    f = pkg.rope_frequencies(8, inv_freq=[7.0, -1.0, 4.0, 0.0], device="cpu")
    turns = [7.0 / (2 * math.pi) % 1.0, -1.0 / (2 * math.pi) % 1.0, 4.0 / (2 * math.pi), 0.0]
    got = [(int(x) % (1 << 64)) / 2.0 ** 64 for x in f]
    assert all(abs(a - b) < 1e-15 for a, b in zip(got, turns))
    assert pkg.rope_frequencies(0, device="cpu").shape == (0,)
    for bad in (dict(R=3), dict(R=-2), dict(R=4, inv_freq=[1.0]), dict(R=2, inv_freq=[float("inf")])):
        with pytest.raises(ValueError):
            pkg.rope_frequencies(**bad, device="cpu")


def test_empty_caches():
    c = KVCache.empty(3, 2, 16, 64, device="cpu")
    assert c.k.dtype == BF and c.k_scale is None and c.k.shape == c.v.shape == (3, 2, 16, 64)
    c = KVCache.empty(3, 2, 16, 64, E4M3, device="cpu")
    assert c.k.dtype == E4M3 and c.k_scale.dtype == E8M0 and c.v_scale.shape == (3, 2, 16)
    with pytest.raises(TypeError):
        KVCache.empty(3, 2, 16, 64, torch.float16, device="cpu")


def test_rounding_reference():
    """The reference's 8-bit rounding against torch's conversion, and its power of two against the definition."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(500, 64, generator=g, dtype=torch.float64) * torch.exp(torch.randn(500, 1, generator=g, dtype=torch.float64) * 5)
    unit = aref.row_unit(x)
    top = x.abs().amax(-1)
    assert bool((top <= 448 * unit).all()) and bool((top > 224 * unit).all())
    y = (x / unit[..., None]).float()  # one rounding more than the reference's, the same for torch's conversion
    assert torch.equal(aref.e4m3_round(y.double()), y.to(E4M3).double())


def test_reference_attention_against_one_softmax():
    g = torch.Generator().manual_seed(1)
    cache, table = filled(g, [40], 16, 2, 32, F)
    q = torch.randn(1, 3, 4, 32, generator=g)
    o, lse = aref.attention(q, cache, table, [40], 0.3)
    k, v = aref.gather(cache, table, 0, 40, 16)
    for t in range(3):
        for h in range(4):
            s = 0.3 * k[h // 2, :38 + t] @ q[0, t, h].double()
            assert torch.allclose(o[0, t, h], torch.softmax(s, 0) @ v[h // 2, :38 + t], rtol=1e-12, atol=1e-12)
            assert abs(float(lse[0, t, h] - s.exp().sum().log())) < 1e-12


def test_reference_norm_gradients_against_differences():
    """autograd through the 64-bit definition, which the GPU tests compare with, against central differences along a
    random direction (error of second order: 1e-6 squared times curvature)."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    pos = torch.tensor([0, 5, 1000])
    for interleaved in (False, True):
        fn = lambda x, w: aref.norm_rope(x, w, pos, aref.inv_freq(4), 1e-6, interleaved)  # noqa: E731,B023
        args = [r(3, 2, 6).requires_grad_(), r(6).requires_grad_()]
        y = fn(*args)
        cot, way, eps = r(*y.shape), [r(*a.shape) for a in args], 1e-6
        got = torch.autograd.grad((y * cot).sum(), args)
        value = lambda e: (fn(*[a.detach() + e * w for a, w in zip(args, way)]) * cot).sum()  # noqa: E731,B023
        diff = float((value(eps) - value(-eps)) / (2 * eps))
        want = float(sum((a * w).sum() for a, w in zip(got, way)))
        assert abs(diff - want) <= 1e-7 * (1 + abs(want))
