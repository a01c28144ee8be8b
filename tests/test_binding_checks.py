"""The Python binding's argument checks (host only, no GPU): every tensor's shape and dtype
is checked before anything reaches the library, whose kernels cannot check a raw pointer's
extent. CPU tensors of the right shapes get as far as the device check."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")


def _fwd_args(B=1, T=70, H=2, D=128, dtype=torch.bfloat16):
    q = torch.zeros(B, T, H, D, dtype=dtype)
    k = torch.zeros(B, T, H, D, dtype=dtype)
    v = torch.zeros(B, T, H, D, dtype=dtype)
    g = torch.zeros(B, T, H, D, dtype=torch.float32)
    beta = torch.zeros(B, T, H, dtype=torch.float32)
    return q, k, v, g, beta


def test_forward_well_formed_reaches_the_device_check():
    from chunkwise_gated_linear_gb300 import chunk_kda_fwd

    q, k, v, g, beta = _fwd_args()
    h0 = torch.zeros(1, 2, 128, 128)
    o = torch.zeros(1, 70, 2, 128, dtype=torch.bfloat16)
    ht = torch.zeros(1, 2, 128, 128)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        chunk_kda_fwd(q, k, v, g, beta, h0=h0, o=o, ht=ht)


@pytest.mark.parametrize("what", ["h0", "o_shape", "o_dtype", "ht", "cu_dtype", "cu_dim", "beta"])
def test_forward_rejects_malformed_arguments(what):
    from chunkwise_gated_linear_gb300 import chunk_kda_fwd

    q, k, v, g, beta = _fwd_args()
    kw = {}
    if what == "h0":
        kw["h0"] = torch.zeros(1, 2, 128, 64)
    elif what == "o_shape":
        kw["o"] = torch.zeros(1, 70, 2, 64, dtype=torch.bfloat16)
    elif what == "o_dtype":
        kw["o"] = torch.zeros(1, 70, 2, 128, dtype=torch.float32)
    elif what == "ht":
        kw["ht"] = torch.zeros(2, 2, 128, 128)
    elif what == "cu_dtype":
        kw["cu_seqlens"] = torch.tensor([0, 30, 70], dtype=torch.int64)
    elif what == "cu_dim":
        kw["cu_seqlens"] = torch.tensor([[0, 30, 70]], dtype=torch.int32)
    else:
        beta = torch.zeros(1, 70, 3)
    with pytest.raises((ValueError, TypeError)) as ei:
        chunk_kda_fwd(q, k, v, g, beta, **kw)
    assert "CUDA" not in str(ei.value)


def test_forward_ht_is_ignored_without_final_state():
    from chunkwise_gated_linear_gb300 import chunk_kda_fwd

    q, k, v, g, beta = _fwd_args()
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        chunk_kda_fwd(q, k, v, g, beta, ht=torch.zeros(3), output_final_state=False)


def test_backward_well_formed_reaches_the_device_check():
    from chunkwise_gated_linear_gb300 import chunk_kda_bwd

    q, k, v, g, beta = _fwd_args()
    do = torch.zeros_like(v)
    with pytest.raises(ValueError, match="contiguous CUDA tensor"):
        chunk_kda_bwd(q, k, v, g, beta, do, h0=torch.zeros(1, 2, 128, 128), dht=torch.zeros(1, 2, 128, 128))


@pytest.mark.parametrize("what", ["g_dtype", "beta_shape", "beta_dtype", "h0", "dht", "cu_dtype", "do"])
def test_backward_rejects_malformed_arguments(what):
    from chunkwise_gated_linear_gb300 import chunk_kda_bwd

    q, k, v, g, beta = _fwd_args()
    do = torch.zeros_like(v)
    kw = {}
    if what == "g_dtype":
        g = g.to(torch.bfloat16)
    elif what == "beta_shape":
        beta = torch.zeros(1, 70, 3)
    elif what == "beta_dtype":
        beta = beta.to(torch.bfloat16)
    elif what == "h0":
        kw["h0"] = torch.zeros(1, 2, 64, 128)
    elif what == "dht":
        kw["dht"] = torch.zeros(1, 2, 128, 128, dtype=torch.bfloat16)
    elif what == "cu_dtype":
        kw["cu_seqlens"] = torch.tensor([0, 30, 70], dtype=torch.int64)
    else:
        do = torch.zeros(1, 70, 2, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, TypeError)) as ei:
        chunk_kda_bwd(q, k, v, g, beta, do, **kw)
    assert "CUDA" not in str(ei.value)


class _OnGpu(torch.Tensor):
    """A host tensor that says it lies on the GPU ``gpu``: what the binding's checks see of a device."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.gpu


def _on(t, gpu):
    t = t.as_subclass(_OnGpu)
    t.gpu = gpu
    return t


def _device_call(which):
    """A call with all its tensor arguments, as (function, arguments by name, the C call's name)."""
    from chunkwise_gated_linear_gb300 import chunk_kda_bwd, chunk_kda_fwd

    q, k, v, g, beta = _fwd_args()
    h = torch.zeros(2, 2, 128, 128)
    args = dict(q=q, k=k, v=v, g=g, beta=beta, h0=h, cu_seqlens=torch.tensor([0, 30, 70], dtype=torch.int32))
    if which == "bwd":
        return chunk_kda_bwd, dict(args, do=torch.zeros_like(v), dht=h.clone()), "kda_chunk_bwd"
    args.update(o=torch.zeros_like(v), ht=h.clone())
    if which == "fused":
        return chunk_kda_fwd, dict(args, A_log=torch.zeros(2), dt_bias=torch.zeros(2, 128)), "kda_chunk_fwd_fused"
    return chunk_kda_fwd, args, "kda_chunk_fwd_ex"


@pytest.fixture
def on_gpus(monkeypatch):
    """Device 0 is current; the library's calls are recorded with the device that is current then."""
    from chunkwise_gated_linear_gb300 import kda

    current, calls = [0], []

    class device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            current.append(self.d)

        def __exit__(self, *a):
            current.pop()

    class stream:
        cuda_stream = 0

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[-1])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: stream)
    for name in ("kda_chunk_fwd_ex", "kda_chunk_fwd_fused", "kda_recurrent_fwd_ex", "kda_chunk_bwd"):
        monkeypatch.setattr(kda, name, lambda *a, name=name: calls.append((name, current[-1])) or 0)
    return calls


@pytest.mark.parametrize("which", ["fwd", "fused", "bwd"])
def test_tensors_of_two_devices_are_rejected(on_gpus, which):
    fn, args, name = _device_call(which)
    fn(**{k: _on(t, 0) for k, t in args.items()})
    assert on_gpus == [(name, 0)]
    for other in args:
        with pytest.raises(ValueError, match="one CUDA device"):
            fn(**{k: _on(t, 1 if k == other else 0) for k, t in args.items()})
    assert on_gpus == [(name, 0)]


@pytest.mark.parametrize("which", ["fwd", "fused", "bwd"])
def test_calls_run_on_the_tensors_device(on_gpus, which):
    fn, args, name = _device_call(which)
    for kw in ({}, dict(stream=7)):
        fn(**{k: _on(t, 1) for k, t in args.items()}, **kw)
    assert on_gpus == [(name, 1)] * 2
