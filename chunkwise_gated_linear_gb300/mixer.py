"""Python binding of the token-mixer operators of ``libkda.so`` (``include/kda_mixer.h``): the
short causal convolution, the selective state space scan, the gated output norm and the
block's residual update with its norms, each with its gradient.

As in :mod:`.kda`, the functions take torch CUDA tensors, check shapes and dtypes, allocate
the outputs with torch and call the C ABI on the current torch stream (or ``stream``); every
step of the computation runs in the library's CUDA kernels. Data tensors are bf16 or fp32;
parameters and recurrence states are fp32. The data inputs of the convolution and the scan may be
slices of wider tensors as long as their tokens are evenly spaced and each token's channels
contiguous; all other tensors are contiguous. All tensors of a call lie on one device, which need
not be the current one. With ``cu_seqlens`` (int32 [N + 1] on the device) the batch
dimension is 1 and holds N packed sequences.
"""

from __future__ import annotations

import ctypes
import sys

from .kda import KDA_DTYPE_BF16, KDA_DTYPE_F32, KDA_OK, KdaError, _ptr, lib

KDA_ACT_NONE = 0
KDA_ACT_SILU = 1
KDA_ACT_SIGMOID = 2

EXPORTED = ("kda_conv_fwd", "kda_conv_step", "kda_conv_bwd", "kda_conv_bwd_workspace",
            "kda_scan_fwd", "kda_scan_fwd_workspace", "kda_scan_step", "kda_scan_bwd", "kda_scan_bwd_workspace",
            "kda_gated_norm_fwd", "kda_gated_norm_bwd", "kda_gated_norm_bwd_workspace",
            "kda_block_norm_fwd", "kda_block_norm_bwd", "kda_block_norm_bwd_workspace")

_P, _I, _L, _F, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


def _fields(*groups):
    return [(name, ctype) for ctype, names in groups for name in names.split()]


class kda_conv_params(ctypes.Structure):
    _fields_ = _fields((_P, "x weight bias s0 y st"), (_L, "x_stride"), (_I, "B T D W"), (_P, "cu_seqlens"),
                       (_I, "dtype activation"))


class kda_conv_bwd_params(ctypes.Structure):
    _fields_ = _fields((_P, "x weight bias s0 dy dst dx dweight dbias ds0"), (_L, "x_stride"), (_I, "B T D W"),
                       (_P, "cu_seqlens"), (_I, "dtype activation"), (_P, "workspace"), (_S, "workspace_bytes"))


class kda_scan_params(ctypes.Structure):
    _fields_ = _fields((_P, "u dt A B C D z dt_bias h0 y ht"), (_L, "u_stride dt_stride B_stride C_stride z_stride"),
                       (_I, "batch T channels N G"), (_P, "cu_seqlens"), (_I, "dtype dt_softplus"),
                       (_P, "workspace"), (_S, "workspace_bytes"))


class kda_scan_bwd_params(ctypes.Structure):
    _fields_ = _fields((kda_scan_params, "f"), (_P, "dy dht du ddt dA dB dC dD dz ddt_bias dh0 workspace"),
                       (_S, "workspace_bytes"))


class kda_gated_norm_params(ctypes.Structure):
    _fields_ = _fields((_P, "x z weight y"), (_L, "rows"), (_I, "D"), (_F, "eps"), (_I, "dtype activation"))


class kda_gated_norm_bwd_params(ctypes.Structure):
    _fields_ = _fields((kda_gated_norm_params, "f"), (_P, "dy dx dz dweight workspace"), (_S, "workspace_bytes"))


class kda_block_norm_params(ctypes.Structure):
    _fields_ = _fields((_P, "x residual weight post_weight z scale y new_residual"), (_L, "rows"), (_I, "D"),
                       (_F, "eps"), (_I, "dtype res_dtype activation"))


class kda_block_norm_bwd_params(ctypes.Structure):
    _fields_ = _fields((kda_block_norm_params, "f"),
                       (_P, "dy dres dx dresidual dweight dpost_weight dz dscale workspace"), (_S, "workspace_bytes"))


_PARAMS = dict(kda_conv_fwd=kda_conv_params, kda_conv_step=kda_conv_params, kda_conv_bwd=kda_conv_bwd_params,
               kda_scan_fwd=kda_scan_params, kda_scan_step=kda_scan_params, kda_scan_bwd=kda_scan_bwd_params,
               kda_gated_norm_fwd=kda_gated_norm_params, kda_gated_norm_bwd=kda_gated_norm_bwd_params,
               kda_block_norm_fwd=kda_block_norm_params, kda_block_norm_bwd=kda_block_norm_bwd_params)

_fns = {}


def _fn(name):
    """The C function, its argument types set on first use."""
    fn = _fns.get(name)
    if fn is None:
        fn = getattr(lib(), name)
        if name.endswith("_workspace"):
            fn.argtypes = [ctypes.POINTER(_PARAMS[name[:-len("_workspace")]])]
            fn.restype = _S
        else:
            fn.argtypes = [ctypes.POINTER(_PARAMS[name]), _P]
            fn.restype = _I
        _fns[name] = fn
    return fn


# ---- raw C entry points -------------------------------------------------------------------

def kda_conv_fwd(params, stream) -> int:
    return _fn("kda_conv_fwd")(params, stream or None)


def kda_conv_step(params, stream) -> int:
    return _fn("kda_conv_step")(params, stream or None)


def kda_conv_bwd(params, stream) -> int:
    return _fn("kda_conv_bwd")(params, stream or None)


def kda_conv_bwd_workspace(params) -> int:
    return _fn("kda_conv_bwd_workspace")(params)


def kda_scan_fwd(params, stream) -> int:
    return _fn("kda_scan_fwd")(params, stream or None)


def kda_scan_fwd_workspace(params) -> int:
    return _fn("kda_scan_fwd_workspace")(params)


def kda_scan_step(params, stream) -> int:
    return _fn("kda_scan_step")(params, stream or None)


def kda_scan_bwd(params, stream) -> int:
    return _fn("kda_scan_bwd")(params, stream or None)


def kda_scan_bwd_workspace(params) -> int:
    return _fn("kda_scan_bwd_workspace")(params)


def kda_gated_norm_fwd(params, stream) -> int:
    return _fn("kda_gated_norm_fwd")(params, stream or None)


def kda_gated_norm_bwd(params, stream) -> int:
    return _fn("kda_gated_norm_bwd")(params, stream or None)


def kda_gated_norm_bwd_workspace(params) -> int:
    return _fn("kda_gated_norm_bwd_workspace")(params)


def kda_block_norm_fwd(params, stream) -> int:
    return _fn("kda_block_norm_fwd")(params, stream or None)


def kda_block_norm_bwd(params, stream) -> int:
    return _fn("kda_block_norm_bwd")(params, stream or None)


def kda_block_norm_bwd_workspace(params) -> int:
    return _fn("kda_block_norm_bwd_workspace")(params)


# ---- checks -------------------------------------------------------------------------------

def _dtype(t, name):
    torch = sys.modules["torch"]

    if t.dtype == torch.bfloat16:
        return KDA_DTYPE_BF16
    if t.dtype == torch.float32:
        return KDA_DTYPE_F32
    raise TypeError(f"{name} must be bf16 or fp32")


def _want(t, name, shape, dtype):
    """A tensor argument's dtype and shape (None passes)."""
    if t is None or (t.dtype is dtype and t.shape == shape):
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {str(dtype).replace('torch.', '')}")
    raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")


def _token_stride(t, name, lead=2):
    """Elements between consecutive tokens of a tensor whose first ``lead`` dimensions are its
    tokens; the others have to be contiguous and the tokens evenly spaced."""
    if t.is_contiguous():
        return 0
    inner = 1
    for n, st in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
        if n != 1 and st != inner:
            raise ValueError(f"{name}: the channels of a token must be contiguous")
        inner *= n
    step = None  # between tokens
    span = 1
    for n, st in zip(reversed(t.shape[:lead]), reversed(t.stride()[:lead])):
        if n != 1:
            if step is None:
                step = st // span if st % span == 0 else -1
            if step < inner or st != step * span:
                raise ValueError(f"{name}: the tokens must be evenly spaced")
        span *= n
    return 0 if step is None or step == inner else step


def _device(lead, strided, dense):
    """Every tensor on the CUDA device of ``lead``, those of ``dense`` contiguous."""
    device = lead.get_device()  # -1 on the host
    good = device >= 0
    for t in dense:
        if t is not None and (t.get_device() != device or not t.is_contiguous()):
            good = False
    for t in strided:
        if t is not None and t.get_device() != device:
            good = False
    if good:
        return
    devices = {t.get_device() for t in (lead, *strided, *dense) if t is not None}
    if len(devices) > 1 and -1 not in devices:
        raise ValueError("every tensor must be on one CUDA device")
    raise ValueError("every tensor must be a CUDA tensor and contiguous (the data inputs of the convolution and the scan: "
                     "evenly spaced tokens)")


def _sequences(cu_seqlens, B):
    """The number of sequences."""
    torch = sys.modules["torch"]

    if cu_seqlens is None:
        return B
    if B != 1:
        raise ValueError("packed sequences need B == 1")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise TypeError("cu_seqlens must be int32 [N + 1]")
    return cu_seqlens.numel() - 1


def _act(activation, allowed):
    known = {None: KDA_ACT_NONE, "silu": KDA_ACT_SILU, "sigmoid": KDA_ACT_SIGMOID}
    if activation not in allowed:
        raise ValueError(f"activation must be one of {', '.join(repr(a) for a in allowed)}")
    return known[activation]


# torch's own raw getters: no Stream object, no check that CUDA has been initialised (2 us less per
# call). The public ways where a torch version lacks them.

def _stream(device):
    """The handle of torch's current stream on a device."""
    torch = sys.modules["torch"]

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return torch.cuda.current_stream(device).cuda_stream if raw is None else raw(device)


def _current_device():
    torch = sys.modules["torch"]

    raw = getattr(torch._C, "_cuda_getDevice", None)
    return torch.cuda.current_device() if raw is None else raw()


def _call(name, p, t, stream, workspace=False):
    """Run a C entry point; ``workspace``: give it torch memory for its scratch. On a stream
    that torch does not know of, the library takes the scratch from its own pool instead: torch
    would hand the memory out again before that stream is done with it. The library launches on the
    current device: that of the tensors, of which ``t`` is one, is made current for the call."""
    device = t.get_device()
    if device != _current_device():
        with sys.modules["torch"].cuda.device(device):
            return _call(name, p, t, stream, workspace)
    ws = None  # keeps the scratch until the call has been queued
    if stream is None:
        stream = _stream(device)
        if workspace:
            n = _fn(name + "_workspace")(p)
            if n:
                torch = sys.modules["torch"]
                ws = torch.empty(n, dtype=torch.uint8, device=t.device)
                p.workspace = ws.data_ptr()
                p.workspace_bytes = n
    st = _fn(name)(p, stream or None)
    if st != KDA_OK:
        raise KdaError(st, name)


# ---- short causal convolution -------------------------------------------------------------

def _conv_check(x, weight, bias, s0, cu_seqlens):
    torch = sys.modules["torch"]

    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    B, T, D = x.shape
    dtype = _dtype(x, "x")
    if weight.dim() != 2 or weight.shape[0] != D or weight.shape[1] not in (2, 3, 4):
        raise ValueError("weight must be [D, W] with W 2, 3 or 4")
    W = weight.shape[1]
    _want(weight, "weight", (D, W), torch.float32)
    _want(bias, "bias", (D,), torch.float32)
    N = _sequences(cu_seqlens, B)
    _want(s0, "s0", (N, W - 1, D), x.dtype)
    return B, T, D, W, N, dtype


def causal_conv_fwd(x, weight, bias=None, *, s0=None, activation="silu", cu_seqlens=None,
                    output_final_state=False, y=None, st=None, stream=None):
    """Short causal depthwise convolution; returns ``(y, st)``.

    x [B, T, D] bf16 or fp32; weight fp32 [D, W], W 2 to 4, the last tap being the current token;
    bias fp32 [D] or None; ``activation`` "silu" or None. s0 [N, W - 1, D] in the dtype of x holds
    the inputs before each sequence (None: zeros), st the last ones, for the next call (None in
    the result unless ``output_final_state``). ``y`` and ``st`` may be given to write into.
    """
    torch = sys.modules["torch"]

    B, T, D, W, N, dtype = _conv_check(x, weight, bias, s0, cu_seqlens)
    act = _act(activation, ("silu", None))
    _want(y, "y", (B, T, D), x.dtype)
    if not output_final_state:
        st = None
    _want(st, "st", (N, W - 1, D), x.dtype)
    stride = _token_stride(x, "x")
    _device(x, (), (weight, bias, s0, cu_seqlens, y, st))
    if y is None:
        y = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    if output_final_state and st is None:
        st = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device)
    p = kda_conv_params(_ptr(x), _ptr(weight), _ptr(bias), _ptr(s0), _ptr(y), _ptr(st), stride, N, T, D, W,
                        _ptr(cu_seqlens), dtype, act)
    _call("kda_conv_fwd", p, x, stream)
    return y, st


def causal_conv_step(x, state, weight, bias=None, *, activation="silu", y=None, stream=None):
    """The convolution of the next tokens of B sequences: x [B, T, D] (T typically 1), ``state``
    [B, W - 1, D] updated in place. Returns y."""
    torch = sys.modules["torch"]

    B, T, D, W, _, dtype = _conv_check(x, weight, bias, state, None)
    act = _act(activation, ("silu", None))
    _want(y, "y", (B, T, D), x.dtype)
    stride = _token_stride(x, "x")
    _device(x, (), (weight, bias, state, y))
    if y is None:
        y = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    p = kda_conv_params(_ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), _ptr(state), stride, B, T, D, W,
                        None, dtype, act)
    _call("kda_conv_step", p, x, stream)
    return y


def causal_conv_bwd(x, weight, bias, dy, *, s0=None, dst=None, activation="silu", cu_seqlens=None, want_ds0=True,
                    stream=None):
    """Backward of :func:`causal_conv_fwd`: same inputs plus ``dy`` (of y) and ``dst`` (of st, or
    None). Returns ``(dx, dweight, dbias, ds0)``: dx and ds0 in the dtype of x, the others fp32;
    dbias is None without bias, ds0 None when ``want_ds0`` is False."""
    torch = sys.modules["torch"]

    B, T, D, W, N, dtype = _conv_check(x, weight, bias, s0, cu_seqlens)
    act = _act(activation, ("silu", None))
    _want(dy, "dy", (B, T, D), x.dtype)
    _want(dst, "dst", (N, W - 1, D), x.dtype)
    stride = _token_stride(x, "x")
    _device(x, (), (weight, bias, s0, cu_seqlens, dy, dst))
    dx = torch.empty((B, T, D), dtype=x.dtype, device=x.device)
    dweight = torch.empty_like(weight)
    dbias = None if bias is None else torch.empty_like(bias)
    ds0 = torch.empty((N, W - 1, D), dtype=x.dtype, device=x.device) if want_ds0 else None
    p = kda_conv_bwd_params(_ptr(x), _ptr(weight), _ptr(bias), _ptr(s0), _ptr(dy), _ptr(dst), _ptr(dx), _ptr(dweight),
                            _ptr(dbias), _ptr(ds0), stride, N, T, D, W, _ptr(cu_seqlens), dtype, act, None, 0)
    _call("kda_conv_bwd", p, x, stream, workspace=True)
    return dx, dweight, dbias, ds0


# ---- selective state space scan -------------------------------------------------------------

def _scan_params(u, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, y, ht, dense=()):
    """Checks shared by the three calls; the argument struct and the number of sequences."""
    torch = sys.modules["torch"]

    if u.dim() != 3:
        raise ValueError("u must be [B, T, channels]")
    nb, T, ch = u.shape
    dtype = _dtype(u, "u")
    if A.dim() != 2 or A.shape[0] != ch or not 1 <= A.shape[1] <= 64:
        raise ValueError("A must be [channels, N] with 1 <= N <= 64")
    N = A.shape[1]
    if B.dim() != 4 or B.shape[2] < 1 or ch % B.shape[2] != 0:
        raise ValueError("B must be [B, T, G, N], G a divisor of the channels")
    G = B.shape[2]
    _want(A, "A", (ch, N), torch.float32)
    _want(dt, "dt", u.shape, u.dtype)
    _want(B, "B", (nb, T, G, N), u.dtype)
    _want(C, "C", (nb, T, G, N), u.dtype)
    _want(z, "z", u.shape, u.dtype)
    _want(D, "D", (ch,), torch.float32)
    _want(dt_bias, "dt_bias", (ch,), torch.float32)
    ns = _sequences(cu_seqlens, nb)
    _want(h0, "h0", (ns, ch, N), torch.float32)
    _want(y, "y", u.shape, u.dtype)
    _want(ht, "ht", (ns, ch, N), torch.float32)
    strides = [0 if t is None else _token_stride(t, name) for name, t in (("u", u), ("dt", dt), ("B", B), ("C", C), ("z", z))]
    _device(u, (dt, B, C, z), (A, D, dt_bias, h0, cu_seqlens, y, ht, *dense))
    p = kda_scan_params(_ptr(u), _ptr(dt), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(h0), None,
                        None, *strides, ns, T, ch, N, G, _ptr(cu_seqlens), dtype, 1 if dt_softplus else 0, None, 0)
    return p, ns


def selective_scan_fwd(u, dt, A, B, C, D=None, z=None, *, dt_bias=None, dt_softplus=True, h0=None, cu_seqlens=None,
                       output_final_state=True, y=None, ht=None, stream=None):
    """Selective state space scan; returns ``(y, ht)``.

    u, dt, z [B, T, channels] and B, C [B, T, G, N], all bf16 or all fp32; A fp32 [channels, N],
    N up to 64; D, dt_bias fp32 [channels] or None; h0 fp32 [N_seq, channels, N] or None. With
    delta = softplus(dt + dt_bias) (no softplus with ``dt_softplus`` False),
    h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t and y_t = (C_t . h_t + D u_t) silu(z_t), the
    channels of group g reading B and C of that group. ``ht`` is None in the result when
    ``output_final_state`` is False.
    """
    torch = sys.modules["torch"]

    if not output_final_state:
        ht = None
    p, ns = _scan_params(u, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, y, ht)
    if y is None:
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    if output_final_state and ht is None:
        ht = torch.empty((ns, *A.shape), dtype=torch.float32, device=u.device)
    p.y, p.ht = _ptr(y), _ptr(ht)
    _call("kda_scan_fwd", p, u, stream, workspace=True)
    return y, ht


def selective_scan_step(u, dt, A, B, C, h, D=None, z=None, *, dt_bias=None, dt_softplus=True, y=None, stream=None):
    """The scan of the next tokens of B sequences (u [B, T, channels], T typically 1), the states
    ``h`` [B, channels, N] updated in place. Returns y."""
    torch = sys.modules["torch"]

    if h is None:
        raise ValueError("h is required")
    p, _ = _scan_params(u, dt, A, B, C, D, z, dt_bias, dt_softplus, h, None, y, None)
    if y is None:
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    p.y, p.ht = _ptr(y), _ptr(h)
    _call("kda_scan_step", p, u, stream)
    return y


def selective_scan_bwd(u, dt, A, B, C, dy, D=None, z=None, *, dt_bias=None, dt_softplus=True, h0=None, dht=None,
                       cu_seqlens=None, want_dh0=True, stream=None):
    """Backward of :func:`selective_scan_fwd`: same inputs plus ``dy`` (of y) and ``dht`` (of ht, or
    None). Returns ``(du, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)``: du, ddt, dz, dB, dC in the
    dtype of u, the others fp32; dD, dz and ddt_bias are None where the argument is, dh0 when
    ``want_dh0`` is False."""
    torch = sys.modules["torch"]

    _want(dy, "dy", u.shape, u.dtype)
    f, ns = _scan_params(u, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, None, None, (dy, dht))
    _want(dht, "dht", (ns, *A.shape), torch.float32)
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)  # noqa: E731
    du, ddt, dA, dB, dC, dD, dz, dbias = (new(t) for t in (u, dt, A, B, C, D, z, dt_bias))
    dh0 = torch.empty((ns, *A.shape), dtype=torch.float32, device=u.device) if want_dh0 else None
    p = kda_scan_bwd_params(f, _ptr(dy), _ptr(dht), _ptr(du), _ptr(ddt), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dz),
                            _ptr(dbias), _ptr(dh0), None, 0)
    _call("kda_scan_bwd", p, u, stream, workspace=True)
    return du, ddt, dA, dB, dC, dD, dz, dbias, dh0


# ---- gated output norm ------------------------------------------------------------------------

def _rows(t):
    n = 1
    for s in t.shape[:-1]:
        n *= s
    return n


def _gated_norm_params(x, z, weight, eps, activation, y, dense=()):
    torch = sys.modules["torch"]

    if x.dim() < 1 or not 1 <= x.shape[-1] <= 8192:
        raise ValueError("x must be [..., D] with 1 <= D <= 8192")
    dtype = _dtype(x, "x")
    act = _act(activation, ("silu", "sigmoid"))
    _want(z, "z", x.shape, x.dtype)
    _want(weight, "weight", x.shape[-1:], torch.float32)
    _want(y, "y", x.shape, x.dtype)
    _device(x, (), (x, z, weight, y, *dense))
    return kda_gated_norm_params(_ptr(x), _ptr(z), _ptr(weight), None, _rows(x), x.shape[-1], eps, dtype, act)


def gated_norm_fwd(x, z, weight, *, eps=1e-6, activation="silu", y=None, stream=None):
    """x / rms(x) * weight * act(z) over the last dimension (the recurrence's output x, normed per
    head, times its gate). x, z [..., D] bf16 or fp32, D up to 8192; weight fp32 [D];
    ``activation`` "silu" or "sigmoid". Returns y like x."""
    torch = sys.modules["torch"]

    p = _gated_norm_params(x, z, weight, eps, activation, y)
    if y is None:
        y = torch.empty_like(x)
    p.y = _ptr(y)
    _call("kda_gated_norm_fwd", p, x, stream)
    return y


def gated_norm_bwd(x, z, weight, dy, *, eps=1e-6, activation="silu", stream=None):
    """Backward of :func:`gated_norm_fwd`; returns ``(dx, dz, dweight)``, dweight fp32."""
    torch = sys.modules["torch"]

    _want(dy, "dy", x.shape, x.dtype)
    f = _gated_norm_params(x, z, weight, eps, activation, None, (dy,))
    dx, dz, dw = torch.empty_like(x), torch.empty_like(z), torch.empty_like(weight)
    p = kda_gated_norm_bwd_params(f, _ptr(dy), _ptr(dx), _ptr(dz), _ptr(dw), None, 0)
    _call("kda_gated_norm_bwd", p, x, stream, workspace=True)
    return dx, dz, dw


# ---- residual update and norm -------------------------------------------------------------------

def _block_norm_params(x, residual, weight, post_weight, z, scale, eps, activation, y, new_residual, dense=()):
    torch = sys.modules["torch"]

    if x.dim() < 1 or not 1 <= x.shape[-1] <= 8192:
        raise ValueError("x must be [..., D] with 1 <= D <= 8192")
    dtype = _dtype(x, "x")
    act = _act(activation, ("silu", "sigmoid"))
    ch = x.shape[-1:]
    if residual.dtype not in (x.dtype, torch.float32):
        raise TypeError("residual must be fp32 or have the dtype of x")
    _want(residual, "residual", x.shape, residual.dtype)
    _want(weight, "weight", ch, torch.float32)
    _want(post_weight, "post_weight", ch, torch.float32)
    _want(z, "z", x.shape, x.dtype)
    _want(scale, "scale", ch, torch.float32)
    _want(y, "y", x.shape, x.dtype)
    _want(new_residual, "new_residual", x.shape, residual.dtype)
    _device(x, (), (x, residual, weight, post_weight, z, scale, y, new_residual, *dense))
    return kda_block_norm_params(_ptr(x), _ptr(residual), _ptr(weight), _ptr(post_weight), _ptr(z), _ptr(scale), None, None,
                                 _rows(x), x.shape[-1], eps, dtype, _dtype(residual, "residual"), act)


def block_norm_fwd(x, residual, weight, *, post_weight=None, z=None, scale=None, eps=1e-6, activation="sigmoid", y=None,
                   new_residual=None, stream=None):
    """The end of a block and the start of the next: ``new_residual = residual + scale * act(z) *
    (x / rms(x) * post_weight)`` and ``y = new_residual / rms(new_residual) * weight``; returns
    ``(y, new_residual)``.

    x (the block's output) and z [..., D] bf16 or fp32; residual fp32 or in the dtype of x; weight,
    post_weight, scale fp32 [D]. Without post_weight x is not normed, without z not gated,
    without scale not scaled. ``new_residual`` may be ``residual`` (updated in place).
    """
    torch = sys.modules["torch"]

    p = _block_norm_params(x, residual, weight, post_weight, z, scale, eps, activation, y, new_residual)
    if y is None:
        y = torch.empty_like(x)
    if new_residual is None:
        new_residual = torch.empty_like(residual)
    p.y, p.new_residual = _ptr(y), _ptr(new_residual)
    _call("kda_block_norm_fwd", p, x, stream)
    return y, new_residual


def block_norm_bwd(x, residual, weight, dy, dresidual=None, *, post_weight=None, z=None, scale=None, eps=1e-6,
                   activation="sigmoid", stream=None):
    """Backward of :func:`block_norm_fwd` for the gradients ``dy`` of y and ``dresidual`` of
    new_residual (None: none); ``residual`` is the tensor before the update. Returns
    ``(dx, dresidual, dweight, dpost_weight, dz, dscale)``, None where the argument is."""
    torch = sys.modules["torch"]

    _want(dy, "dy", x.shape, x.dtype)
    _want(dresidual, "dresidual", residual.shape, residual.dtype)
    f = _block_norm_params(x, residual, weight, post_weight, z, scale, eps, activation, None, None, (dy, dresidual))
    new = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
    dx, dr, dw, dpw, dz, ds = (new(t) for t in (x, residual, weight, post_weight, z, scale))
    p = kda_block_norm_bwd_params(f, _ptr(dy), _ptr(dresidual), _ptr(dx), _ptr(dr), _ptr(dw), _ptr(dpw), _ptr(dz), _ptr(ds),
                                  None, 0)
    _call("kda_block_norm_bwd", p, x, stream, workspace=True)
    return dx, dr, dw, dpw, dz, ds
