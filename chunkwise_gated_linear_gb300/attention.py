"""Python binding of the attention-layer operators of ``libkda.so`` (``include/kda_attention.h``): the
norms of queries and keys with the position rotation, a paged key-value cache written and read
back, and the attention of the next tokens over it.

As in :mod:`.mixer`, the functions take torch CUDA tensors, check shapes and dtypes, allocate the
outputs with torch and call the C ABI on the current torch stream (or ``stream``); every step of
the computation runs in the library's CUDA kernels. Data tensors are bf16 or fp32, weights fp32. q, k
and v may be slices of wider tensors as long as their tokens are evenly spaced and each token's
heads and channels contiguous; all other tensors are contiguous. All tensors of a call lie on one
device, which need not be the current one. With ``cu_seqlens`` (int32 [N + 1] on the device)
the batch dimension is 1 and holds N packed sequences.

A cache is a :class:`KVCache` with a ``block_table`` [N, pages per sequence] (int32: which pages hold a
sequence's tokens) and ``lens`` [N] (int32: the sequences' lengths with the call's new tokens in them).
Of n new tokens, token i stands at position lens - n + i; one at a negative position is not there, so
that a sequence at rest in a batch has length 0.
"""

from __future__ import annotations

import ctypes
import math
import sys
from typing import Any, NamedTuple

from .kda import KDA_DTYPE_BF16, KDA_DTYPE_F32, _ptr
from .mixer import _F, _I, _L, _P, _S, _call, _dtype, _fields, _PARAMS, _fn, _sequences, _token_stride, _want

KDA_DTYPE_E4M3 = 2
KDA_DEVICE_ERR_CACHE = 4

EXPORTED = ("kda_qk_norm_fwd", "kda_qk_norm_bwd", "kda_qk_norm_bwd_workspace", "kda_qk_norm_step", "kda_kv_cache_write",
            "kda_kv_cache_read", "kda_attn_step", "kda_attn_step_workspace")


class kda_kv_cache(ctypes.Structure):
    _fields_ = _fields((_P, "k v k_scale v_scale"), (_L, "page_stride scale_stride"), (_I, "pages heads page_size D dtype"),
                       (_P, "block_table"), (_I, "max_pages"), (_L, "table_stride"), (_P, "lens"))


class kda_qk_norm_params(ctypes.Structure):
    _fields_ = _fields((_P, "q k q_weight k_weight freq positions q_out k_out"), (_L, "q_stride k_stride"),
                       (_I, "B T q_heads k_heads D R"), (_P, "cu_seqlens"), (_F, "eps"), (_I, "dtype interleaved"))


class kda_qk_norm_bwd_params(ctypes.Structure):
    _fields_ = _fields((kda_qk_norm_params, "f"), (_P, "dq_out dk_out dq dk dq_weight dk_weight workspace"), (_S, "workspace_bytes"))


class kda_qk_norm_step_params(ctypes.Structure):
    _fields_ = _fields((kda_qk_norm_params, "f"), (_P, "v"), (_L, "v_stride"), (kda_kv_cache, "cache"))


class kda_kv_cache_write_params(ctypes.Structure):
    _fields_ = _fields((_P, "k v"), (_L, "k_stride v_stride"), (_I, "B T"), (_P, "cu_seqlens"), (_I, "dtype"), (kda_kv_cache, "cache"))


class kda_kv_cache_read_params(ctypes.Structure):
    _fields_ = _fields((_P, "k v"), (_I, "B T"), (_P, "cu_seqlens"), (_I, "dtype"), (kda_kv_cache, "cache"))


class kda_attn_step_params(ctypes.Structure):
    _fields_ = _fields((_P, "q o lse"), (_L, "q_stride"), (_I, "B T q_heads"), (_F, "scale"), (_I, "dtype"), (kda_kv_cache, "cache"),
                       (_P, "workspace"), (_S, "workspace_bytes"))


_PARAMS.update(kda_qk_norm_fwd=kda_qk_norm_params, kda_qk_norm_bwd=kda_qk_norm_bwd_params, kda_qk_norm_step=kda_qk_norm_step_params,
               kda_kv_cache_write=kda_kv_cache_write_params, kda_kv_cache_read=kda_kv_cache_read_params,
               kda_attn_step=kda_attn_step_params)


# ---- raw C entry points -------------------------------------------------------------------

def kda_qk_norm_fwd(params, stream) -> int:
    return _fn("kda_qk_norm_fwd")(params, stream or None)


def kda_qk_norm_bwd(params, stream) -> int:
    return _fn("kda_qk_norm_bwd")(params, stream or None)


def kda_qk_norm_bwd_workspace(params) -> int:
    return _fn("kda_qk_norm_bwd_workspace")(params)


def kda_qk_norm_step(params, stream) -> int:
    return _fn("kda_qk_norm_step")(params, stream or None)


def kda_kv_cache_write(params, stream) -> int:
    return _fn("kda_kv_cache_write")(params, stream or None)


def kda_kv_cache_read(params, stream) -> int:
    return _fn("kda_kv_cache_read")(params, stream or None)


def kda_attn_step(params, stream) -> int:
    return _fn("kda_attn_step")(params, stream or None)


def kda_attn_step_workspace(params) -> int:
    return _fn("kda_attn_step_workspace")(params)


# ---- checks -------------------------------------------------------------------------------

def _place(lead, others):
    """Every tensor on the CUDA device of ``lead``."""
    device = lead.get_device()  # -1 on the host
    good = device >= 0
    for t in others:
        if t is not None and t.get_device() != device:
            good = False
    if good:
        return
    devices = {t.get_device() for t in (lead, *others) if t is not None}
    if len(devices) > 1 and -1 not in devices:
        raise ValueError("every tensor must be on one CUDA device")
    raise ValueError("every tensor must be a CUDA tensor")


def _like(t):
    """An empty contiguous tensor like ``t``."""
    torch = sys.modules["torch"]
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _dense(names, *tensors):
    for t in tensors:
        if t is not None and not t.is_contiguous():
            bad = [n for n, x in zip(names.split(), tensors) if x is not None and not x.is_contiguous()]
            raise ValueError(f"{bad[0]} must be contiguous")


def _heads(t, name, B, T, D, dtype):
    """The heads of a tensor [B, T, heads, D] and its token stride."""
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != T or shape[3] != D or shape[2] < 1:
        raise ValueError(f"{name} must be [{B}, {T}, heads, {D}], not {list(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must have the dtype of the other data tensors")
    return shape[2], _tokens(t, name, B, T, shape[2], D)


def _tokens(t, name, B, T, H, D):
    """Elements between consecutive tokens: :func:`mixer._token_stride`, its usual cases first."""
    s = t.stride()
    if s[3] == 1 and s[2] == D:
        step = s[1] if T > 1 else s[0] if B > 1 else H * D
        if step >= H * D and (B == 1 or T == 1 or s[0] == T * step):
            return step
    return _token_stride(t, name)


# ---- the cache ------------------------------------------------------------------------------

class KVCache(NamedTuple):
    """Pages of keys and values: k, v [pages, heads, page_size, D] bf16, fp32 or float8_e4m3fn, the last with
    k_scale, v_scale [pages, heads, page_size] float8_e8m0fnu (a row's values are its e4m3 numbers times
    its power of two). Pages may lie apart (slices of one buffer for several layers), k like v."""

    k: Any
    v: Any
    k_scale: Any = None
    v_scale: Any = None

    @classmethod
    def empty(cls, pages, heads, page_size, D, dtype=None, device="cuda"):
        """A cache of ``pages`` pages, zeroed; ``dtype``: torch.bfloat16 (the default), torch.float32 or
        torch.float8_e4m3fn."""
        torch = sys.modules["torch"]

        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
            raise TypeError("a cache holds bf16, fp32 or float8_e4m3fn")
        shape = (pages, heads, page_size, D)
        if dtype != torch.float8_e4m3fn:
            return cls(torch.zeros(shape, dtype=dtype, device=device), torch.zeros(shape, dtype=dtype, device=device))
        new = lambda s, t, fill: torch.full(s, fill, dtype=torch.uint8, device=device).view(t)  # noqa: E731
        return cls(new(shape, torch.float8_e4m3fn, 0), new(shape, torch.float8_e4m3fn, 0),
                   new(shape[:3], torch.float8_e8m0fnu, 1), new(shape[:3], torch.float8_e8m0fnu, 1))


def _page_stride(t, name):
    """Elements between consecutive pages (0: contiguous); a page itself has to be contiguous."""
    if t.is_contiguous():
        return 0
    inner = 1
    for n, st in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and st != inner:
            raise ValueError(f"{name}: a page must be contiguous")
        inner *= n
    if t.shape[0] == 1:
        return 0
    if t.stride(0) < inner:
        raise ValueError(f"{name}: pages must not overlap")
    return t.stride(0)


def _cache(cache, block_table, lens, N, data):
    """The C struct of a cache that N sequences of tensors of type ``data`` use."""
    torch = sys.modules["torch"]

    k, v, ks, vs = cache
    shape, kind = k.shape, k.dtype
    if len(shape) != 4 or min(shape) < 1 or shape[3] % 16 != 0 or shape[3] > 256:
        raise ValueError("the cache must be [pages, heads, page_size, D], D a multiple of 16 up to 256")
    pages, heads, page, D = shape
    scale_stride = 0
    if kind is torch.float8_e4m3fn:
        code = KDA_DTYPE_E4M3
        if ks is None or vs is None:
            raise ValueError("a float8_e4m3fn cache has k_scale and v_scale")
        rows, bits = shape[:3], torch.float8_e8m0fnu
        if not (ks.dtype is bits and vs.dtype is bits and ks.shape == rows and vs.shape == rows):
            _want(ks, "k_scale", rows, bits)
            _want(vs, "v_scale", rows, bits)
        if not (ks.is_contiguous() and vs.is_contiguous()):
            scale_stride = _page_stride(ks, "k_scale")
            if _page_stride(vs, "v_scale") != scale_stride:
                raise ValueError("k_scale and v_scale must have the same strides")
    else:
        if kind is not data:
            raise TypeError("the cache must have the dtype of the data or float8_e4m3fn")
        if ks is not None or vs is not None:
            raise ValueError("only a float8_e4m3fn cache has scales")
        code = KDA_DTYPE_BF16 if data is torch.bfloat16 else KDA_DTYPE_F32
    if not (v.dtype is kind and v.shape == shape):
        _want(v, "v of the cache", shape, kind)
    page_stride = 0
    if not (k.is_contiguous() and v.is_contiguous()):
        page_stride = _page_stride(k, "k of the cache")
        if _page_stride(v, "v of the cache") != page_stride:
            raise ValueError("k and v of the cache must have the same strides")
        if page_stride % D != 0:
            raise ValueError("the pages of the cache must lie a multiple of D elements apart")
    if block_table.dtype is not torch.int32 or lens.dtype is not torch.int32:
        raise TypeError("block_table and lens must be int32")
    table = block_table.shape
    if len(table) != 2 or table[0] != N or table[1] < 1:
        raise ValueError(f"block_table must be [{N}, pages per sequence], not {list(table)}")
    if lens.shape != (N,):
        raise ValueError(f"lens must be [{N}], not {list(lens.shape)}")
    width = table[1]
    row = width
    if not block_table.is_contiguous():
        row = block_table.stride(0) if N > 1 else width
        if width > 1 and block_table.stride(1) != 1 or row < width:
            raise ValueError("block_table: the entries of a sequence must be contiguous")
    if not lens.is_contiguous():
        raise ValueError("lens must be contiguous")
    return kda_kv_cache(k.data_ptr(), v.data_ptr(), _ptr(ks), _ptr(vs), page_stride, scale_stride, pages, heads, page, D, code,
                        block_table.data_ptr(), width, row, lens.data_ptr())


def kv_cache_write(k, v, cache, block_table, lens, *, cu_seqlens=None, stream=None):
    """The new tokens k, v [B, T, heads, D] (bf16 or fp32) into the cache, each at its position; other places
    stay as they are. A float8_e4m3fn cache takes each row with the least power of two that leaves its
    largest entry at 448 or below, rounded to nearest. No two tokens of a call may have one place."""
    shape = k.shape
    if len(shape) != 4:
        raise ValueError("k must be [B, T, heads, D]")
    B, T, H, D = shape
    dtype = _dtype(k, "k")
    N = _sequences(cu_seqlens, B)
    Hv, v_stride = _heads(v, "v", B, T, D, k.dtype)
    k_stride = _tokens(k, "k", B, T, H, D)
    c = _cache(cache, block_table, lens, N, k.dtype)
    if Hv != H or c.heads != H or c.D != D:
        raise ValueError("k, v and the cache must have the same heads and channels")
    _dense("cu_seqlens", cu_seqlens)
    _place(k, (v, cu_seqlens, *cache, block_table, lens))
    p = kda_kv_cache_write_params(_ptr(k), _ptr(v), k_stride, v_stride, N, T, _ptr(cu_seqlens), dtype, c)
    _call("kda_kv_cache_write", p, k, stream)


def kv_cache_read(cache, block_table, lens, tokens, *, cu_seqlens=None, dtype=None, k=None, v=None, stream=None):
    """The last ``tokens`` tokens of each sequence out of the cache: (k, v) [B, tokens, heads, D]; with
    ``cu_seqlens`` as many of each sequence as it says, in [1, tokens, heads, D]. Zeros for tokens that are not
    there. ``dtype``: the cache's own, or bf16 (the default) or fp32 for a float8_e4m3fn cache."""
    torch = sys.modules["torch"]

    if dtype is None:
        dtype = torch.bfloat16 if cache.k.dtype == torch.float8_e4m3fn else cache.k.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("dtype must be bf16 or fp32")
    B = 1 if cu_seqlens is not None else block_table.shape[0]
    N = _sequences(cu_seqlens, B)
    if tokens < 0:
        raise ValueError("tokens must not be negative")
    c = _cache(cache, block_table, lens, N, dtype)
    shape = (B, tokens, c.heads, c.D)
    _want(k, "k", shape, dtype)
    _want(v, "v", shape, dtype)
    _dense("k v cu_seqlens", k, v, cu_seqlens)
    _place(cache.k, (*cache, block_table, lens, k, v, cu_seqlens))
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache.k.device)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=cache.k.device)
    kind = KDA_DTYPE_BF16 if dtype == torch.bfloat16 else KDA_DTYPE_F32
    p = kda_kv_cache_read_params(_ptr(k), _ptr(v), N, tokens, _ptr(cu_seqlens), kind, c)
    _call("kda_kv_cache_read", p, cache.k, stream)
    return k, v


# ---- norms of queries and keys with the position rotation -------------------------------------

def rope_frequencies(R, theta=10000.0, *, inv_freq=None, device="cuda"):
    """The rotation's frequencies for :func:`qk_norm_fwd` and its like: int64 [R / 2], turns per position in
    units of 2^-64. Pair i turns by theta^(-2 i / R) radians per position, or by ``inv_freq[i]`` (any R / 2
    numbers, taken in 64 bits)."""
    torch = sys.modules["torch"]

    if R < 0 or R % 2 != 0:
        raise ValueError("R must be even")
    if inv_freq is None:
        per = [theta ** (-2.0 * i / R) for i in range(R // 2)]
    else:
        per = [float(x) for x in inv_freq]
        if len(per) != R // 2 or not all(math.isfinite(x) for x in per):
            raise ValueError(f"inv_freq must be {R // 2} finite numbers")
    turns = [int(math.fmod(x / (2.0 * math.pi), 1.0) * 2.0 ** 64) % (1 << 64) for x in per]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in turns], dtype=torch.int64, device=device)


def _norm_check(q, k, q_weight, k_weight, freq, positions, cu_seqlens, eps, interleaved, q_out, k_out):
    torch = sys.modules["torch"]

    shape, kind = q.shape, q.dtype
    if len(shape) != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, Hq, D = shape
    if not 1 <= D <= 256 or Hq < 1:
        raise ValueError("q must be [B, T, heads, D] with 1 <= D <= 256")
    dtype = _dtype(q, "q")
    N = _sequences(cu_seqlens, B)
    Hk, k_stride = _heads(k, "k", B, T, D, kind)
    q_stride = _tokens(q, "q", B, T, Hq, D)
    _want(q_weight, "q_weight", (D,), torch.float32)
    _want(k_weight, "k_weight", (D,), torch.float32)
    R = 0
    if freq is not None:
        if freq.dtype is not torch.int64:
            raise TypeError("freq must be int64 (rope_frequencies)")
        R = 2 * freq.numel()
        if freq.dim() != 1 or R > D:
            raise ValueError("freq must be [R / 2] with R <= D")
    if positions is not None:
        _want(positions, "positions", (B, T), torch.int32)
    if q_out is not None:
        _want(q_out, "q_out", shape, kind)
    if k_out is not None:
        _want(k_out, "k_out", k.shape, kind)
    _dense("q_weight k_weight freq positions cu_seqlens q_out k_out", q_weight, k_weight, freq, positions, cu_seqlens, q_out, k_out)
    return kda_qk_norm_params(q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(freq) if R else None, _ptr(positions),
                              _ptr(q_out), _ptr(k_out), q_stride, k_stride, N, T, Hq, Hk, D, R, _ptr(cu_seqlens), eps, dtype,
                              1 if interleaved else 0)


def qk_norm_fwd(q, k, q_weight=None, k_weight=None, freq=None, *, positions=None, cu_seqlens=None, eps=1e-6, interleaved=False,
                q_out=None, k_out=None, stream=None):
    """Norms of queries and keys per head and the position rotation; returns ``(q_out, k_out)``.

    q [B, T, q_heads, D], k [B, T, k_heads, D] bf16 or fp32, D up to 256: each row divided by its root mean
    square and times q_weight or k_weight (fp32 [D]; None: not normed), then pairs of its first R channels
    turned by position * freq (:func:`rope_frequencies`, R = 2 len(freq); None: not turned): channels
    (i, i + R / 2), or (2 i, 2 i + 1) with ``interleaved``. ``positions`` int32 [B, T]; None: the token's index in
    its sequence. ``q_out`` may be q and ``k_out`` may be k where those are contiguous.
    """
    p = _norm_check(q, k, q_weight, k_weight, freq, positions, cu_seqlens, eps, interleaved, q_out, k_out)
    _place(q, (k, q_weight, k_weight, freq, positions, cu_seqlens, q_out, k_out))
    if q_out is None:
        q_out = _like(q)
    if k_out is None:
        k_out = _like(k)
    p.q_out, p.k_out = _ptr(q_out), _ptr(k_out)
    _call("kda_qk_norm_fwd", p, q, stream)
    return q_out, k_out


def qk_norm_bwd(q, k, q_weight, k_weight, freq, dq_out, dk_out, *, positions=None, cu_seqlens=None, eps=1e-6, interleaved=False,
                stream=None):
    """Backward of :func:`qk_norm_fwd`: same inputs plus the gradients of its results. Returns ``(dq, dk, dq_weight,
    dk_weight)``, the last two fp32, None where the weight is."""
    torch = sys.modules["torch"]

    f = _norm_check(q, k, q_weight, k_weight, freq, positions, cu_seqlens, eps, interleaved, None, None)
    _want(dq_out, "dq_out", q.shape, q.dtype)
    _want(dk_out, "dk_out", k.shape, q.dtype)
    _dense("dq_out dk_out", dq_out, dk_out)
    _place(q, (k, q_weight, k_weight, freq, positions, cu_seqlens, dq_out, dk_out))
    dq, dk = _like(q), _like(k)
    dqw, dkw = (None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
    p = kda_qk_norm_bwd_params(f, _ptr(dq_out), _ptr(dk_out), _ptr(dq), _ptr(dk), _ptr(dqw), _ptr(dkw), None, 0)
    _call("kda_qk_norm_bwd", p, q, stream, workspace=True)
    return dq, dk, dqw, dkw


def qk_norm_step(q, k, v, cache, block_table, lens, q_weight=None, k_weight=None, freq=None, *, positions=None, cu_seqlens=None,
                 eps=1e-6, interleaved=False, q_out=None, stream=None):
    """:func:`qk_norm_fwd` on the new tokens of the cache's sequences, k after norm and rotation and v
    [B, T, k_heads, D] as it is going straight into the cache (:func:`kv_cache_write`). Positions are those in the
    cache unless ``positions`` gives others for the rotation. Returns q_out."""
    f = _norm_check(q, k, q_weight, k_weight, freq, positions, cu_seqlens, eps, interleaved, q_out, None)
    shape = q.shape
    Hv, v_stride = _heads(v, "v", shape[0], shape[1], shape[3], q.dtype)
    c = _cache(cache, block_table, lens, f.B, q.dtype)
    if Hv != f.k_heads or c.heads != f.k_heads or c.D != f.D:
        raise ValueError("k, v and the cache must have the same heads and channels")
    _place(q, (k, v, q_weight, k_weight, freq, positions, cu_seqlens, q_out, *cache, block_table, lens))
    if q_out is None:
        q_out = _like(q)
        f.q_out = q_out.data_ptr()
    p = kda_qk_norm_step_params(f, _ptr(v), v_stride, c)
    _call("kda_qk_norm_step", p, q, stream)
    return q_out


# ---- attention over the cache -------------------------------------------------------------------

def paged_attn_step(q, cache, block_table, lens, *, scale=None, want_lse=False, o=None, lse=None, stream=None):
    """Attention of the next tokens of B sequences over the cache, in which their keys and values already lie.

    q [B, T, q_heads, D] bf16 or fp32, T typically 1, q_heads a multiple of the cache's heads (query head h
    reads key head h // (q_heads // heads)): token t of a sequence attends to the positions below
    lens - T + t + 1, with softmax(scale q . k), ``scale`` D ** -0.5 by default. A token that sees nothing gives
    zeros. Returns o like q, or ``(o, lse)`` with ``want_lse`` or a given ``lse``: lse fp32 [B, T, q_heads], the logarithm of the
    sum of e^score (-inf where nothing is seen), with which results over several caches can be joined.
    """
    torch = sys.modules["torch"]

    shape, kind = q.shape, q.dtype
    if len(shape) != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, Hq, D = shape
    dtype = _dtype(q, "q")
    stride = _tokens(q, "q", B, T, Hq, D)
    c = _cache(cache, block_table, lens, B, kind)
    if c.D != D or Hq < 1 or Hq % c.heads != 0:
        raise ValueError("q must have the cache's channels and a multiple of its heads")
    if scale is None:
        scale = D ** -0.5
    if o is not None:
        _want(o, "o", shape, kind)
    if lse is not None:
        _want(lse, "lse", (B, T, Hq), torch.float32)
    _dense("o lse", o, lse)
    _place(q, (o, lse, *cache, block_table, lens))
    if o is None:
        o = _like(q)
    if want_lse and lse is None:
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=q.device)
    p = kda_attn_step_params(_ptr(q), _ptr(o), _ptr(lse), stride, B, T, Hq, scale, dtype, c, None, 0)
    _call("kda_attn_step", p, q, stream, workspace=True)
    return o if lse is None else (o, lse)
