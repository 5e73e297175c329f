"""Binding of the serving operators in ``include/attn_paged.h``: rotary positions, the paged
K/V cache's write and read-back, and attention of new tokens over the paged cache.

Argument marshalling only, as in ``binding``.  Tensors may be views as long as their last
dimension is contiguous (slices of a fused projection, a cache interleaved page by page);
the others' strides are passed on.  All tensors of a call are on one CUDA device, which
need not be the current one; the work goes to that device's current stream unless
``stream`` is given.  Outputs that a call allocates belong to the stream that it works on:
memory that another stream may still be using is not taken for them, and a fill that they
need is ordered before the kernel.  A caller who hands ``stream`` orders the inputs' producers
and the outputs' users against it, as for any work on a second stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import binding
from .binding import ATTN_OK, AttnError

_BF16, _F32, _E4M3 = 0, 1, 2
_vp, _i, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong


class _Cache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("page_stride", _ll),
                ("num_pages", _i), ("page_size", _i), ("Hkv", _i), ("d", _i), ("dtype", _i)]


class _Batch(ctypes.Structure):
    _fields_ = [("cu_q", _vp), ("kv_len", _vp), ("block_table", _vp), ("B", _i), ("T", _i), ("max_pages", _i)]


class _Rope(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("rot", _i), ("interleaved", _i), ("mscale", ctypes.c_float)]


class _Strides(ctypes.Structure):
    _fields_ = [("batch", _ll), ("head", _ll), ("token", _ll)]


def declare(L):
    """Signatures of the serving entry points on a loaded library."""
    f, sz = ctypes.c_float, ctypes.c_size_t
    ps, pc, pb, pr = (ctypes.POINTER(t) for t in (_Strides, _Cache, _Batch, _Rope))
    L.attn_rope.argtypes = [_vp, ps, _vp, ps, _i, _vp, ps, _vp, ps, _i, _i, _i, _i, _i, _vp, _ll, pr, _i, _vp]
    L.attn_rope.restype = _i
    L.attn_cache_write.argtypes = [pc, pb, _vp, ps, _vp, ps, pr, _vp, ps, _vp, ps, _i, _vp]
    L.attn_cache_write.restype = _i
    L.attn_cache_read.argtypes = [pc, pb, _vp, _vp, _i, _vp]
    L.attn_cache_read.restype = _i
    L.attn_paged_workspace_size.argtypes = [_i, _i, _i, _i, _i]
    L.attn_paged_workspace_size.restype = sz
    L.attn_paged.argtypes = [_vp, ps, pc, pb, _vp, _vp, _i, f, _i, _i, _vp, sz, _vp]
    L.attn_paged.restype = _i
    return L


_same_device = contextlib.nullcontext()
_bf16, _f32, _i32, _e4m3 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn


def _on(index):
    """Context with device ``index`` current (nothing to do where it is already)."""
    return _same_device if index == torch.cuda.current_device() else torch.cuda.device(index)


def _stream(stream, index):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(index)       # torch.cuda.current_stream, without the object


def _new(like, shape, dtype, stream, zero=False):
    """An output on like's device, in memory of the call's stream and, with zero, filled on it."""
    make = like.new_zeros if zero else like.new_empty
    if stream is None:
        return make(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype)


def _tensor(t, name, dtype, index=None, dim=None, contiguous=False):
    """Raise unless t is such a tensor; a decoding step checks a dozen, so the good case is one
    expression."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and (index is None or t.get_device() == index)
            and (dim is None or t.dim() == dim) and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{index}")
    if dim is not None and t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    if contiguous:
        raise ValueError(f"{name} must be contiguous")
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _strides(t):
    """Strides of a packed [T, H, d] or dense [B, H, N, d] tensor.  The stride of a dimension of
    one entry is never followed and may be anything in torch: zero here."""
    st, sh = t.stride(), t.shape
    if len(sh) == 3:
        return _Strides(0, st[1] if sh[1] > 1 else 0, st[0] if sh[0] > 1 else 0)
    return _Strides(st[0] if sh[0] > 1 else 0, st[1] if sh[1] > 1 else 0, st[2] if sh[2] > 1 else 0)


_no_strides = _Strides()


def _rope_struct(inv_freq, interleaved, mscale, index):
    _tensor(inv_freq, "inv_freq", torch.float64, index, 1, contiguous=True)
    return _Rope(inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0, mscale)


def _check_out(out, like, name, index):
    _tensor(out, name, like.dtype, index)
    if out.shape != like.shape:
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(out.shape)}")


def rope_inv_freq(rot, base=10000.0, *, scaling=None, factor=1.0, original=None, beta_fast=32.0, beta_slow=1.0,
                  device="cuda"):
    """Frequencies of the rotary pairs, ``(inv_freq fp64 [rot / 2], mscale)`` for attn_rope
    and attn_cache_write: inv_freq[i] = base^(-2i / rot), scaled for contexts ``factor`` times
    as long as the ``original`` ones.

    scaling: None; ``"linear"``, positions compressed by factor; ``"ntk"``, the base raised so
    that the slowest pair is slowed by factor and the fastest keeps its pace; ``"yarn"``, pairs
    that turn more than beta_fast times over the original length keep their pace, those that
    turn less than beta_slow times are slowed by factor, the others in between, and outputs
    grow by 0.1 ln(factor) + 1 (mscale; 1 otherwise).
    """
    if rot < 16 or rot % 16:
        raise ValueError("rot must be a multiple of 16, at least 16")
    if not (base > 1 and factor >= 1):
        raise ValueError("base must exceed 1 and factor must be at least 1")
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    mscale = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-i / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if not original:
            raise ValueError("yarn needs the original context length")
        if not beta_fast > beta_slow > 0:
            raise ValueError("yarn needs beta_fast > beta_slow > 0")
        # pair index at which the original length holds `turns` turns
        at = [rot * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (beta_fast, beta_slow)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        slow = ((i / 2 - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - slow) + f / factor * slow
        mscale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    return f.to(device), mscale


def _rope_call(name, inverse, q, k, positions, inv_freq, interleaved, mscale, q_out, k_out, stream):
    if not isinstance(q, torch.Tensor) or (q.dtype is not _bf16 and q.dtype is not _f32):
        raise TypeError("q must be a bfloat16 or float32 tensor")
    dt = q.dtype
    _tensor(q, "q", dt)
    dev = q.get_device()
    sh = q.shape
    if len(sh) == 4:
        B, Hq, N, d = sh
    elif len(sh) == 3:
        (N, Hq, d), B = sh, 1
    else:
        raise ValueError("q must be [B, H, N, d] or [T, H, d]")
    Hkv, kp, kop, ks, kos = 0, None, None, _no_strides, _no_strides
    if k is not None:
        _tensor(k, "k", dt, dev, len(sh))
        Hkv = k.shape[1]
        if k.shape != ((B, Hkv, N, d) if len(sh) == 4 else (N, Hkv, d)):
            raise ValueError("k must have q's shape apart from the number of heads")
        if k_out is None:
            k_out = _new(k, k.shape, dt, stream)
        else:
            _check_out(k_out, k, "k_out", dev)
        kp, kop, ks, kos = k.data_ptr(), k_out.data_ptr(), _strides(k), _strides(k_out)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _tensor(positions, "positions", _i32, dev, contiguous=True)
    per_batch = positions.dim() == 2
    if positions.shape != ((B, N) if per_batch and len(sh) == 4 else (N,)):
        raise ValueError("positions must have one entry per token: [N], or [B, N] for dense tensors")
    rope = _rope_struct(inv_freq, interleaved, mscale, dev)
    if q_out is None:
        q_out = _new(q, sh, dt, stream)
    else:
        _check_out(q_out, q, "q_out", dev)
    with _on(dev):
        rc = binding.lib().attn_rope(
            q.data_ptr(), _strides(q), q_out.data_ptr(), _strides(q_out), Hq, kp, ks, kop, kos, Hkv,
            _BF16 if dt is _bf16 else _F32, B, N, d, positions.data_ptr(), N if per_batch else 0, rope, inverse,
            _stream(stream, dev))
    if rc != ATTN_OK:
        raise AttnError(rc, name)
    return q_out, k_out


def attn_rope(q, k=None, *, positions, inv_freq, interleaved=False, mscale=1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions of q and k in one launch; returns (q_out, k_out).

    q: [B, Hq, N, d] or packed [T, Hq, d], bf16 or fp32; k (optional): the same with its own
    heads; positions: int32 [N] or [B, N] ([T] when packed); inv_freq: fp64 [rot / 2], radians
    per position (``rope_inv_freq``).  The first rot of d columns turn, the rest is copied; the
    outputs are multiplied by mscale.  interleaved: pairs (2i, 2i+1) instead of (i, i + rot/2).
    q_out may be q, k_out may be k.
    """
    return _rope_call("attn_rope", 0, q, k, positions, inv_freq, interleaved, mscale, q_out, k_out, stream)


def attn_rope_bwd(dq, dk=None, *, positions, inv_freq, interleaved=False, mscale=1.0, dq_out=None, dk_out=None,
                  stream=None):
    """Gradients of attn_rope's inputs from those of its outputs (the transposed rotation, same
    arguments); returns (dq_out, dk_out), which may be the inputs themselves."""
    return _rope_call("attn_rope_bwd", 1, dq, dk, positions, inv_freq, interleaved, mscale, dq_out, dk_out, stream)


def _cache_struct(k_cache, v_cache, k_scale, v_scale):
    if not isinstance(k_cache, torch.Tensor) or (k_cache.dtype is not _bf16 and k_cache.dtype is not _e4m3):
        raise TypeError("k_cache must be a bfloat16 or float8_e4m3fn tensor")
    dt = k_cache.dtype
    _tensor(k_cache, "k_cache", dt, None, 4)
    dev = k_cache.get_device()
    _tensor(v_cache, "v_cache", dt, dev, 4)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape, [num_pages, Hkv, page_size, d]")
    pages, Hkv, page, d = shape
    stride = Hkv * page * d
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        if pages > 1:
            stride = k_cache.stride(0)
            if v_cache.stride(0) != stride:
                raise ValueError("k_cache and v_cache must have one page stride")
        for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            if (Hkv > 1 and t.stride(1) != page * d) or (page > 1 and t.stride(2) != d):
                raise ValueError(f"{n}: a page must be contiguous")
    ks = vs = None
    if dt is _e4m3:
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _tensor(t, n, torch.uint8, dev, 3, contiguous=True)
            if t.shape != shape[:3]:
                raise ValueError(f"{n} must be [num_pages, Hkv, page_size]")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("a bfloat16 cache has no scales")
    return _Cache(k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, stride, pages, page, Hkv, d,
                  _E4M3 if dt is _e4m3 else _BF16), dev, Hkv, d


def _batch_struct(block_table, cu_q, kv_len, T, dev):
    _tensor(block_table, "block_table", _i32, dev, 2, contiguous=True)
    _tensor(kv_len, "kv_len", _i32, dev, 1, contiguous=True)
    B = kv_len.shape[0]
    rows, width = block_table.shape
    if rows != B:
        raise ValueError("block_table must have a row per sequence")
    cu = None
    if cu_q is not None:
        _tensor(cu_q, "cu_q", _i32, dev, 1, contiguous=True)
        if cu_q.shape[0] != B + 1:
            raise ValueError("cu_q must have one entry more than kv_len")
        cu = cu_q.data_ptr()
    return _Batch(cu, kv_len.data_ptr(), block_table.data_ptr(), B, T, width)


def attn_cache_write(k, v, k_cache, v_cache, block_table, cu_q, kv_len, *, k_scale=None, v_scale=None, inv_freq=None,
                     interleaved=False, mscale=1.0, q=None, q_out=None, stream=None):
    """Write the new tokens' K and V [T, Hkv, d] (bf16, packed) into the paged cache, in place.

    k_cache, v_cache: [num_pages, Hkv, page_size, d], bf16, or float8_e4m3fn with k_scale,
    v_scale uint8 [num_pages, Hkv, page_size] (powers of two, 2^(byte - 127), one per token and
    head); block_table: int32 [B, max_pages]; cu_q: int32 [B + 1]; kv_len: int32 [B], the new
    tokens included.  With inv_freq, K is rotated on its way by each token's position, and so
    is q [T, Hq, d] if given, into q_out (allocated if None; may be q), all in one launch.
    Returns q_out (None without q).
    """
    cache, dev, Hkv, d = _cache_struct(k_cache, v_cache, k_scale, v_scale)
    _tensor(k, "k", _bf16, dev, 3)
    _tensor(v, "v", _bf16, dev, 3)
    T = k.shape[0]
    if k.shape != (T, Hkv, d) or v.shape != (T, Hkv, d):
        raise ValueError("k and v must be [T, Hkv, d] with the cache's heads and head size")
    batch = _batch_struct(block_table, cu_q, kv_len, T, dev)
    rope = None if inv_freq is None else _rope_struct(inv_freq, interleaved, mscale, dev)
    Hq, qp, qop, qs, qos = 0, None, None, _no_strides, _no_strides
    if q is not None:
        if rope is None:
            raise ValueError("q is rotated only: give inv_freq")
        _tensor(q, "q", _bf16, dev, 3)
        Hq = q.shape[1]
        if q.shape != (T, Hq, d):
            raise ValueError("q must be [T, Hq, d]")
        if q_out is None:
            q_out = _new(q, q.shape, _bf16, stream)
        else:
            _check_out(q_out, q, "q_out", dev)
        qp, qop, qs, qos = q.data_ptr(), q_out.data_ptr(), _strides(q), _strides(q_out)
    elif q_out is not None:
        raise ValueError("q_out without q")
    with _on(dev):
        rc = binding.lib().attn_cache_write(cache, batch, k.data_ptr(), _strides(k), v.data_ptr(), _strides(v), rope,
                                            qp, qs, qop, qos, Hq, _stream(stream, dev))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_write")
    return q_out


def attn_cache_read(k_cache, v_cache, block_table, kv_len, *, k_scale=None, v_scale=None, N=None, k_out=None,
                    v_out=None, stream=None):
    """Positions [0, min(kv_len[b], N)) of every sequence as dense bf16 [B, Hkv, N, d], the
    layout of attn_fwd and attn_decode; returns (k_out, v_out).

    Rows behind a sequence's length keep what k_out and v_out hold (zeros where they are
    allocated here, which needs N).
    """
    cache, dev, Hkv, d = _cache_struct(k_cache, v_cache, k_scale, v_scale)
    batch = _batch_struct(block_table, None, kv_len, 0, dev)
    if N is None:
        if k_out is None:
            raise ValueError("give N or k_out and v_out")
        N = k_out.shape[2]
    shape = (batch.B, Hkv, int(N), d)
    if k_out is None:
        k_out = _new(kv_len, shape, _bf16, stream, zero=True)
    if v_out is None:
        v_out = _new(kv_len, shape, _bf16, stream, zero=True)
    for t, n in ((k_out, "k_out"), (v_out, "v_out")):
        _tensor(t, n, _bf16, dev, 4, contiguous=True)
        if t.shape != shape:
            raise ValueError(f"{n} must have shape {shape}")
    with _on(dev):
        rc = binding.lib().attn_cache_read(cache, batch, k_out.data_ptr(), v_out.data_ptr(), int(N),
                                           _stream(stream, dev))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_cache_read")
    return k_out, v_out


def attn_paged_workspace_size(T, B, Hq, Hkv, d) -> int:
    return int(binding.lib().attn_paged_workspace_size(T, B, Hq, Hkv, d))


def attn_paged(q, k_cache, v_cache, block_table, cu_q, kv_len, *, k_scale=None, v_scale=None, o=None, lse=None,
               scale=None, causal=True, window_left=None, workspace=None, stream=None):
    """Attention of packed new tokens q [T, Hq, d] (bf16) over the paged cache; returns
    (o bf16 [T, Hq, d], lse fp32 [T, Hq]).

    Token t of sequence b has position kv_len[b] - cu_q[b+1] + t and sees the cached keys up
    to it (causal), no further back than window_left positions (None or negative: no limit).
    Rows that see no key get o = 0 and lse = -inf; rows from cu_q[B] on are left alone.
    The kernel is picked by the mean number of new tokens, T / B: a long chunk among mostly
    empty sequences is better called without them (include/attn_paged.h).
    workspace: a device tensor of attn_paged_workspace_size(T, B, Hq, Hkv, d) bytes, one for
    each call that may run at the same time; None lets the library allocate it on the stream.
    """
    cache, dev, _, dc = _cache_struct(k_cache, v_cache, k_scale, v_scale)
    _tensor(q, "q", _bf16, dev, 3)
    T, Hq, d = q.shape
    if d != dc:
        raise ValueError("q and the cache differ in head size")
    batch = _batch_struct(block_table, cu_q, kv_len, T, dev)
    if o is None:
        o = _new(q, (T, Hq, d), _bf16, stream)
    else:
        _tensor(o, "o", _bf16, dev, 3, contiguous=True)
        if o.shape != (T, Hq, d):
            raise ValueError("o must be [T, Hq, d]")
    if lse is None:
        lse = _new(q, (T, Hq), _f32, stream)
    else:
        _tensor(lse, "lse", _f32, dev, 2, contiguous=True)
        if lse.shape != (T, Hq):
            raise ValueError("lse must be [T, Hq]")
    ws, ws_bytes = None, 0
    if workspace is not None:
        if not workspace.is_cuda or workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous and on the call's device")
        ws, ws_bytes = workspace.data_ptr(), workspace.nbytes
    with _on(dev):
        rc = binding.lib().attn_paged(q.data_ptr(), _strides(q), cache, batch, o.data_ptr(), lse.data_ptr(), Hq,
                                      d ** -0.5 if scale is None else scale, 1 if causal else 0,
                                      -1 if window_left is None else max(-1, min(window_left, 1 << 30)), ws, ws_bytes,
                                      _stream(stream, dev))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_paged")
    return o, lse
