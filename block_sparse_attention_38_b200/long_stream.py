"""Long streams: a key/value cache held in 4 bits and decode steps over long
caches, with a sliding window and first tokens that stay visible (sinks) or
with a block pattern.  Marshalling only, as in the rest of the binding; the
functions are those of the last section of include/bsa.h.

H query heads share Hkv cached heads: query head h reads cached head
h // (H // Hkv).
"""
from __future__ import annotations

import ctypes
import math
from typing import NamedTuple, Optional

from . import BsaError, _check, library  # noqa: F401  (defined before this module is imported)

torch = None  # imported by the first call that takes tensors: the package loads without it


def _load():
    global torch
    import torch as module

    torch = module


_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


class _View(ctypes.Structure):
    _fields_ = [("data", _vp), ("stride_b", _i64), ("stride_h", _i64), ("stride_n", _i64)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_codes", _vp), ("k_params", _vp), ("v_codes", _vp), ("v_params", _vp),
                ("B", _i32), ("H", _i32), ("L", _i32), ("d", _i32)]


def _declare(lib) -> None:
    """Argument types of this module's entry points (called once by library())."""
    i, f, view, cache = ctypes.c_int, ctypes.c_float, ctypes.POINTER(_View), ctypes.POINTER(_Cache)
    for name, types in (
            ("bsa_q4_write", [cache, view, view, _vp, _vp, i, _vp]),
            ("bsa_q4_read", [cache, _vp, _vp, i, _vp, _vp, _vp]),
            ("bsa_q4_decode", [_vp, _vp, _vp, cache, _vp, _vp, _vp, i, i, f, _vp, _vp, _vp]),
            ("bsa_q4_window_decode", [_vp, _vp, _vp, cache, _vp, i, i, i, f, _vp, _vp, _vp]),
            ("bsa_window_decode", [_vp] * 6 + [i] * 7 + [f, _vp, _vp, _vp]),
            ("bsa_window_forward", [view] * 3 + [_vp] + [i] * 7 + [f, view, _vp, _vp]),
            ("bsa_window_backward", [view] * 5 + [_vp, _vp] + [i] * 7 + [f] + [view] * 3
             + [_vp, ctypes.c_size_t, _vp]),
            ("bsa_stream_status", [ctypes.POINTER(ctypes.c_uint32), i])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, types
    lib.bsa_window_backward_workspace_bytes.restype = ctypes.c_size_t
    lib.bsa_window_backward_workspace_bytes.argtypes = [i] * 7


class Q4Cache(NamedTuple):
    """The four tensors of a 4-bit cache of Hkv heads: codes uint8 [B, Hkv, L, d/2]
    and parameters fp16 [B, Hkv, L, d/32, 2] (scale, minimum), for keys and values."""

    k_codes: "torch.Tensor"  # noqa: F821
    k_params: "torch.Tensor"  # noqa: F821
    v_codes: "torch.Tensor"  # noqa: F821
    v_params: "torch.Tensor"  # noqa: F821


def q4_cache(B: int, Hkv: int, L: int, d: int, device="cuda") -> Q4Cache:
    """A 4-bit cache with room for L tokens of B sequences; every row reads back as 0."""
    if torch is None:
        _load()
    def codes():
        return torch.zeros((B, Hkv, L, d // 2), dtype=torch.uint8, device=device)

    def params():
        return torch.zeros((B, Hkv, L, d // 32, 2), dtype=torch.float16, device=device)

    return Q4Cache(codes(), params(), codes(), params())


# The checks below run on every call and cost as much as a small kernel, so they
# stick to cheap attributes: `dev` is a CUDA device's index.


def _ints(name, t, n, dev):
    if t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n} entries on cuda:{dev}")
    return t.data_ptr()


def _rows(name, t, shape, dev, dtype):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{dev}")
    return t.data_ptr()


def _cache_arg(cache):
    """(ctypes struct, B, Hkv, L, d, device index) of a checked Q4Cache."""
    kc, kp, vc, vp = cache
    shape = kc.shape
    if len(shape) != 4:
        raise ValueError("k_codes must be [B, Hkv, L, d/2]")
    B, H, L, half = shape
    dev = kc.get_device()
    if dev < 0:
        raise ValueError("the cache's tensors must be CUDA tensors")
    params = (B, H, L, half // 16, 2)
    return (_Cache(_rows("k_codes", kc, shape, dev, torch.uint8), _rows("k_params", kp, params, dev, torch.float16),
                   _rows("v_codes", vc, shape, dev, torch.uint8), _rows("v_params", vp, params, dev, torch.float16),
                   B, H, L, 2 * half), B, H, L, 2 * half, dev)


def _view(name, t, shape, dev):
    """bsa_view of a bf16 tensor whose last dimension is contiguous."""
    if t.shape != shape or t.dtype is not torch.bfloat16 or t.get_device() != dev:
        raise ValueError(f"{name} must be a bf16 tensor {list(shape)} on cuda:{dev}, got {list(t.shape)}")
    sb, sh, sn, sd = t.stride()
    # the stride of a dimension of one entry is never used
    if shape[0] == 1:
        sb = 0
    if shape[1] == 1:
        sh = 0
    if shape[2] == 1:
        sn = 0
    if sd != 1 or (sb | sh | sn) & 7:
        raise ValueError(f"{name} must have a contiguous last dimension and other strides that are "
                         "multiples of 8")
    return _View(t.data_ptr(), sb, sh, sn)


def _call(dev, name, *args):
    """The library function `name` with device `dev` current, on its current stream."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(library(), name)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if rc:
        _check(rc, name)


_functions = {}


def q4_write(cache: Q4Cache, k, v, start, lens=None) -> None:
    """Quantises rows into the cache (bsa_q4_write): row i of k, v (CUDA bf16
    [B, Hkv, T, d], any strides that are multiples of 8 with d contiguous)
    becomes cached row start[b] + i, for i < lens[b] (T where lens is None).

    start, lens: CUDA int32 [B].  One token of each sequence is T = 1 with
    start its position; other cached rows stay as they were.
    """
    if torch is None:
        _load()
    arg, B, H, L, d, dev = _cache_arg(cache)
    if k.dim() != 4:
        raise ValueError("k, v must be [B, Hkv, T, d]")
    shape = (B, H, k.shape[2], d)
    kv, vv = _view("k", k, shape, dev), _view("v", v, shape, dev)
    _call(dev, "bsa_q4_write", arg, kv, vv, _ints("start", start, B, dev),
          None if lens is None else _ints("lens", lens, B, dev), shape[2])


def q4_read(cache: Q4Cache, start, T: int, lens=None, out=None):
    """The cached rows start[b] .. start[b] + T - 1 as bf16 (k, v), each
    [B, Hkv, T, d] contiguous (bsa_q4_read); rows from lens[b] on are zero.

    out: a pair of tensors to write into.
    """
    if torch is None:
        _load()
    arg, B, H, L, d, dev = _cache_arg(cache)
    shape = (B, H, int(T), d)
    if out is None:
        k = cache.k_codes.new_empty(shape, dtype=torch.bfloat16)
        v = torch.empty_like(k)
    else:
        k, v = out
    _call(dev, "bsa_q4_read", arg, _ints("start", start, B, dev),
          None if lens is None else _ints("lens", lens, B, dev), shape[2],
          _rows("out k", k, shape, dev, torch.bfloat16), _rows("out v", v, shape, dev, torch.bfloat16))
    return k, v


def _step(q, B, Hkv, d, dev, k_new, v_new, scale, out, lse):
    """Checked pieces every decode step shares: (q, k_new, v_new pointers, H, scale, O, LSE)."""
    bf16 = torch.bfloat16
    if q.dim() != 3 or q.shape[0] != B or q.shape[2] != d or q.shape[1] % max(Hkv, 1):
        raise ValueError("q must be [B, H, d] with the cache's B and d, and H a multiple of its heads")
    H = q.shape[1]
    if (k_new is None) != (v_new is None):
        raise ValueError("give both k_new and v_new, or neither")
    qp = _rows("q", q, (B, H, d), dev, bf16)
    kn = vn = None
    if k_new is not None:
        kn, vn = (_rows(n, t, (B, Hkv, d), dev, bf16) for n, t in (("k_new", k_new), ("v_new", v_new)))
    if out is None:
        out = torch.empty_like(q)
    else:
        _rows("out", out, (B, H, d), dev, bf16)
    if lse is None:
        lse = q.new_empty((B, H), dtype=torch.float32)
    else:
        _rows("lse", lse, (B, H), dev, torch.float32)
    return qp, kn, vn, H, 1.0 / math.sqrt(d) if scale is None else float(scale), out, lse


def q4_decode(q, cache: Q4Cache, seq_len, row_ptr, col_idx, block_size: int, scale: Optional[float] = None,
              k_new=None, v_new=None, out=None, lse=None):
    """One decode step over a 4-bit cache by a block pattern (bsa_q4_decode).

    q: CUDA bf16 [B, H, d]; seq_len: CUDA int32 [B], tokens including the new
    one; row_ptr, col_idx: CUDA int32 block-CSR over the cached heads' L //
    block_size block rows.  With k_new, v_new (bf16 [B, Hkv, d]) the new token is
    quantised into row seq_len[b] - 1 first.  Returns (O bf16 [B, H, d], LSE
    fp32 [B, H]).
    """
    if torch is None:
        _load()
    arg, B, Hkv, L, d, dev = _cache_arg(cache)
    qp, kn, vn, H, scale, out, lse = _step(q, B, Hkv, d, dev, k_new, v_new, scale, out, lse)
    rp = _ints("row_ptr", row_ptr, Hkv * (L // int(block_size)) + 1, dev)
    ci = _ints("col_idx", col_idx, col_idx.numel(), dev) if col_idx.numel() else rp
    _call(dev, "bsa_q4_decode", qp, kn, vn, arg, rp, ci, _ints("seq_len", seq_len, B, dev), H,
          int(block_size), scale, out.data_ptr(), lse.data_ptr())
    return out, lse


def q4_window_decode(q, cache: Q4Cache, seq_len, window: int, sinks: int = 0, scale: Optional[float] = None,
                     k_new=None, v_new=None, out=None, lse=None):
    """One decode step over a 4-bit cache with a sliding window (bsa_q4_window_decode):
    the rows k <= t = seq_len[b] - 1 with k > t - window or k < sinks; window >= L
    sees every row.  Arguments and result as `q4_decode`."""
    if torch is None:
        _load()
    arg, B, Hkv, L, d, dev = _cache_arg(cache)
    qp, kn, vn, H, scale, out, lse = _step(q, B, Hkv, d, dev, k_new, v_new, scale, out, lse)
    _call(dev, "bsa_q4_window_decode", qp, kn, vn, arg, _ints("seq_len", seq_len, B, dev), H, int(window),
          int(sinks), scale, out.data_ptr(), lse.data_ptr())
    return out, lse


def window_decode(q, k_cache, v_cache, seq_len, window: int, sinks: int = 0, scale: Optional[float] = None,
                  k_new=None, v_new=None, out=None, lse=None):
    """One decode step over a bf16 cache [B, Hkv, L, d] with a sliding window
    (bsa_window_decode); arguments and result as `q4_window_decode`."""
    if torch is None:
        _load()
    if k_cache.dim() != 4:
        raise ValueError("the caches must be [B, Hkv, L, d]")
    B, Hkv, L, d = k_cache.shape
    dev = k_cache.get_device()
    if dev < 0:
        raise ValueError("the caches must be CUDA tensors")
    kc, vc = (_rows(n, t, (B, Hkv, L, d), dev, torch.bfloat16)
              for n, t in (("k_cache", k_cache), ("v_cache", v_cache)))
    qp, kn, vn, H, scale, out, lse = _step(q, B, Hkv, d, dev, k_new, v_new, scale, out, lse)
    _call(dev, "bsa_window_decode", qp, kn, vn, kc, vc, _ints("seq_len", seq_len, B, dev), B, H, Hkv, L, d,
          int(window), int(sinks), scale, out.data_ptr(), lse.data_ptr())
    return out, lse


def _heads(q, k):
    """(B, H, Hkv, N, d) of [B, H, N, d] queries and [B, Hkv, N, d] keys."""
    if q.dim() != 4 or k.dim() != 4 or q.shape[1] % max(int(k.shape[1]), 1):
        raise ValueError("q must be [B, H, N, d] and k, v [B, Hkv, N, d], H a multiple of Hkv")
    B, H, N, d = q.shape
    return B, H, k.shape[1], N, d


def window_forward(q, k, v, window: int, sinks: int = 0, scale: Optional[float] = None, lens=None, out=None,
                   lse=None):
    """Attention with a sliding window and first tokens that stay visible
    (bsa_window_forward): query i sees the keys k <= i with k > i - window or k < sinks.

    q: CUDA bf16 [B, H, N, d]; k, v: [B, Hkv, N, d]; any strides that are
    multiples of 8 with d contiguous and rows that do not overlap, so a
    sequence-major tensor is passed as its transpose(1, 2).  lens: CUDA int32
    [B], tokens of each sequence (all N where None); rows past them give O = 0
    and LSE = -inf.  Returns (O like q, LSE fp32 [B, H, N]).
    """
    if torch is None:
        _load()
    B, H, Hkv, N, d = _heads(q, k)
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    qv = _view("q", q, (B, H, N, d), dev)
    kv, vv = _view("k", k, (B, Hkv, N, d), dev), _view("v", v, (B, Hkv, N, d), dev)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = q.new_empty((B, H, N), dtype=torch.float32)
    _call(dev, "bsa_window_forward", qv, kv, vv, None if lens is None else _ints("lens", lens, B, dev), B, H,
          Hkv, N, d, int(window), int(sinks), 1.0 / math.sqrt(d) if scale is None else float(scale),
          _view("out", out, (B, H, N, d), dev), _rows("lse", lse, (B, H, N), dev, torch.float32))
    return out, lse


def window_backward_workspace_bytes(B: int, H: int, Hkv: int, N: int, d: int, window: int, sinks: int = 0) -> int:
    """Workspace bytes `window_backward` needs for these sizes."""
    n = int(library().bsa_window_backward_workspace_bytes(B, H, Hkv, N, d, window, sinks))
    if n == 0:
        raise ValueError("no workspace for these sizes: check H % Hkv, d in (64, 128), window >= 1, sinks >= 0")
    return n


def window_backward(q, k, v, o, do, lse, window: int, sinks: int = 0, scale: Optional[float] = None, lens=None,
                    workspace=None):
    """Gradients of `window_forward` (bsa_window_backward): (dQ like q, dK like k,
    dV like v) for the gradient do of its output o; lse as it returned it (copied
    first where it is not contiguous).

    workspace: a CUDA tensor of at least window_backward_workspace_bytes(...)
    bytes (allocated on the current stream when not given); calls that may run
    at the same time need one each.
    """
    if torch is None:
        _load()
    B, H, Hkv, N, d = _heads(q, k)
    dev = q.get_device()
    if dev < 0:
        raise ValueError("q must be a CUDA tensor")
    qs, ks = (B, H, N, d), (B, Hkv, N, d)
    views = [_view(n, t, s, dev) for n, t, s in (("q", q, qs), ("k", k, ks), ("v", v, ks), ("o", o, qs),
                                                    ("do", do, qs))]
    lse = lse.contiguous()
    lp = _rows("lse", lse, (B, H, N), dev, torch.float32)
    nbytes = window_backward_workspace_bytes(B, H, Hkv, N, d, int(window), int(sinks))
    if workspace is None:
        workspace = q.new_empty(nbytes, dtype=torch.uint8)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on q's device")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    _call(dev, "bsa_window_backward", *views, lp, None if lens is None else _ints("lens", lens, B, dev), B, H,
          Hkv, N, d, int(window), int(sinks), 1.0 / math.sqrt(d) if scale is None else float(scale),
          _view("dq", dq, qs, dev), _view("dk", dk, ks, dev), _view("dv", dv, ks, dev),
          workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return dq, dk, dv


def stream_status(clear: bool = True) -> int:
    """OR of STATUS_* bits raised by this module's kernels on the current device (synchronises it)."""
    v = ctypes.c_uint32(0)
    _check(library().bsa_stream_status(ctypes.byref(v), int(bool(clear))), "bsa_stream_status")
    return int(v.value)
