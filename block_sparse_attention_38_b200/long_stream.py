"""Long streams: a key/value cache held in 4 bits and decode steps over long
caches, with a sliding window and first tokens that stay visible (sinks) or
with a block pattern.  Marshalling only, as in the rest of the binding; the
functions are those of the last section of include/bsa.h.  The checks of tensors
and the outputs' allocation are in _bsa_torch.so (csrc/bsa_torch.cpp): at a decode
step's sizes they take as long in Python as the kernels on the device.

H query heads share Hkv cached heads: query head h reads cached head
h // (H // Hkv).
"""
from __future__ import annotations

import ctypes
import sysconfig
from typing import NamedTuple, Optional

from . import _check, library  # defined before this module is imported

_marshal = None  # csrc/bsa_torch.cpp, loaded by the first call that takes tensors: the package loads without torch


def marshal_tag(torch_version: str) -> str:
    """What _bsa_torch.so is built for; the module has it as a constant."""
    return f"torch {torch_version}, {sysconfig.get_config_var('SOABI')}"


def _load():
    global _marshal
    import torch  # its libraries come first

    try:
        from . import _bsa_torch as module
    except ImportError as e:
        raise ImportError(f"_bsa_torch.so is missing or does not load ({e}): build it with "
                          "`python -m block_sparse_attention_38_b200.build`") from e
    made_for, here = getattr(module, "built_for", "an earlier version of this package"), marshal_tag(torch.__version__)
    if made_for != here:
        raise ImportError(f"_bsa_torch.so was built for {made_for}, not for {here}: build it with "
                          "`python -m block_sparse_attention_38_b200.build`")
    lib = library()
    module.init(_check, *(ctypes.cast(getattr(lib, "bsa_" + name), ctypes.c_void_p).value for name in (
        "q4_write", "q4_read", "q4_decode", "q4_window_decode", "window_decode", "window_forward",
        "window_backward", "window_backward_workspace_bytes")))
    _marshal = module
    return module


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
    import torch

    def codes():
        return torch.zeros((B, Hkv, L, d // 2), dtype=torch.uint8, device=device)

    def params():
        return torch.zeros((B, Hkv, L, d // 32, 2), dtype=torch.float16, device=device)

    return Q4Cache(codes(), params(), codes(), params())


def q4_write(cache: Q4Cache, k, v, start, lens=None) -> None:
    """Quantises rows into the cache (bsa_q4_write): row i of k, v (CUDA bf16
    [B, Hkv, T, d], any strides that are multiples of 8 with d contiguous)
    becomes cached row start[b] + i, for i < lens[b] (T where lens is None).

    start, lens: CUDA int32 [B].  One token of each sequence is T = 1 with
    start its position; other cached rows stay as they were.
    """
    (_marshal or _load()).q4_write(cache, k, v, start, lens)


def q4_read(cache: Q4Cache, start, T: int, lens=None, out=None):
    """The cached rows start[b] .. start[b] + T - 1 as bf16 (k, v), each
    [B, Hkv, T, d] contiguous (bsa_q4_read); rows from lens[b] on are zero.

    out: a pair of tensors to write into.
    """
    return (_marshal or _load()).q4_read(cache, start, T, lens, out)


def q4_decode(q, cache: Q4Cache, seq_len, row_ptr, col_idx, block_size: int, scale: Optional[float] = None,
              k_new=None, v_new=None, out=None, lse=None):
    """One decode step over a 4-bit cache by a block pattern (bsa_q4_decode).

    q: CUDA bf16 [B, H, d]; seq_len: CUDA int32 [B], tokens including the new
    one; row_ptr, col_idx: CUDA int32 block-CSR over the cached heads' L //
    block_size block rows.  With k_new, v_new (bf16 [B, Hkv, d]) the new token is
    quantised into row seq_len[b] - 1 first.  Returns (O bf16 [B, H, d], LSE
    fp32 [B, H]).
    """
    return (_marshal or _load()).q4_decode(q, cache, seq_len, row_ptr, col_idx, block_size, scale, k_new, v_new, out,
                                           lse)


def q4_window_decode(q, cache: Q4Cache, seq_len, window: int, sinks: int = 0, scale: Optional[float] = None,
                     k_new=None, v_new=None, out=None, lse=None):
    """One decode step over a 4-bit cache with a sliding window (bsa_q4_window_decode):
    the rows k <= t = seq_len[b] - 1 with k > t - window or k < sinks; window >= L
    sees every row.  Arguments and result as `q4_decode`."""
    return (_marshal or _load()).q4_window_decode(q, cache, seq_len, window, sinks, scale, k_new, v_new, out, lse)


def window_decode(q, k_cache, v_cache, seq_len, window: int, sinks: int = 0, scale: Optional[float] = None,
                  k_new=None, v_new=None, out=None, lse=None):
    """One decode step over a bf16 cache [B, Hkv, L, d] with a sliding window
    (bsa_window_decode); arguments and result as `q4_window_decode`."""
    return (_marshal or _load()).window_decode(q, k_cache, v_cache, seq_len, window, sinks, scale, k_new, v_new, out,
                                               lse)


def window_forward(q, k, v, window: int, sinks: int = 0, scale: Optional[float] = None, lens=None, out=None,
                   lse=None):
    """Attention with a sliding window and first tokens that stay visible
    (bsa_window_forward): query i sees the keys k <= i with k > i - window or k < sinks.

    q: CUDA bf16 [B, H, N, d]; k, v: [B, Hkv, N, d]; any strides that are
    multiples of 8 with d contiguous and rows that do not overlap, so a
    sequence-major tensor is passed as its transpose(1, 2).  lens: CUDA int32
    [B], tokens of each sequence (all N where None); rows past them may hold
    anything and give O = 0 and LSE = -inf.  Returns (O like q, LSE fp32 [B, H, N]).

    A NaN or infinity in a value row inside its sequence can also reach queries
    that do not see that row (their weight for it is 0, and 0 times NaN is NaN):
    those up to 255 tokens before it or 384 past its window and, where its 128-row
    tile holds sinks, every later one.
    """
    return (_marshal or _load()).window_forward(q, k, v, window, sinks, scale, lens, out, lse)


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

    A NaN or infinity inside a sequence can also reach gradients of rows up to 384
    tokens from those that its row meets, and of 128-row tiles with sinks.

    workspace: a CUDA tensor of at least window_backward_workspace_bytes(...)
    bytes (allocated on the current stream when not given); calls that may run
    at the same time need one each.
    """
    return (_marshal or _load()).window_backward(q, k, v, o, do, lse, window, sinks, scale, lens, workspace)


def stream_status(clear: bool = True) -> int:
    """OR of STATUS_* bits raised by this module's kernels on the current device (synchronises it)."""
    v = ctypes.c_uint32(0)
    _check(library().bsa_stream_status(ctypes.byref(v), int(bool(clear))), "bsa_stream_status")
    return int(v.value)
