"""fp64 oracle of the long-stream operators: the 4-bit cache, decode steps over
a window with sinks or over block rows, and sliding-window attention with its
gradients.  Plain numpy from the definitions; nothing is shared with the CUDA
path.
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def _f64(x):
    import torch

    return x.double().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)


# ------------------------------------------------------------------ 4-bit rows
def quantise(x):
    """(codes uint8 [..., d], scale fp16 [..., d/32], minimum fp16) of rows [..., d].

    scale = fp16(fp32((max - min) / 15)), minimum = fp16(min), both limited to
    +-65504; code = floor((x - minimum) / scale + 1/2) in 0..15, 0 where the scale
    is 0.  A NaN makes its group's scale and minimum NaN, with codes 0.
    """
    x = _f64(x)
    x = x.reshape(x.shape[:-1] + (x.shape[-1] // GROUP, GROUP))
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        lo, hi = x.min(-1), x.max(-1)
        wide = np.where(hi == lo, np.float32(0), (hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15))
        scale = np.where(wide > 65504, np.float32(65504), wide).astype(np.float16)
        least = np.clip(lo, -65504, 65504).astype(np.float16)
        s, m = scale.astype(np.float64)[..., None], least.astype(np.float64)[..., None]
        t = x - m
        y = t - x
        low = (x - (t - y)) - (m + y)  # x - m = t + low exactly
        code = np.clip(np.floor(t / np.where(s > 0, s, 1.0) + 0.5), 0, 15)
        bound = (code - 0.5) * s       # exact: 5 bits times 11
        code -= (code > 0) & ((t < bound) | ((t == bound) & (low < 0)))
        code = np.where(s > 0, code, 0.0)
    return code.reshape(code.shape[:-2] + (code.shape[-2] * GROUP,)).astype(np.uint8), scale, least


def values(codes, scale, least):
    """What codes [..., d] stand for, fp64."""
    c = codes.reshape(codes.shape[:-1] + (codes.shape[-1] // GROUP, GROUP)).astype(np.float64)
    v = c * scale.astype(np.float64)[..., None] + least.astype(np.float64)[..., None]
    return v.reshape(codes.shape)


def nibble_of(channel, d, is_key):
    """Place of a channel's code in its packed row, in nibbles."""
    g, c = divmod(channel, GROUP)
    run = 8 if is_key else 4
    y, i = divmod(c, run)
    return (y * (d // GROUP) + g) * run + i


def pack(codes, is_key):
    """Codes [..., d] as bytes [..., d/2] in the cache's order."""
    d = codes.shape[-1]
    nib = np.zeros_like(codes)
    for ch in range(d):
        nib[..., nibble_of(ch, d, is_key)] = codes[..., ch]
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed, is_key):
    d = packed.shape[-1] * 2
    nib = np.empty(packed.shape[:-1] + (d,), np.uint8)
    nib[..., 0::2], nib[..., 1::2] = packed & 15, packed >> 4
    return nib[..., [nibble_of(ch, d, is_key) for ch in range(d)]]


# ----------------------------------------------------------------- visible rows
def window_rows(t, window, sinks):
    """Rows that position t sees: k <= t with k > t - window or k < sinks."""
    k = np.arange(t + 1)
    return k[(k > t - window) | (k < sinks)]


def block_rows(t, row_ptr, col_idx, h, M, bs):
    """Rows <= t of the blocks that block row t // bs of head h lists."""
    r = h * M + t // bs
    cols = sorted({int(j) for j in col_idx[row_ptr[r]:row_ptr[r + 1]] if j <= t // bs})
    k = np.concatenate([np.arange(j * bs, (j + 1) * bs) for j in cols]) if cols else np.zeros(0, int)
    return k[k <= t]


# ------------------------------------------------------------------ decode step
def decode(q, k, v, seq_len, rows_of, scale):
    """q [B, H, d]; k, v [B, Hkv, L, d]; rows_of(b, cached head, t) -> rows.

    Returns (O [B, H, d], LSE [B, H]); an entry of no rows gives 0 and -inf.
    """
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, d = q.shape
    G = H // k.shape[1]
    O, L = np.zeros((B, H, d)), np.full((B, H), -np.inf)
    for b in range(B):
        t = int(seq_len[b]) - 1
        if t < 0:
            continue
        for h in range(H):
            rows = rows_of(b, h // G, t)
            if len(rows) == 0:
                continue
            x = scale * (k[b, h // G, rows] @ q[b, h])
            top = x.max()
            e = np.exp(x - top)
            O[b, h] = (e @ v[b, h // G, rows]) / e.sum()
            L[b, h] = top + np.log(e.sum())
    return O, L


# ------------------------------------------------------- sliding-window attention
def _mask(n, window, sinks):
    q, k = np.arange(n)[:, None], np.arange(n)[None]
    return (k <= q) & ((k > q - window) | (k < sinks))


def window_forward(q, k, v, window, sinks, scale, lens=None):
    """q [B, H, N, d]; k, v [B, Hkv, N, d]; rows from lens[b] on give 0 and -inf."""
    q, k, v = _f64(q), _f64(k), _f64(v)
    B, H, N, d = q.shape
    G = H // k.shape[1]
    O, L = np.zeros(q.shape), np.full((B, H, N), -np.inf)
    for b in range(B):
        n = N if lens is None else int(lens[b])
        if n == 0:
            continue
        m = _mask(n, window, sinks)
        for h in range(H):
            x = np.where(m, scale * (q[b, h, :n] @ k[b, h // G, :n].T), -np.inf)
            top = x.max(-1, keepdims=True)
            e = np.exp(x - top)
            s = e.sum(-1, keepdims=True)
            O[b, h, :n] = (e / s) @ v[b, h // G, :n]
            L[b, h, :n] = (top + np.log(s))[:, 0]
    return O, L


def window_backward(q, k, v, do, window, sinks, scale, lens=None, magnitudes=False):
    """(dQ, dK, dV) of window_forward for the output gradient do, by the chain rule.

    With magnitudes also, for each element, the sum of its terms' magnitudes, and
    what a relative error of 1 in every O element and in every term of the sum that
    it is can move the element by (through D = dO . O).
    """
    O, L = window_forward(q, k, v, window, sinks, scale, lens)
    q, k, v, do = _f64(q), _f64(k), _f64(v), _f64(do)
    B, H, N, d = q.shape
    G = H // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    size, moved = [np.zeros(x.shape) for x in (q, k, v)], [np.zeros(x.shape) for x in (q, k, v)]
    for b in range(B):
        n = N if lens is None else int(lens[b])
        if n == 0:
            continue
        m = _mask(n, window, sinks)
        for h in range(H):
            c = h // G
            x = scale * (q[b, h, :n] @ k[b, c, :n].T)
            p = np.where(m, np.exp(np.where(m, x, 0.0) - L[b, h, :n, None]), 0.0)
            g = do[b, h, :n]
            ds = p * (g @ v[b, c, :n].T - (g * O[b, h, :n]).sum(-1, keepdims=True)) * scale
            dq[b, h, :n] = ds @ k[b, c, :n]
            dk[b, c, :n] += ds.T @ q[b, h, :n]
            dv[b, c, :n] += p.T @ g
            if magnitudes:
                weight = np.abs(O[b, h, :n]) + p @ np.abs(v[b, c, :n])
                e = p * (np.abs(g) * weight).sum(-1, keepdims=True) * abs(scale)
                size[0][b, h, :n], moved[0][b, h, :n] = np.abs(ds) @ np.abs(k[b, c, :n]), e @ np.abs(k[b, c, :n])
                size[1][b, c, :n] += np.abs(ds).T @ np.abs(q[b, h, :n])
                moved[1][b, c, :n] += e.T @ np.abs(q[b, h, :n])
                size[2][b, c, :n] += p.T @ np.abs(g)
    return ((dq, dk, dv), size, moved) if magnitudes else (dq, dk, dv)
