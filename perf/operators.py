"""Cases, plain forms and 64-bit results of the long-stream operators: the key/value cache held in 4 bits
(written, read back and attended to) and attention with a sliding window and first tokens that stay visible.

`run(state)` makes one pass: with `own` false in elementary torch operations, with `own` true through
`block_sparse_attention_38_b200`.  Notation: H query heads share Hkv key/value heads (H = Hkv * G); a query at
position t sees the keys k <= t with k > t - window or k < sinks.
"""
import math

import torch

own = False

GROUP = 32  # channels that share one scale and one minimum in the 4-bit cache


# ----------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of each sequence goes into the cache (the smallest call: latency)
        dict(name="cache_token", op="cache", B=4, Hkv=16, d=64, L=4096, T=1, back=1, ragged=False),
        # a padded batch of short prompts, odd sizes
        dict(name="cache_prompt_ragged", op="cache", B=3, Hkv=5, d=64, L=1500, T=1003, back=1003, ragged=True),
        # the next 2048-token chunk of a long prompt is written and the whole 32K prefix read back for it
        dict(name="cache_chunk_32k", op="cache", B=1, Hkv=16, d=128, L=32768, T=2048, back=32000, ragged=False),
        # one decode step over 4 bits, shapes and pattern of decode_loglinear_4k, four query heads a cached head
        dict(name="q4_decode_4k", op="q4_decode", B=4, Hkv=4, G=4, d=64, L=4096, bs=32, kmax=6, append=True),
        # one decode step over 4 bits, shapes and pattern of decode_loglinear_32k
        dict(name="q4_decode_32k", op="q4_decode", B=8, Hkv=32, G=1, d=128, L=32768, bs=128, kmax=7, append=False),
        # the whole of a 128K cache is visible, few sequences: the long axis has to be split
        dict(name="q4_dense_128k", op="q4_window", B=2, Hkv=8, G=4, d=128, L=131072, window=131072, sinks=0,
             append=False),
        # a stream far past its window, bf16 cache, new token appended
        dict(name="window_decode", op="window_decode", B=4, Hkv=8, G=4, d=128, L=8192, window=4096, sinks=4,
             append=True),
        # a short window over 4 bits, odd sizes: latency again
        dict(name="q4_window_small", op="q4_window", B=2, Hkv=2, G=7, d=64, L=3001, window=333, sinks=5, append=True),
        # prefill of a long prompt
        dict(name="window_fwd_32k", op="window_fwd", B=1, Hkv=8, G=4, d=128, N=32768, window=1024, sinks=4,
             ragged=False, seq_major=False),
        # a padded batch, sequence-major tensors, odd sizes
        dict(name="window_fwd_ragged", op="window_fwd", B=3, Hkv=4, G=2, d=64, N=1001, window=200, sinks=1,
             ragged=True, seq_major=True),
        # training on long sequences: the gradients of the forward
        dict(name="window_bwd_8k", op="window_bwd", B=1, Hkv=8, G=4, d=128, N=8192, window=1024, sinks=4,
             ragged=False, seq_major=False),
        # a padded batch, odd sizes, window longer than some sequences
        dict(name="window_bwd_ragged", op="window_bwd", B=2, Hkv=3, G=3, d=64, N=777, window=300, sinks=3,
             ragged=True, seq_major=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["cache", "q4_decode", "q4_window", "window_decode", "window_fwd", "window_bwd"])
    d = rng.choice([64, 128])
    if op == "cache":
        Hkv, back = _log(rng, 1, 16), _log(rng, 1, 32000)
        B = _log(rng, 1, max(1, min(8, 16 * 32000 // (Hkv * back))))
        T = rng.choice([1, back, _log(rng, 1, back)])
        return dict(op=op, B=B, Hkv=Hkv, d=d, L=back + rng.randrange(0, 800), T=T, back=back,
                    ragged=rng.random() < 0.5)
    if op == "q4_decode":
        bs = rng.choice([32, 64, 128])
        return dict(op=op, B=_log(rng, 1, 8), Hkv=_log(rng, 1, 32), G=rng.choice([1, 2, 3, 4, 8]), d=d,
                    L=bs * _log(rng, 4, 256), bs=bs, kmax=rng.randrange(3, 8), append=rng.random() < 0.5)
    if op == "q4_window":
        L, Hkv = _log(rng, 16, 131072), _log(rng, 1, 8)
        B = _log(rng, 1, max(1, min(16, 16 * 131072 // (Hkv * L))))
        return dict(op=op, B=B, Hkv=Hkv, G=rng.choice([1, 2, 4, 7, 8, 12, 16]), d=d, L=L,
                    window=rng.choice([L, _log(rng, 1, L)]), sinks=rng.choice([0, 1, 4, 37]),
                    append=rng.random() < 0.5)
    if op == "window_decode":
        L, Hkv = _log(rng, 16, 8192), _log(rng, 1, 8)
        return dict(op=op, B=_log(rng, 1, 4), Hkv=Hkv, G=rng.choice([1, 2, 4, 7, 8, 12]), d=d, L=L,
                    window=_log(rng, 1, min(L, 4096)), sinks=rng.choice([0, 1, 4, 37]), append=rng.random() < 0.5)
    big = 32768 if op == "window_fwd" else 8192
    N = _log(rng, 1, big)
    heads = max(1, min(32, 32 * big // N))
    Hkv = _log(rng, 1, min(8, heads))
    G = _log(rng, 1, max(1, min(8, heads // Hkv)))
    B = _log(rng, 1, max(1, min(4, heads // (Hkv * G))))
    return dict(op=op, B=B, Hkv=Hkv, G=G, d=d, N=N, window=_log(rng, 1, 1024), sinks=rng.choice([0, 1, 4, 40]),
                ragged=rng.random() < 0.5, seq_major=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------- inputs
def _keys(shape, g):
    """Keys as a model's cache holds them: unit noise about an offset of its own for each head and channel."""
    offset = torch.randn((1, shape[1], 1, shape[3]), generator=g, device="cuda") * 1.5
    return (torch.randn(shape, generator=g, device="cuda") + offset).to(torch.bfloat16)


def _noise(shape, g):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def _lengths(lo, hi, B, g):
    return torch.randint(lo, hi + 1, (B,), generator=g, device="cuda").to(torch.int32)


def _causal_loglinear(M, H, kmax):
    """Block-CSR over H heads: columns {i, i-1}, i - 2^k for k <= kmax and the anchors 0, M//2, M-1 that are <= i."""
    rows = [sorted({j for j in [i, i - 1, 0, M // 2, M - 1] + [i - 2 ** k for k in range(kmax + 1)] if 0 <= j <= i})
            for i in range(M)]
    cols = torch.tensor([j for r in rows for j in r], dtype=torch.int32, device="cuda").repeat(H)
    ptr = torch.tensor([len(r) for r in rows], device="cuda").repeat(H).cumsum(0)
    return torch.cat([ptr.new_zeros(1), ptr]).to(torch.int32), cols


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    c = dict(case)
    s = {"case": c}
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "cache":
        L, T, back = c["L"], c["T"], c["back"]
        s["cache"] = _quantised(_keys((B, Hkv, L, d), g), _noise((B, Hkv, L, d), g))
        s["k"], s["v"] = _keys((B, Hkv, T, d), g), _noise((B, Hkv, T, d), g)
        s["lens"] = _lengths(0, T, B, g) if c["ragged"] else None
        s["first"] = _lengths(0, L - back, B, g)  # the first row read back
        s["start"] = s["first"] + (back - T)      # the first row written
        return s
    if c["op"] in ("q4_decode", "q4_window", "window_decode"):
        L, H = c["L"], Hkv * c["G"]
        low = L // 2 if c["op"] == "q4_decode" else max(1, L - L // 8)
        s["seq_len"] = _lengths(low, L, B, g)
        s["q"] = _noise((B, H, d), g) * 2
        s["k_new"] = _keys((B, Hkv, 1, d), g)[:, :, 0].contiguous() if c["append"] else None
        s["v_new"] = _noise((B, Hkv, d), g) if c["append"] else None
        k, v = _keys((B, Hkv, L, d), g), _noise((B, Hkv, L, d), g)
        if c["op"] == "window_decode":
            s["k_cache"], s["v_cache"] = k, v
        else:
            s["cache"] = _quantised(k, v)
        if c["op"] == "q4_decode":
            s["row_ptr"], s["col_idx"] = _causal_loglinear(L // c["bs"], Hkv, c["kmax"])
        return s
    N, H = c["N"], Hkv * c["G"]
    s["q"], s["k"], s["v"] = _noise((B, H, N, d), g) * 2, _keys((B, Hkv, N, d), g), _noise((B, Hkv, N, d), g)
    s["lens"] = _lengths(N // 2, N, B, g) if c["ragged"] else None
    if c["op"] == "window_bwd":
        s["o"], s["lse"] = _window_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"], s["lens"])
        s["do"] = _noise((B, H, N, d), g)
    if c["seq_major"]:
        for n in ("q", "k", "v", "o", "do"):
            if n in s:
                s[n] = s[n].transpose(1, 2).contiguous().transpose(1, 2)
    return s


# --------------------------------------------------------------------------------- plain forms: 4 bits
# A row of d channels is held as d/2 bytes of codes and, for each group of 32 channels, a scale and a minimum in
# fp16: value = code * scale + minimum.  Codes of a key row: the 32-bit word t * (d/32) + g holds channels
# 32g + 8t .. +7 (lowest nibble first); of a value row: the 16-bit piece y * (d/32) + g holds channels
# 32g + 4y .. +3.
def _quantise(x):
    """(codes 0..15 [..., d], parameters fp16 [..., d/32, 2])"""
    x = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = x.amin(-1), x.amax(-1)
    p = torch.stack([((hi - lo) / 15).clamp(max=65504), lo.clamp(-65504, 65504)], -1).half()
    scale, least = p[..., 0:1].float(), p[..., 1:2].float()
    twice = torch.floor((x - least) / scale * 2)
    code = torch.floor((twice + 1) / 2).clamp(0, 15)
    return torch.where(scale > 0, code, torch.zeros_like(code)).flatten(-2).to(torch.uint8), p


def _pack(code, run):
    """Codes [..., d] to bytes [..., d/2]: `run` neighbouring channels stay together, groups alternate."""
    code = code.unflatten(-1, (-1, GROUP // run, run)).transpose(-2, -3).flatten(-3)
    return code[..., 0::2] | code[..., 1::2] << 4


def _unpack(byte, run):
    code = torch.stack([byte & 15, byte >> 4], -1).flatten(-2)
    return code.unflatten(-1, (GROUP // run, -1, run)).transpose(-2, -3).flatten(-3)


def _value(byte, p, run):
    """The values that packed codes and parameters stand for, fp32."""
    code = _unpack(byte, run).float().unflatten(-1, (-1, GROUP))
    return (code * p[..., 0:1].float() + p[..., 1:2].float()).flatten(-2)


def _quantised(k, v):
    (kc, kp), (vc, vp) = _quantise(k), _quantise(v)
    return _pack(kc, 8), kp, _pack(vc, 4), vp


def _rows(first, n, lens=None):
    """Row numbers [B, n] from first[b] on, and which of them count."""
    at = torch.arange(n, device="cuda")
    live = torch.ones((first.numel(), n), dtype=torch.bool, device="cuda") if lens is None else at < lens[:, None]
    return first[:, None].long() + at, live


def _store(cache, k, v, start, lens=None):
    at, live = _rows(start, k.shape[2], lens)
    b = torch.arange(at.shape[0], device="cuda")[:, None].expand_as(at)[live]
    for kept, x in zip(cache, _quantised(k, v)):
        kept[b, :, at[live]] = x.transpose(1, 2)[live]


def _load(cache, first, n):
    at, _ = _rows(first, n)
    b = torch.arange(at.shape[0], device="cuda")[:, None]
    kc, kp, vc, vp = (x.transpose(1, 2)[b, at].transpose(1, 2) for x in cache)
    return _value(kc, kp, 8), _value(vc, vp, 4)


# ------------------------------------------------------------------------------ plain forms: attention
def _attend(q, k, v, seen):
    """One query a head: q [B, H, d]; k, v [B, Hkv, n, d] fp32; seen [B, Hkv or 1, n]."""
    B, H, d = q.shape
    x = q.float().unflatten(1, (k.shape[1], -1)) @ k.transpose(-1, -2) / math.sqrt(d)
    x = torch.where(seen[:, :, None], x, -math.inf)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    o = (e / total) @ torch.where(seen[..., None], v, 0.0)
    return o.flatten(1, 2).to(torch.bfloat16), (top + torch.log(total)).flatten(1)


def _window_step(q, k, v, seq_len, window, sinks):
    at = torch.arange(k.shape[2], device="cuda")
    t = seq_len[:, None].long() - 1
    return _attend(q, k, v, ((at <= t) & ((at > t - window) | (at < sinks)))[:, None])


def _block_step(q, cache, seq_len, row_ptr, col_idx, bs):
    """The blocks of each sequence's own row, gathered and read back."""
    B, Hkv, L = cache[0].shape[:3]
    t = seq_len.long() - 1
    row = torch.arange(Hkv, device="cuda") * (L // bs) + (t // bs)[:, None]          # [B, Hkv]
    first, count = row_ptr[row].long(), (row_ptr[row + 1] - row_ptr[row]).long()
    slot = torch.arange(32, device="cuda")  # no row of these patterns lists more
    used = slot < count[..., None]
    col = col_idx[(first[..., None] + slot).clamp(max=col_idx.numel() - 1)].long()   # [B, Hkv, 32]
    at = (col[..., None] * bs + torch.arange(bs, device="cuda")).flatten(-2)         # [B, Hkv, 32 bs]
    seen = used.repeat_interleave(bs, -1) & (at <= t[:, None, None])
    b, h = torch.arange(B, device="cuda")[:, None, None], torch.arange(Hkv, device="cuda")[:, None]
    at = torch.where(seen, at, 0)
    kc, kp, vc, vp = (x[b, h, at] for x in cache)
    return _attend(q, _value(kc, kp, 8), _value(vc, vp, 4), seen)


def _bands(N, window):
    """Chunk length C and front padding F of the banded form: chunk c's queries see rows cC - F .. cC + C - 1."""
    C = min(N, max(128, min(window, 1024)))
    return C, window - 1 if window <= N else N - 1


def _banded(x, C, F, chunks):
    """[B, Hkv, N, d] to the rows that each chunk sees, [B, Hkv, chunks, F + C, d], zeros outside, fp32."""
    N = x.shape[2]
    x = torch.nn.functional.pad(x.float(), (0, 0, F, chunks * C - N))
    return x.unfold(2, F + C, C).transpose(-1, -2)


def _chunked(x, Hkv, C, chunks):
    """[B, H, N, ...] to [B, Hkv, chunks, G * C, ...], fp32."""
    x = torch.nn.functional.pad(x.float(), (0, 0, 0, chunks * C - x.shape[2]))
    return x.unflatten(2, (chunks, C)).unflatten(1, (Hkv, -1)).transpose(2, 3).flatten(3, 4)


def _unchunked(x, G, N):
    return x.unflatten(3, (G, -1)).transpose(2, 3).flatten(3, 4).flatten(1, 2)[:, :, :N]


def _visible(N, G, C, F, chunks, window, sinks, lens, B):
    """Which rows of the band, and which first rows before it, each query sees: [B or 1, 1, chunks, G * C, F + C + sinks]."""
    c = torch.arange(chunks, device="cuda")[:, None, None] * C
    t = c + torch.arange(C, device="cuda")[None, :, None]
    k = c - F + torch.arange(F + C, device="cuda")[None, None]
    band = (k >= 0) & (k <= t) & (t - k < window)
    first = torch.arange(min(sinks, N), device="cuda")[None, None]
    early = (first <= t - window) & (first < t + 1)
    seen = torch.cat([band, early.expand(chunks, C, -1)], -1)[None, None]
    if lens is not None:
        seen = seen & (t < lens.long()[:, None, None, None])[:, None]
    else:
        seen = seen & (t < N)[None, None]
    return seen.repeat(1, 1, 1, G, 1)


def _scores(q, k, window, sinks, lens):
    """Scaled scores [B, Hkv, chunks, G * C, F + C + sinks], -inf where unseen, and the pieces they came from."""
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    C, F = _bands(N, window)
    chunks = -(-N // C)
    qc, kb = _chunked(q, Hkv, C, chunks), _banded(k, C, F, chunks)
    first = k[:, :, :min(sinks, N)].float()[:, :, None]
    x = torch.cat([qc @ kb.transpose(-1, -2), qc @ first.transpose(-1, -2)], -1) / math.sqrt(d)
    seen = _visible(N, H // Hkv, C, F, chunks, window, sinks, lens, B)
    return torch.where(seen, x, -math.inf), seen, qc, kb, first, C, F, chunks


def _window_forward(q, k, v, window, sinks, lens):
    B, H, N, d = q.shape
    Hkv, G = k.shape[1], H // k.shape[1]
    x, seen, _, _, _, C, F, chunks = _scores(q, k, window, sinks, lens)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    o = p[..., :F + C] @ _banded(v, C, F, chunks) + p[..., F + C:] @ v[:, :, :min(sinks, N)].float()[:, :, None]
    lse = _unchunked(top + torch.log(total), G, N)[..., 0]
    return _unchunked(o, G, N).to(torch.bfloat16), lse


def _window_backward(q, k, v, o, do, lse, window, sinks, lens):
    B, H, N, d = q.shape
    Hkv, G = k.shape[1], H // k.shape[1]
    x, seen, qc, kb, kf, C, F, chunks = _scores(q, k, window, sinks, lens)
    l = _chunked(lse[..., None], Hkv, C, chunks)
    p = torch.where(seen, torch.exp(x - torch.where(torch.isinf(l), 0.0, l)), 0.0)
    doc = _chunked(do, Hkv, C, chunks)
    delta = (doc * _chunked(o, Hkv, C, chunks)).sum(-1, keepdim=True)
    vf = v[:, :, :min(sinks, N)].float()[:, :, None]
    dp = torch.cat([doc @ _banded(v, C, F, chunks).transpose(-1, -2), doc @ vf.transpose(-1, -2)], -1)
    ds = p * (dp - delta) / math.sqrt(d)
    dq = _unchunked(ds[..., :F + C] @ kb + ds[..., F + C:] @ kf, G, N)
    return dq.to(torch.bfloat16), _shared(ds, qc, N, C, F, chunks), _shared(p, doc, N, C, F, chunks)


def _shared(w, y, N, C, F, chunks):
    """Sum over the queries of w y for each key row, over bands and first rows: the gradient of a shared head."""
    band = w[..., :F + C].transpose(-1, -2) @ y                       # [B, Hkv, chunks, F + C, d]
    at = (torch.arange(chunks, device="cuda")[:, None] * C + torch.arange(F + C, device="cuda")).flatten()
    whole = torch.zeros(*band.shape[:2], F + chunks * C, band.shape[-1], device="cuda")
    whole = whole.index_add_(2, at, band.flatten(2, 3))[:, :, F:F + N]
    first = (w[..., F + C:].transpose(-1, -2) @ y).sum(2)
    whole[:, :, :first.shape[2]] += first
    return whole.to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    if c["op"] == "cache":
        _store(s["cache"], s["k"], s["v"], s["start"], s["lens"])
        k, v = _load(s["cache"], s["first"], c["back"])
        return k.to(torch.bfloat16), v.to(torch.bfloat16)
    if c["op"] == "window_decode":
        if c["append"]:
            b, t = torch.arange(c["B"], device="cuda"), s["seq_len"].long() - 1
            s["k_cache"][b, :, t], s["v_cache"][b, :, t] = s["k_new"], s["v_new"]
        o, lse = _window_step(s["q"], s["k_cache"].float(), s["v_cache"].float(), s["seq_len"], c["window"], c["sinks"])
        return (o, lse, s["k_cache"], s["v_cache"]) if c["append"] else (o, lse)
    if c["op"] in ("q4_decode", "q4_window"):
        if c["append"]:
            _store(s["cache"], s["k_new"][:, :, None], s["v_new"][:, :, None], s["seq_len"] - 1)
        if c["op"] == "q4_decode":
            out = _block_step(s["q"], s["cache"], s["seq_len"], s["row_ptr"], s["col_idx"], c["bs"])
        else:
            k, v = _value(*s["cache"][:2], 8), _value(*s["cache"][2:], 4)
            out = _window_step(s["q"], k, v, s["seq_len"], c["window"], c["sinks"])
        if c["append"]:  # the row that the step added to the cache
            k, v = _load(s["cache"], s["seq_len"] - 1, 1)
            out = (*out, k.to(torch.bfloat16), v.to(torch.bfloat16))
        return out
    if c["op"] == "window_fwd":
        return _window_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"], s["lens"])
    return _window_backward(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], c["window"], c["sinks"], s["lens"])


def _run_own(s):
    import block_sparse_attention_38_b200 as bsa

    c = s["case"]
    if c["op"] == "cache":
        cache = bsa.Q4Cache(*s["cache"])
        bsa.q4_write(cache, s["k"], s["v"], s["start"], lens=s["lens"])
        return bsa.q4_read(cache, s["first"], c["back"])
    if c["op"] == "window_decode":
        out = bsa.window_decode(s["q"], s["k_cache"], s["v_cache"], s["seq_len"], c["window"], c["sinks"],
                                k_new=s["k_new"], v_new=s["v_new"])
        return (*out, s["k_cache"], s["v_cache"]) if c["append"] else out
    if c["op"] in ("q4_decode", "q4_window"):
        cache = bsa.Q4Cache(*s["cache"])
        if c["op"] == "q4_decode":
            out = bsa.q4_decode(s["q"], cache, s["seq_len"], s["row_ptr"], s["col_idx"], c["bs"],
                                k_new=s["k_new"], v_new=s["v_new"])
        else:
            out = bsa.q4_window_decode(s["q"], cache, s["seq_len"], c["window"], c["sinks"],
                                       k_new=s["k_new"], v_new=s["v_new"])
        return (*out, *bsa.q4_read(cache, s["seq_len"] - 1, 1)) if c["append"] else out
    if c["op"] == "window_fwd":
        return bsa.window_forward(s["q"], s["k"], s["v"], c["window"], c["sinks"], lens=s["lens"])
    return bsa.window_backward(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], c["window"], c["sinks"],
                               lens=s["lens"])


# ------------------------------------------------------------------------------------------------ work
def _pairs(N, window, sinks):
    """Visible (query, key) pairs of one sequence of N tokens."""
    n, w = N, min(window, N)
    near = w * (w + 1) // 2 + (n - w) * w
    far = max(0, n - w)  # queries that have rows before their window: query w + i has i + 1 of them
    s = min(sinks, far)
    return near + s * (s + 1) // 2 + (far - s) * s


def work(case):
    c = dict(case)
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    q4 = d // 2 + d // 8  # bytes of one row of the 4-bit cache
    if c["op"] == "cache":
        written = B * Hkv * c["T"] * (0.5 if c["ragged"] else 1.0)
        read = B * Hkv * c["back"]
        return {"bytes": 2 * written * (2 * d + q4) + 2 * read * (q4 + 2 * d), "flops": 2.0 * d * (3 * written + read)}
    if c["op"] in ("q4_decode", "q4_window", "window_decode"):
        H, L = Hkv * c["G"], c["L"]
        if c["op"] == "q4_decode":
            mean = 0.75 * L / c["bs"]  # sequences of L/2 .. L tokens
            blocks = min(mean, 3 + c["kmax"] + 1)
            tokens = blocks * c["bs"]
        else:
            tokens = min(0.94 * L, c["window"] + c["sinks"])
        row = 2 * d if c["op"] == "window_decode" else q4
        moved = 2 * B * Hkv * tokens * row + B * H * (4 * d + 4) + (B * Hkv * 2 * (2 * d + row) if c["append"] else 0)
        return {"bytes": moved, "flops": 4.0 * B * H * tokens * d}
    N, H = c["N"], Hkv * c["G"]
    n = int(N * 0.75) if c["ragged"] else N
    pairs = B * H * _pairs(n, c["window"], c["sinks"])
    io = 2 * d * B * N * (2 * H + 2 * Hkv) + 4 * B * H * N
    if c["op"] == "window_fwd":
        return {"bytes": io, "flops": 4.0 * pairs * d}
    return {"bytes": io + 2 * d * B * N * (2 * H + 2 * Hkv), "flops": 10.0 * pairs * d}


# ----------------------------------------------------------------------------------------------- exact
def _exact_values(byte, p, words):
    """Packed rows to values in 64 bits, channel by channel from the layout's definition."""
    d = byte.shape[-1] * 2
    value = torch.empty(*byte.shape[:-1], d, dtype=torch.float64, device=byte.device)
    groups = d // GROUP
    per = 8 if words else 4  # channels in a word (keys) or piece (values)
    for ch in range(d):
        grp, y, i = ch // GROUP, ch % GROUP // per, ch % per
        nibble = (y * groups + grp) * per + i
        code = (byte[..., nibble // 2] >> (4 * (nibble % 2))) & 15
        value[..., ch] = code.double() * p[..., grp, 0].double() + p[..., grp, 1].double()
    return value


def _exact_round(x):
    """What a row [..., d] reads back as after it was written, in 64 bits."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    x = x.double()
    for a in range(0, x.shape[-1], GROUP):
        y = x[..., a:a + GROUP]
        least, most = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        scale = ((most - least) / 15).half().double()
        least = least.half().double()
        code = torch.floor((y - least) / torch.where(scale > 0, scale, 1.0) + 0.5).clamp(0, 15)
        out[..., a:a + GROUP] = code * scale + least
    return out


def _exact_row(q, k, v, keys):
    """One query over the listed rows: q [G, d]; k, v [n, d]."""
    x = (q @ k[keys].T) / math.sqrt(q.shape[-1])
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]) @ v[keys], lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    B, Hkv, d = c["B"], c["Hkv"], c["d"]
    if c["op"] == "cache":
        k, v = _exact_values(*s["cache"][:2], True), _exact_values(*s["cache"][2:], False)
        ks, vs = [], []
        for b in range(B):
            n = c["T"] if s["lens"] is None else int(s["lens"][b])
            at, first = int(s["start"][b]), int(s["first"][b])
            k[b, :, at:at + n], v[b, :, at:at + n] = _exact_round(s["k"][b, :, :n]), _exact_round(s["v"][b, :, :n])
            ks.append(k[b, :, first:first + c["back"]])
            vs.append(v[b, :, first:first + c["back"]])
        return torch.stack(ks), torch.stack(vs)
    if c["op"] in ("q4_decode", "q4_window", "window_decode"):
        G, q = c["G"], s["q"].double()
        o = torch.empty(q.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        rows = []
        for b in range(B):
            t = int(s["seq_len"][b]) - 1
            for h in range(Hkv):
                if c["op"] == "window_decode":
                    k, v = s["k_cache"][b, h].double(), s["v_cache"][b, h].double()
                else:
                    kc, kp, vc, vp = (x[b, h] for x in s["cache"])
                    k, v = _exact_values(kc, kp, True), _exact_values(vc, vp, False)
                if c["append"]:
                    same = c["op"] == "window_decode"
                    k[t] = s["k_new"][b, h].double() if same else _exact_round(s["k_new"][b, h])
                    v[t] = s["v_new"][b, h].double() if same else _exact_round(s["v_new"][b, h])
                if c["op"] == "q4_decode":
                    r = h * (c["L"] // c["bs"]) + t // c["bs"]
                    cols = s["col_idx"][int(s["row_ptr"][r]):int(s["row_ptr"][r + 1])].tolist()
                    keys = torch.cat([torch.arange(j * c["bs"], min((j + 1) * c["bs"], t + 1), device="cuda") for j in cols])
                else:
                    w0 = max(0, t - c["window"] + 1)
                    keys = torch.cat([torch.arange(0, min(c["sinks"], w0), device="cuda"), torch.arange(w0, t + 1, device="cuda")])
                o[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G] = _exact_row(q[b, h * G:(h + 1) * G], k, v, keys)
                rows.append((k[t], v[t]))
        if not c["append"]:
            return o, lse
        if c["op"] == "window_decode":
            return o, lse, None, None
        back = [torch.stack([r[i] for r in rows]).view(B, Hkv, 1, d) for i in (0, 1)]
        return o, lse, back[0], back[1]
    N, G = c["N"], c["G"]
    if B * Hkv * G * N * N > 1.1e11 / 3:  # over about 20 seconds
        return None
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    at = torch.arange(N, device="cuda")
    seen = (at[None] <= at[:, None]) & ((at[:, None] - at[None] < c["window"]) | (at[None] < c["sinks"]))
    outs = [torch.zeros_like(q), torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")]
    if c["op"] == "window_bwd":
        outs = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)]
        o, do, given = s["o"].double(), s["do"].double(), s["lse"].double()
    for b in range(B):
        n = N if s["lens"] is None else int(s["lens"][b])
        for h in range(Hkv * G):
            kh, vh = k[b, h // G, :n], v[b, h // G, :n]
            x = (q[b, h, :n] @ kh.T / math.sqrt(d)).masked_fill(~seen[:n, :n], -math.inf)
            if c["op"] == "window_fwd":
                outs[1][b, h, :n] = torch.logsumexp(x, -1)
                outs[0][b, h, :n] = torch.softmax(x, -1) @ vh
                continue
            p = torch.exp(x - given[b, h, :n, None])
            y = do[b, h, :n]
            ds = p * (y @ vh.T - (y * o[b, h, :n]).sum(-1, keepdim=True)) / math.sqrt(d)
            outs[0][b, h, :n] = ds @ kh
            outs[1][b, h // G, :n] += ds.T @ q[b, h, :n]
            outs[2][b, h // G, :n] += p.T @ y
    return tuple(outs)
