"""Decode steps over long caches (4 bits and bf16) against the fp64 oracle.

Tolerances.  O is rounded once to bf16 (off by at most 2^-8 of the value, half a
step).  Over 4 bits the weights p_k s_kG are rounded to fp16 (2^-11 each), over
bf16 they are kept to 2^-16; sums run in fp32.  With weights p that sum to 1 the
error of a channel is at most max_k |v_k| 2^-11, plus the scores' fp32 error: x is
a sum of d products held to 2^-20 of its largest term, which moves a weight by less
than 2^-12.  So |O - exact| <= 2^-8 |O| + 2^-10 max|v|, and the LSE within 2^-13 of
it for scores below 2^6 (2^-20 of 128 terms, ex2.approx 2^-22).
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

pytestmark = pytest.mark.gpu


def _bf16(shape, g, mul=1.0):
    return (torch.randn(shape, generator=g) * mul).to(torch.bfloat16)


def _make(B, Hkv, G, L, d, seed, vmul=1.0, qmul=1.0):
    g = torch.Generator().manual_seed(seed)
    q = _bf16((B, Hkv * G, d), g, qmul)
    k = _bf16((B, Hkv, L, d), g) + torch.randn(1, Hkv, 1, d, generator=g).to(torch.bfloat16)
    v = _bf16((B, Hkv, L, d), g, vmul)
    kn, vn = _bf16((B, Hkv, d), g), _bf16((B, Hkv, d), g, vmul)
    return q, k, v, kn, vn


def _pack(k, v):
    parts = []
    for x, is_key in ((k, True), (v, False)):
        c, s, m = o.quantise(x)
        parts += [torch.from_numpy(o.pack(c, is_key)).cuda(),
                  torch.from_numpy(np.stack([s, m], -1)).cuda()]
    return bsa.Q4Cache(*parts)


def _close(got, lse, want, lw, vmax):
    got, lse = got.float().cpu().numpy(), lse.cpu().numpy()
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(lw))
    live = ~np.isneginf(lw)
    np.testing.assert_allclose(lse[live], lw[live], rtol=2.0 ** -20, atol=2.0 ** -13)
    assert (got[~live] == 0).all()
    np.testing.assert_allclose(got, want, rtol=2.0 ** -8 + 2.0 ** -20, atol=2.0 ** -10 * vmax)


def _lens(B, L, low=1):
    return [max(low, L - (37 * b) % L) for b in range(B)]


def _with_new(x, new, lens):
    x = x.clone()
    for b, n in enumerate(lens):
        if n:
            x[b, :, n - 1] = new[b]
    return x


def _poison(cache_k, cache_v, lens, window, sinks):
    """NaN in every row that is not visible."""
    for b, n in enumerate(lens):
        seen = np.zeros(cache_k.shape[2], bool)
        if n:
            seen[o.window_rows(n - 1, window, sinks)] = True
        cache_k[b, :, ~seen] = float("nan")
        cache_v[b, :, ~seen] = float("nan")


CASES = [  # B, Hkv, G, L, window, sinks
    (1, 1, 1, 1, 1, 0), (2, 1, 1, 2, 1, 1), (1, 1, 3, 17, 5, 2), (2, 2, 8, 33, 33, 0),
    (1, 3, 7, 64, 10, 40), (3, 1, 9, 100, 31, 4), (1, 1, 16, 257, 100, 1), (2, 1, 20, 129, 64, 3),
    (1, 2, 4, 1000, 1000, 0), (1, 1, 2, 5000, 4097, 33), (2, 8, 4, 700, 1, 0), (1, 1, 1, 3000, 2048, 5000),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("B,Hkv,G,L,window,sinks", CASES)
def test_window_over_bf16(B, Hkv, G, L, window, sinks, d, append):
    q, k, v, kn, vn = _make(B, Hkv, G, L, d, 11)
    lens = _lens(B, L)
    _poison(k, v, lens, window, sinks)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kc, vc = k.cuda(), v.cuda()
    new = dict(k_new=kn.cuda(), v_new=vn.cuda()) if append else {}
    got, lse = bsa.window_decode(q.cuda(), kc, vc, seq, window, sinks, **new)
    assert bsa.stream_status() == 0
    if append:
        k, v = _with_new(k, kn, lens), _with_new(v, vn, lens)
    assert torch.equal(kc.cpu().view(torch.int16), k.view(torch.int16))  # only row t changed
    assert torch.equal(vc.cpu().view(torch.int16), v.view(torch.int16))
    want, lw = o.decode(q, k, v, lens, lambda b, h, t: o.window_rows(t, window, sinks), d ** -0.5)
    _close(got, lse, want, lw, 5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("B,Hkv,G,L,window,sinks", CASES)
def test_window_over_4_bits(B, Hkv, G, L, window, sinks, d, append):
    q, k, v, kn, vn = _make(B, Hkv, G, L, d, 12)
    lens = _lens(B, L)
    _poison(k, v, lens, window, sinks)
    cache = _pack(k, v)
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = dict(k_new=kn.cuda(), v_new=vn.cuda()) if append else {}
    got, lse = bsa.q4_window_decode(q.cuda(), cache, seq, window, sinks, **new)
    assert bsa.stream_status() == 0
    if append:
        k, v = _with_new(k, kn, lens), _with_new(v, vn, lens)
    for a, b in zip(cache, _pack(k, v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # only row t changed
    kq, vq = o.values(*o.quantise(k)), o.values(*o.quantise(v))
    want, lw = o.decode(q, kq, vq, lens, lambda b, h, t: o.window_rows(t, window, sinks), d ** -0.5)
    _close(got, lse, want, lw, 5)


@pytest.mark.parametrize("d,bs", [(64, 32), (128, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("B,Hkv,G,M,append", [(1, 1, 1, 1, False), (2, 2, 4, 5, True), (3, 1, 8, 12, False),
                                              (2, 3, 12, 7, True)])
def test_blocks_over_4_bits(B, Hkv, G, M, append, d, bs):
    L = M * bs
    q, k, v, kn, vn = _make(B, Hkv, G, L, d, 13)
    lens = _lens(B, L)
    lens[-1] = max(1, L - bs // 2 - 1)  # ends inside a block
    rng = np.random.default_rng(5)
    rows = []
    for h in range(Hkv):
        for i in range(M):  # future blocks, repeats, any order, some rows empty
            cols = rng.permutation(M)[:rng.integers(0, M + 1)].tolist()
            rows.append(cols + cols[:1])
    rp = np.cumsum([0] + [len(r) for r in rows]).astype(np.int32)
    ci = np.array([j for r in rows for j in r] or [0], np.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            seen = np.zeros(L, bool)
            seen[o.block_rows(n - 1, rp, ci, h, M, bs)] = True
            k[b, h, ~seen] = float("nan")
            v[b, h, ~seen] = float("nan")
    cache = _pack(k, v)
    new = dict(k_new=kn.cuda(), v_new=vn.cuda()) if append else {}
    got, lse = bsa.q4_decode(q.cuda(), cache, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                             torch.from_numpy(rp).cuda(), torch.from_numpy(ci).cuda(), bs, **new)
    assert bsa.stream_status() == 0
    if append:
        k, v = _with_new(k, kn, lens), _with_new(v, vn, lens)
    for a, b in zip(cache, _pack(k, v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    kq, vq = o.values(*o.quantise(k)), o.values(*o.quantise(v))
    want, lw = o.decode(q, kq, vq, lens, lambda b, h, t: o.block_rows(t, rp, ci, h, M, bs), d ** -0.5)
    _close(got, lse, want, lw, 5)


@pytest.mark.parametrize("vmul", [1e-6, 1e-3, 300.0, 20000.0])
def test_small_and_large_values_lose_nothing(vmul):
    """Value scales from fp16's subnormals to its top: the weights are shifted with them."""
    q, k, v, _, _ = _make(1, 2, 4, 900, 128, 14, vmul=vmul)
    v[0, 0, :400] *= 0.01  # the scale grows along the cache
    cache = _pack(k, v)
    n = torch.tensor([900], dtype=torch.int32, device="cuda")
    got, lse = bsa.q4_window_decode(q.cuda(), cache, n, 900)
    kq, vq = o.values(*o.quantise(k)), o.values(*o.quantise(v))
    want, lw = o.decode(q, kq, vq, [900], lambda b, h, t: np.arange(900), 128 ** -0.5)
    _close(got, lse, want, lw, 5 * vmul)


@pytest.mark.parametrize("qmul", [0.0, 1e-20, 1e-3, 30.0])
def test_query_range(qmul):
    q, k, v, _, _ = _make(1, 1, 8, 300, 128, 15, qmul=qmul)
    cache = _pack(k, v)
    n = torch.tensor([300], dtype=torch.int32, device="cuda")
    got, lse = bsa.q4_window_decode(q.cuda(), cache, n, 300)
    kq, vq = o.values(*o.quantise(k)), o.values(*o.quantise(v))
    want, lw = o.decode(q, kq, vq, [300], lambda b, h, t: np.arange(300), 128 ** -0.5)
    if qmul > 10:
        # scores up to 2^9 are held to 2^-20 of their largest term: weights move by
        # 2^-9 times their distance from the mean, below 2^-8 max|v|
        np.testing.assert_allclose(lse.cpu().numpy(), lw, atol=2.0 ** -10)
        np.testing.assert_allclose(got.float().cpu().numpy(), want, rtol=2.0 ** -8, atol=2.0 ** -8 * 5)
    else:
        _close(got, lse, want, lw, 5)


def test_bad_and_empty_lengths():
    q, k, v, kn, vn = _make(4, 1, 2, 64, 64, 16)
    cache = _pack(k, v)
    before = [t.clone() for t in cache]
    seq = torch.tensor([0, 65, -3, 0], dtype=torch.int32, device="cuda")
    for call in (lambda: bsa.q4_window_decode(q.cuda(), cache, seq, 8, 2, k_new=kn.cuda(), v_new=vn.cuda()),
                 lambda: bsa.window_decode(q.cuda(), k.cuda(), v.cuda(), seq, 8, 2)):
        got, lse = call()
        assert bsa.stream_status() == bsa.STATUS_BAD_SEQ_LEN
        assert float(got.abs().sum()) == 0 and bool(torch.isneginf(lse).all())
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    empty = torch.zeros(4, dtype=torch.int32, device="cuda")
    bsa.q4_window_decode(q.cuda(), cache, empty, 8)
    assert bsa.stream_status() == 0


def test_bad_block_rows_are_reported():
    q, k, v, _, _ = _make(1, 1, 1, 128, 64, 17)
    cache = _pack(k, v)
    seq = torch.tensor([100], dtype=torch.int32, device="cuda")
    rp = torch.tensor([0, 0, 0, 0, 4], dtype=torch.int32, device="cuda")
    ci = torch.tensor([4, -1, 3, 0], dtype=torch.int32, device="cuda")
    got, lse = bsa.q4_decode(q.cuda(), cache, seq, rp, ci, 32)
    assert bsa.stream_status() == bsa.STATUS_BAD_COLUMN
    kq, vq = o.values(*o.quantise(k)), o.values(*o.quantise(v))
    rows = np.r_[0:32, 96:100]
    want, lw = o.decode(q, kq, vq, [100], lambda b, h, t: rows, 64 ** -0.5)
    _close(got, lse, want, lw, 5)
    rp[3] = 5
    got, lse = bsa.q4_decode(q.cuda(), cache, seq, rp, ci, 32)
    assert bsa.stream_status() == bsa.STATUS_BAD_ROW_PTR
    assert bool(torch.isneginf(lse).all())


def test_same_bits_on_a_side_stream_and_in_a_graph():
    q, k, v, kn, vn = _make(2, 2, 4, 900, 128, 18)
    cache = _pack(k, v)
    q, kn, vn = q.cuda(), kn.cuda(), vn.cuda()
    seq = torch.tensor([900, 411], dtype=torch.int32, device="cuda")
    first = bsa.q4_window_decode(q, cache, seq, 700, 4, k_new=kn, v_new=vn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = bsa.q4_window_decode(q, cache, seq, 700, 4, k_new=kn, v_new=vn)
    side.synchronize()
    out, lse = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsa.q4_window_decode(q, cache, seq, 700, 4, k_new=kn, v_new=vn, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    for got in (second, (out, lse)):
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])
    # the graph follows the device's lengths
    seq.copy_(torch.tensor([300, 899], dtype=torch.int32))
    graph.replay()
    want = bsa.q4_window_decode(q, cache, seq, 700, 4, k_new=kn, v_new=vn)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
