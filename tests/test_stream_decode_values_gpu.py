"""Decode steps over long caches on values at the edges: NaN and infinite scores in
rows that are seen, against the fp64 oracle.

Tolerances as in test_stream_decode_gpu.py: |O - exact| <= 2^-8 |O| + 2^-10 max|v|
(one bf16 rounding; weights to 2^-11 each, and the scores' fp32 error), LSE to 2^-13.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

from test_stream_decode_gpu import _make, _pack

pytestmark = pytest.mark.gpu

# (rows of the cache): one CTA a cached head, and a cluster of them
LENGTHS = [70, 6000]


def _step(bits, q, k, v, lens, window, sinks, new=None):
    """Kernel and oracle on the same rows; the rows that the oracle reads."""
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw = {} if new is None else dict(k_new=new[0].cuda(), v_new=new[1].cuda())
    if bits == 4:
        got = bsa.q4_window_decode(q.cuda(), _pack(k, v), seq, window, sinks, **kw)
    else:
        got = bsa.window_decode(q.cuda(), k.cuda(), v.cuda(), seq, window, sinks, **kw)
    assert bsa.stream_status() == 0
    if new is not None:
        k, v = k.clone(), v.clone()
        for b, n in enumerate(lens):
            k[b, :, n - 1], v[b, :, n - 1] = new[0][b], new[1][b]
    if bits == 4:
        k, v = o.values(*o.quantise(k)), o.values(*o.quantise(v))
    with np.errstate(invalid="ignore"):
        want = o.decode(q, k, v, lens, lambda b, h, t: o.window_rows(t, window, sinks), q.shape[2] ** -0.5)
    return [x.float().cpu().numpy() for x in got], want


def _close(got, want, vmax=5.0):
    np.testing.assert_allclose(got[0], want[0], rtol=2.0 ** -8 + 2.0 ** -20, atol=2.0 ** -10 * vmax)
    np.testing.assert_allclose(got[1], want[1], rtol=2.0 ** -20, atol=2.0 ** -13)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_nan_in_a_query_is_its_head_s_result(bits, L, d):
    q, k, v, _, _ = _make(2, 2, 4, L, d, 41)
    q[0, 5, 3] = float("nan")
    q[1, 0] = float("nan")
    got, want = _step(bits, q, k, v, [L, L - 5], L, 0)
    assert np.isnan(want[0][0, 5]).all() and np.isnan(want[1][1, 0]) and np.isnan(want[0]).sum() == 2 * d
    _close(got, want)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("where", ["alone in its unit", "only key", "new token alone in its unit", "a far warp's"])
def test_a_nan_key_that_is_seen_is_not_dropped(bits, L, where):
    q, k, v, kn, vn = _make(1, 1, 3, L, 128, 42)
    window, sinks, new, n = L, 0, None, L
    if where == "alone in its unit":  # rows 0 .. 32 are seen: row 32 begins a unit of either cache
        n = 33
        k[0, 0, 32, 7] = float("nan")
    elif where == "only key":
        window = 1
        k[0, 0, L - 1, 7] = float("nan")
    elif where == "new token alone in its unit":
        n, new = 65, (kn, vn)
        kn[0, 0, 9] = float("nan")
    else:
        k[0, 0, L // 2, 100] = float("nan")
    got, want = _step(bits, q, k, v, [n], window, sinks, new)
    assert np.isnan(want[0]).all() and np.isnan(want[1]).all()
    _close(got, want)


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("d", [64, 128])
def test_a_score_of_minus_infinity_weighs_nothing(L, d):
    """Keys with -inf in a channel where every query is positive, in whole units and in
    a part of one; the weights of all other keys are as if these were not seen."""
    q, k, v, _, _ = _make(2, 2, 4, L, d, 43)
    q[..., 0] = q[..., 0].abs() + 0.5
    k[0, 0, :16, 0] = k[0, 1, 5:40, 0] = k[1, :, 48:68, 0] = k[1, :, 0, 0] = -float("inf")
    got, want = _step(16, q, k, v, [L, L - 1], L, 0)
    assert np.isfinite(want[0]).all() and np.isfinite(want[1]).all()
    _close(got, want)


@pytest.mark.parametrize("L", LENGTHS)
def test_only_scores_of_minus_infinity(L):
    """The sum of weights is 0: LSE = ln 0, and O = 0 / 0."""
    q, k, v, _, _ = _make(1, 1, 4, L, 64, 44)
    q[..., 0] = q[..., 0].abs() + 0.5
    k[..., 0] = -float("inf")
    got = bsa.window_decode(q.cuda(), k.cuda(), v.cuda(), torch.tensor([L], dtype=torch.int32, device="cuda"), L)
    assert bsa.stream_status() == 0
    assert bool(torch.isnan(got[0]).all()) and bool(torch.isneginf(got[1]).all())


@pytest.mark.parametrize("peaks,bits", [(1, 15), (256, 10), (256, 13)])
@pytest.mark.parametrize("G,d,append", [(1, 64, False), (4, 128, True), (12, 128, False)])
def test_channel_groups_of_unlike_scales_over_a_long_tail(G, d, append, peaks, bits):
    """Value groups whose scales lie 2^10 to 2^22 apart, and keys (one, or one in each
    warp's first rows) that outweigh each other one 2^bits times: each group keeps the
    accuracy that it has alone, so the tolerance takes max|v| of the group."""
    L, ratio = 40000, (0, -22, -20, -10)
    g = torch.Generator().manual_seed(45)
    q = torch.ones(1, G, d, dtype=torch.bfloat16)
    k = (torch.randn(1, 1, L, d, generator=g) * 0.05).to(torch.bfloat16)
    k[0, 0, 7:32 * peaks:32] = bits * np.log(2) / d ** 0.5
    v = torch.randn(1, 1, L, d, generator=g)
    for i in range(d // 32):
        v[..., 32 * i:32 * i + 32] *= 2.0 ** ratio[i]
    v = v.to(torch.bfloat16)
    new = (k[:, :, 5].clone(), v[:, :, 5].clone()) if append else None
    got, want = _step(4, q, k, v, [L], L, 0, new)
    for i in range(d // 32):
        at = slice(32 * i, 32 * i + 32)
        _close((got[0][..., at], got[1]), (want[0][..., at], want[1]), 5 * 2.0 ** ratio[i])


def test_a_group_whose_scale_grows_along_the_cache():
    """One group's scale grows 2^20-fold row by row, another's falls so, a third has none."""
    L, d = 9000, 128
    g = torch.Generator().manual_seed(46)
    q, k, v, _, _ = _make(1, 1, 4, L, d, 46)
    grow = 2.0 ** torch.linspace(-10, 10, L)[:, None]
    v = v.float()
    v[0, 0, :, :32] *= grow
    v[0, 0, :, 32:64] /= grow
    v[0, 0, :, 64:96] = 3.0
    got, want = _step(4, q, k, v.to(torch.bfloat16), [L], L, 0)
    for at, vmax in ((slice(0, 64), 5 * 2.0 ** 10), (slice(64, 96), 3.0), (slice(96, 128), 5.0)):
        _close((got[0][..., at], got[1]), (want[0][..., at], want[1]), vmax)


@pytest.mark.parametrize("B,Hkv,G,L,d,window,sinks,append", [
    (1, 1, 4, 20000, 64, 20000, 0, True), (1, 1, 8, 40000, 128, 40000, 0, False), (1, 1, 1, 33333, 128, 30000, 7, True),
    (2, 8, 4, 12000, 128, 12000, 0, False), (2, 4, 7, 17001, 64, 16900, 33, True)])
def test_long_caches(B, Hkv, G, L, d, window, sinks, append):
    """10 to 40 thousand visible rows of few heads, where clusters are cut off at 16 CTAs
    and blocks of sixteen warps take over; lengths from 3 tokens to all."""
    q, k, v, kn, vn = _make(B, Hkv, G, L, d, 47)
    for lens in ([L, 3][:B], [L - 4999, L][:B]):
        got, want = _step(4, q, k, v, lens, window, sinks, (kn, vn) if append else None)
        _close(got, want)
