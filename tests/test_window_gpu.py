"""Sliding-window attention on the GPU against the fp64 oracle.

Tolerances of the forward.  bf16 rounding is off by at most 2^-8 of the value
(half a step); P is rounded so before P V and O after it, and part of the
exponentials is taken to 7.5e-5.  The errors of P's many terms are independent, so
|O - exact| <= 2^-8 |O| + 2^-8 max |v|: sum_k p_k |v_k| <= max |v|, of which the
rounding of P alone can take 2^-8 only if every term is off by half a step the
same way, and the fp32 scores' share (x to 2^-20 of its largest term) and the
polynomial's fit into what that leaves.  LSE: the sum's relative error, at most
7.5e-5 plus the scores' error, below 2^-12.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

pytestmark = pytest.mark.gpu


def make(B, H, Hkv, N, d, seed, seq_major=False, qmul=1.0):
    g = torch.Generator().manual_seed(seed)

    def one(h, mul=1.0):
        shape = (B, N, h, d) if seq_major else (B, h, N, d)
        x = (torch.randn(shape, generator=g) * mul).to(torch.bfloat16)
        return x.transpose(1, 2) if seq_major else x

    return one(H, qmul), one(Hkv, 1.5), one(Hkv), one(H)


def cuda(x):
    """x on the GPU with its strides."""
    return x.cuda() if x.is_contiguous() else x.transpose(1, 2).contiguous().cuda().transpose(1, 2)


def check_forward(got, lse, want, lw, vmax=5.0):
    got, lse = got.float().cpu().numpy(), lse.cpu().numpy()
    np.testing.assert_array_equal(np.isneginf(lse), np.isneginf(lw))
    live = ~np.isneginf(lw)
    assert (got[~live] == 0).all()
    np.testing.assert_allclose(lse[live], lw[live], rtol=2.0 ** -20, atol=2.0 ** -12)
    np.testing.assert_allclose(got, want, rtol=2.0 ** -8, atol=2.0 ** -8 * vmax)


CASES = [  # B, H, Hkv, N, window, sinks
    (1, 1, 1, 1, 1, 0), (1, 2, 1, 2, 1, 1), (2, 3, 1, 17, 4, 2), (1, 1, 1, 128, 128, 0), (1, 2, 2, 129, 1, 0),
    (2, 4, 2, 300, 77, 3), (1, 3, 3, 511, 129, 33), (1, 2, 1, 700, 700, 0), (1, 6, 2, 513, 5000, 0),
    (1, 5, 1, 1000, 64, 200), (3, 2, 1, 385, 100, 32), (1, 1, 1, 1300, 1024, 4), (1, 2, 1, 900, 1, 900),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks", CASES)
def test_forward(B, H, Hkv, N, window, sinks, d):
    q, k, v, _ = make(B, H, Hkv, N, d, 1)
    got, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), window, sinks)
    assert bsa.stream_status() == 0
    check_forward(got, lse, *o.window_forward(q, k, v, window, sinks, d ** -0.5))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks,lens", [
    (4, 2, 1, 300, 50, 3, [0, 1, 129, 300]), (3, 3, 3, 257, 300, 0, [256, 255, 128]),
    (2, 4, 2, 900, 100, 40, [500, 0]), (2, 1, 1, 260, 20, 1, [127, 258])])
def test_forward_of_padded_sequence_major_batches(B, H, Hkv, N, window, sinks, lens, d):
    q, k, v, _ = make(B, H, Hkv, N, d, 2, seq_major=True)
    for b, n in enumerate(lens):  # what pads the batch may be anything
        for x in (q, k, v):
            x[b, :, n:] = float("nan")
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got, lse = bsa.window_forward(cuda(q), cuda(k), cuda(v), window, sinks, lens=n)
    assert bsa.stream_status() == 0
    assert got.stride() == cuda(q).stride()
    check_forward(got, lse, *o.window_forward(q, k, v, window, sinks, d ** -0.5, lens))


@pytest.mark.parametrize("H,Hkv,d", [(16, 4, 64), (9, 3, 128)])
def test_forward_of_many_tiles_with_empty_ones_between(H, Hkv, d):
    """More tiles than SMs, so that one block takes tiles with and without tokens in turn."""
    B, N, lens = 4, 1900, [1900, 0, 700, 1300]
    q, k, v, _ = make(B, H, Hkv, N, d, 8)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), 150, 4, lens=n)
    assert bsa.stream_status() == 0
    check_forward(got, lse, *o.window_forward(q, k, v, 150, 4, d ** -0.5, lens))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-3, 1.0])
def test_forward_scales(scale):
    q, k, v, _ = make(1, 2, 1, 400, 128, 3)
    got, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), 150, 4, scale=scale)
    want, lw = o.window_forward(q, k, v, 150, 4, scale)
    check_forward(got, lse, want, lw)


def test_forward_with_growing_scores():
    """The running maximum grows by far more than the rescale threshold along the walk."""
    q, k, v, _ = make(1, 2, 2, 1200, 64, 4)
    k = (k.float() * torch.linspace(0.1, 6, 1200)[:, None]).to(torch.bfloat16)
    q = (q.float() * 3).to(torch.bfloat16)
    got, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), 1200, 0)
    # scores to 2^8, held to 2^-16 each: weights move by 2^-16, well inside
    check_forward(got, lse, *o.window_forward(q, k, v, 1200, 0, 64 ** -0.5))


def test_long_forward_against_a_banded_reference():
    N, W, S, d = 20000, 700, 6, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(1, h, N, d, generator=g, device="cuda").to(torch.bfloat16) for h in (4, 2, 2))
    got, lse = bsa.window_forward(q, k, v, W, S)
    for q0 in (0, 690, 9999, 19900):
        rows = torch.arange(q0, min(N, q0 + 100), device="cuda")
        keys = torch.arange(0, min(N, q0 + 100), device="cuda")
        seen = (keys <= rows[:, None]) & ((keys > rows[:, None] - W) | (keys < S))
        for h in range(4):
            x = (q[0, h, rows].double() @ k[0, h // 2, keys].double().T * d ** -0.5).masked_fill(~seen, -torch.inf)
            want = torch.softmax(x, -1) @ v[0, h // 2, keys].double()
            np.testing.assert_allclose(got[0, h, rows].double().cpu(), want.cpu(), rtol=2.0 ** -8, atol=2.0 ** -8 * 5)
            np.testing.assert_allclose(lse[0, h, rows].double().cpu(), torch.logsumexp(x, -1).cpu(), atol=2.0 ** -12)


def test_bad_lengths_are_reported():
    q, k, v, _ = make(3, 2, 2, 140, 64, 6)
    n = torch.tensor([-1, 141, 140], dtype=torch.int32, device="cuda")
    got, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), 30, 2, lens=n)
    assert bsa.stream_status() == bsa.STATUS_BAD_SEQ_LEN
    check_forward(got, lse, *o.window_forward(q, k, v, 30, 2, 64 ** -0.5, [0, 0, 140]))


def test_two_streams_and_a_graph_give_the_same_bits():
    q, k, v, _ = (x.cuda() for x in make(2, 4, 2, 1000, 128, 7))
    first = bsa.window_forward(q, k, v, 300, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = bsa.window_forward(q, k, v, 300, 4)
    third = bsa.window_forward(q, k, v, 300, 4)  # both at once
    torch.cuda.synchronize()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bsa.window_forward(q, k, v, 300, 4, out=out, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    for got in (second, third, (out, lse)):
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("Hkv,d", [(1, 64), (2, 128)])
def test_forward_does_not_move_with_what_is_not_seen(Hkv, d):
    """Large finite values in keys after a query, or before its window, change no bit."""
    q, k, v, _ = (x.cuda() for x in make(1, 2, Hkv, 900, d, 9))
    first, lse = bsa.window_forward(q, k, v, 100, 0)
    for hidden, rows in ((slice(333, None), slice(0, 333)), (slice(0, 333), slice(333 + 99, None))):
        far = [x.clone() for x in (k, v)]
        for x in far:
            x[:, :, hidden] *= 1e6
        got, other = bsa.window_forward(q, *far, 100, 0)
        assert torch.equal(got[:, :, rows], first[:, :, rows]) and torch.equal(other[:, :, rows], lse[:, :, rows])


@pytest.mark.parametrize("B,H,Hkv,N,d,window", [(2, 6, 2, 4000, 64, 4000), (2, 12, 6, 2900, 128, 2000), (40, 8, 8, 900, 128, 900)])
def test_forward_with_several_waves_of_unequal_tiles(B, H, Hkv, N, d, window):
    """More tiles than SMs and rows that see more and more keys, in both orders of the
    items (few heads: all heads of a row in turn; many: one head after another)."""
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k, v = (torch.randn(B, h, N, d, generator=g, device="cuda").to(torch.bfloat16) for h in (H, Hkv, Hkv))
    got, lse = bsa.window_forward(q, k, v, window, 3)
    assert bsa.stream_status() == 0
    i = torch.arange(N, device="cuda")
    seen = (i <= i[:, None]) & ((i > i[:, None] - window) | (i < 3))
    for b in range(0, B, max(1, B // 3)):
        for h in range(H):
            x = (q[b, h].double() @ k[b, h * Hkv // H].double().T * d ** -0.5).masked_fill(~seen, -torch.inf)
            want = torch.softmax(x, -1) @ v[b, h * Hkv // H].double()
            torch.testing.assert_close(got[b, h].double(), want, rtol=2.0 ** -8, atol=2.0 ** -8 * 6)  # |v| below 6
            torch.testing.assert_close(lse[b, h].double(), torch.logsumexp(x, -1), rtol=0, atol=2.0 ** -12)
