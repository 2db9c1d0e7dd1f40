"""Gradients of sliding-window attention on the GPU against the fp64 oracle (the
chain rule) and against differences of the forward.

Tolerances.  bf16 rounding is off by at most 2^-8 of the value (half a step).  P
and dS are rounded so before their products, and P carries the exponential's
7.5e-5 and the LSE's error (together below 2^-12), so an element moves by at most
(2^-8 + 2^-12) times the sum of its terms' magnitudes.  D uses O as the forward
gave it: rounded to bf16, from a P that was too, so each O_c is off by at most
2^-8 (|O_c| + sum P |v_c|), which moves an element by 2^-8 times what the oracle
adds up as `moved`.  The result is rounded once more.  Each element is within the
sum of these.  In the root mean square a rounding is 2^-9.3, and the errors of many
terms are independent, so the whole is within 2^-7 in the 2-norm.  Where dP and D
cancel (a window of one key: dS = 0) what is left is their fp32 sums' error: d terms
whose magnitudes add up to less than d, held to d 2^-24 of that, are off by at most
d^2 2^-24 <= 2^-10 each, so dS by 2^-9, and an element of dQ or dK (sums with
weights p that add up to about 1, |k| and |q| below 2^3) by scale 2^-6.
"""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

from test_window_gpu import cuda, make

pytestmark = pytest.mark.gpu


def check(got, exact, scale):
    want, size, moved = exact
    for name, g, w, s, m in zip(("dQ", "dK", "dV"), got, want, size, moved):
        g = g.float().cpu().numpy().astype(np.float64)
        assert np.isfinite(g).all(), name
        rest = abs(scale) * 2.0 ** -6
        far = np.abs(g - w)
        assert np.linalg.norm(far) <= 2.0 ** -7 * np.linalg.norm(w) + rest * np.sqrt(w.size), name
        most = 2.0 ** -8 * np.abs(w) + (2.0 ** -8 + 2.0 ** -12) * s + 2.0 ** -8 * m + rest
        assert (far <= most).all(), (name, float((far / most).max()))


def exact(*args):
    return o.window_backward(*args, magnitudes=True)


def run(q, k, v, do, window, sinks, lens=None, scale=None):
    q, k, v, do = (cuda(x) for x in (q, k, v, do))
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = bsa.window_forward(q, k, v, window, sinks, scale=scale, lens=n)
    got = bsa.window_backward(q, k, v, out, do, lse, window, sinks, scale=scale, lens=n)
    assert bsa.stream_status() == 0
    assert [x.stride() for x in got] == [x.stride() for x in (q, k, v)]
    return got


CASES = [  # B, H, Hkv, N, window, sinks
    (1, 1, 1, 1, 1, 0), (1, 2, 1, 2, 1, 1), (2, 3, 1, 17, 4, 2), (1, 1, 1, 128, 128, 0), (1, 2, 2, 129, 1, 0),
    (2, 4, 2, 300, 77, 3), (1, 3, 3, 511, 129, 33), (1, 2, 1, 700, 700, 0), (1, 6, 2, 513, 5000, 0),
    (1, 5, 1, 1000, 64, 200), (3, 2, 1, 385, 100, 32), (1, 1, 1, 1300, 1024, 4), (1, 2, 1, 900, 1, 900),
    (1, 2, 1, 1500, 30, 4),
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks", CASES)
def test_backward(B, H, Hkv, N, window, sinks, d):
    q, k, v, do = make(B, H, Hkv, N, d, 21)
    check(run(q, k, v, do, window, sinks), exact(q, k, v, do, window, sinks, d ** -0.5), d ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks,lens", [
    (4, 2, 1, 300, 50, 3, [0, 1, 129, 300]), (3, 3, 3, 257, 300, 0, [256, 255, 128]),
    (2, 4, 2, 900, 100, 40, [500, 0]), (2, 1, 1, 700, 20, 1, [127, 258]), (2, 2, 1, 1500, 40, 5, [1499, 300])])
def test_backward_of_padded_sequence_major_batches(B, H, Hkv, N, window, sinks, lens, d):
    q, k, v, do = make(B, H, Hkv, N, d, 22, seq_major=True)
    for b, n in enumerate(lens):  # what pads the batch may be anything
        for x in (q, k, v, do):
            x[b, :, n:] = float("nan")
    check(run(q, k, v, do, window, sinks, lens), exact(q, k, v, do, window, sinks, d ** -0.5, lens), d ** -0.5)


def test_backward_of_many_tiles_with_empty_ones_between():
    """More tiles than SMs, so that one block takes tiles with and without tokens in turn."""
    B, H, Hkv, N, d, lens = 4, 16, 4, 1900, 64, [1900, 0, 700, 1300]
    q, k, v, do = make(B, H, Hkv, N, d, 26)
    check(run(q, k, v, do, 150, 4, lens), exact(q, k, v, do, 150, 4, d ** -0.5, lens), d ** -0.5)


@pytest.mark.parametrize("N,window,sinks", [(1, 5, 3), (300, 1, 0), (130, 1, 1)])
def test_queries_that_see_one_key_have_no_gradient(N, window, sinks):
    q, k, v, do = make(2, 4, 2, N, 128, 27)
    dq, dk, dv = run(q, k, v, do, window, sinks)
    want = exact(q, k, v, do, window, sinks, 128 ** -0.5)
    check((dq, dk, dv), want, 128 ** -0.5)
    assert float(dq[:, :, 0].abs().max()) == 0
    if N == 1 or sinks == 0:
        assert float(dq.abs().max()) == 0 and float(dk.abs().max()) == 0


@pytest.mark.parametrize("scale", [-0.1, 0.0, 0.3])
def test_backward_scales(scale):
    q, k, v, do = make(1, 2, 1, 400, 128, 23)
    check(run(q, k, v, do, 150, 4, scale=scale), exact(q, k, v, do, 150, 4, scale), scale)


def test_oracle_gradients_against_differences():
    q, k, v, do = (x.double().numpy() for x in make(1, 2, 1, 23, 64, 24))
    grads = o.window_backward(q, k, v, do, 7, 2, 0.125)
    rng, eps = np.random.default_rng(0), 1e-6
    for i, x in enumerate((q, k, v)):
        step = rng.standard_normal(x.shape)
        args = [[q, k, v], [q, k, v]]
        args[0][i], args[1][i] = x + eps * step, x - eps * step
        hi, lo = (o.window_forward(*a, 7, 2, 0.125)[0] for a in args)
        np.testing.assert_allclose(((hi - lo) * do).sum() / (2 * eps), (grads[i] * step).sum(), rtol=1e-6)


def test_same_bits_on_two_streams_and_in_a_graph():
    q, k, v, do = (x.cuda() for x in make(2, 4, 2, 1000, 128, 25))
    out, lse = bsa.window_forward(q, k, v, 200, 4)
    first = bsa.window_backward(q, k, v, out, do, lse, 200, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = bsa.window_backward(q, k, v, out, do, lse, 200, 4)
    third = bsa.window_backward(q, k, v, out, do, lse, 200, 4)  # both at once
    torch.cuda.synchronize()
    ws = torch.full((bsa.window_backward_workspace_bytes(2, 4, 2, 1000, 128, 200, 4),), 255, dtype=torch.uint8,
                    device="cuda")  # NaN everywhere: nothing in it is read before it is written
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fourth = bsa.window_backward(q, k, v, out, do, lse, 200, 4, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    for got in (second, third, fourth):
        assert all(torch.equal(a, b) for a, b in zip(got, first))


@pytest.mark.parametrize("H,Hkv,d,window,sinks", [(2, 1, 64, 100, 0), (2, 2, 128, 300, 0), (1, 1, 128, 40, 3)])
def test_gradients_do_not_move_with_what_is_not_seen(H, Hkv, d, window, sinks):
    """Large finite values in rows that a row does not meet change no bit of its
    gradients: keys after a query or before its window, queries before a key."""
    N, cut = 900, 333
    q, k, v, do = (x.cuda() for x in make(1, H, Hkv, N, d, 28))

    def run(q, k, v, do):
        out, lse = bsa.window_forward(q, k, v, window, sinks)
        return bsa.window_backward(q, k, v, out, do, lse, window, sinks)

    first = run(q, k, v, do)
    large = [x.clone() for x in (k, v)]
    for x in large:
        x[:, :, cut:] *= 1e6
    assert torch.equal(run(q, *large, do)[0][:, :, :cut], first[0][:, :, :cut])
    large = [x.clone() for x in (k, v)]
    for x in large:
        x[:, :, sinks:cut] *= 1e6
    after = slice(cut + window - 1, None)
    assert torch.equal(run(q, *large, do)[0][:, :, after], first[0][:, :, after])
    large = [x.clone() for x in (q, do)]
    for x in large:
        x[:, :, :cut] *= 1e6
    for a, b in zip(run(large[0], k, v, large[1])[1:], first[1:]):
        assert torch.equal(a[:, :, cut:], b[:, :, cut:])


@pytest.mark.parametrize("B,H,Hkv,N,window,sinks,lens", [
    (1, 12, 1, 1100, 300, 0, None), (1, 7, 1, 1600, 200, 5, None), (2, 9, 3, 777, 5000, 3, [500, 777]),
    (1, 3, 1, 4100, 130, 140, None)])
@pytest.mark.parametrize("d", [64, 128])
def test_backward_with_few_key_tiles_and_many_heads(B, H, Hkv, N, window, sinks, lens, d):
    """Groups whose heads are cut into parts, evenly or not, whose sums are added up."""
    q, k, v, do = make(B, H, Hkv, N, d, 29)
    check(run(q, k, v, do, window, sinks, lens), exact(q, k, v, do, window, sinks, d ** -0.5, lens), d ** -0.5)
