"""How exact the window kernels are where the wider bounds of their other tests would
not tell: the LSE, and dQ over keys with an offset that all of them share; and where
they write."""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

from test_window_gpu import CASES, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks", CASES)
def test_lse(B, H, Hkv, N, window, sinks, d):
    """A score is up to d products added in fp32 in d / 16 steps, partial sums below 2^7
    here: off by at most 9 * 2^7 * 2^-23 before the scale of 2^-3 (d = 64) or less, so by
    less than 2^-15.  An exponential is off by 2^-22 (ex2.approx), its argument's rounding
    by 2^-24 of at most 2^5.  A sum of n terms is taken in eight, of n / 8 additions of
    2^-24 each at most: 2^-16.5 at 1300.  Together below 2^-14."""
    q, k, v, _ = make(B, H, Hkv, N, d, 61)
    _, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), window, sinks)
    assert bsa.stream_status() == 0
    _, want = o.window_forward(q, k, v, window, sinks, d ** -0.5)
    np.testing.assert_allclose(lse.cpu().numpy(), want, rtol=0, atol=2.0 ** -14)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,N,window,sinks,lens", [
    (1, 700, 200, 0, None), (2, 900, 64, 4, None), (1, 700, 64, 40, None), (3, 600, 5000, 0, [555]),
    (2, 900, 1, 3, None), (2, 1100, 130, 160, [1000])])
def test_an_offset_of_all_keys_leaves_dq_exact(G, N, window, sinks, lens, d):
    """Keys c + n with |c| sixteen times |n| in every channel, and sinks that draw much
    of the weight.  dS adds up to what the given O and D say, so c drops out of the
    formula's dQ but not out of dS's rounding errors e_k, unless their sum is taken off:
    then what is left of each is e_k (k_k - k'), k' a mean of other keys.

    A rounding error is at most 2^-8 of dS, and 2^-8 / sqrt 3 in the root mean square;
    errors of different terms are independent, so over all elements the square of the
    error is 2^-16 / 3 times sum dS^2 |k_k - k'|^2 <= 2 dS^2 (|n_k|^2 + max|n|^2), where
    the maximum is over the keys of the diagonal tile and their root mean square takes
    its place in the sum over all; dQ's own rounding adds 2^-16 / 3 |dQ|^2.  The bound
    takes 2^-16 for 2^-16 / 3, which also covers the weights' error (scores of about 2^6,
    off by 2^-17 or so: 2^-17 |c| is 2^-13 of |n|)."""
    g = torch.Generator().manual_seed(62)
    B, Hkv = 1, 2
    H = Hkv * G
    q, k, v, do = (torch.randn(B, h, N, d, generator=g) for h in (H, Hkv, Hkv, H))
    way = torch.randn(d, generator=g)
    way /= way.norm()
    q = q + 4 * way
    k[:, :, :sinks] += 8 * way
    c = 16 * torch.sign(torch.randn(Hkv, 1, d, generator=g))
    q, k, v, do = (x.to(torch.bfloat16) for x in (q, k + c, v, do))
    n = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), window, sinks, lens=n)
    dq = bsa.window_backward(q.cuda(), k.cuda(), v.cuda(), out, do.cuda(), lse, window, sinks, lens=n)[0]
    assert bsa.stream_status() == 0
    n, scale = N if lens is None else lens[0], d ** -0.5
    seen = o._mask(n, window, sinks)
    far = near = 0.0
    for h in range(H):
        qh, kh, vh, gh, oh = (x.double().cpu().numpy()[:n] for x in (q[0, h], k[0, h // G], v[0, h // G], do[0, h], out[0, h]))
        p = np.where(seen, np.exp(np.where(seen, scale * qh @ kh.T - lse[0, h, :n, None].double().cpu().numpy(), 0.0)), 0.0)
        ds = p * (gh @ vh.T - (gh * oh).sum(-1, keepdims=True)) * scale
        want = ds @ kh
        size = ((kh - c[h // G].double().numpy()) ** 2).sum(-1)
        far += ((dq[0, h, :n].double().cpu().numpy() - want) ** 2).sum()
        near += 2 * (ds ** 2 @ (size + size[sinks:].mean())).sum() + (want ** 2).sum()
    assert far <= 2.0 ** -16 * near, (far / near) ** 0.5 * 2 ** 8


@pytest.mark.parametrize("strides", [(240, 40, 1), (240, 1, 6), (1, 80, 2), (1, 2, 12), (40, 80, 1), (5000, 3, 100),
                                     (241, 40, 1)], ids=str)
@pytest.mark.parametrize("dk", [0, 8])
def test_an_out_in_any_order_of_its_dimensions(strides, dk):
    """Rows of every order and spacing that do not overlap; the bytes between them stay."""
    q, k, v, _ = (x.cuda() for x in make(2, 6, 3, 40, 64, 63))
    want, lse = bsa.window_forward(q, k, v, 8, 2)
    step = [(64 + dk) * s for s in strides]
    whole = torch.full((sum((n - 1) * s for n, s in zip((2, 6, 40), step)) + 64 + 8,), 7.0, dtype=torch.bfloat16,
                       device="cuda")
    out = whole.as_strided((2, 6, 40, 64), (*step, 1))
    got, other = bsa.window_forward(q, k, v, 8, 2, out=out)
    assert bsa.stream_status() == 0
    assert got is out and torch.equal(out, want) and torch.equal(other, lse)
    out.fill_(7.0)
    assert bool((whole == 7.0).all())
