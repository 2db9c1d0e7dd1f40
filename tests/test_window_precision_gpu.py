"""How exact the window kernels are where the wider bounds of their other tests would
not tell: the LSE, and dQ over keys with an offset that all of them share."""
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
