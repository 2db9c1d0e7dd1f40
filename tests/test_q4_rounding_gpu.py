"""Codes of the 4-bit cache where x - minimum is not a number of fp32's, against the
fp64 oracle, bit for bit."""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

from test_q4_gpu import _check_rows

pytestmark = pytest.mark.gpu


def _written(k, v, append):
    """k, v [T, d] written row by row by a decode step, or by q4_write."""
    T, d = k.shape
    cache = bsa.q4_cache(1, 1, T, d)
    k, v = k.cuda(), v.cuda()
    if not append:
        bsa.q4_write(cache, k[None, None], v[None, None], torch.zeros(1, dtype=torch.int32, device="cuda"))
    else:
        q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")
        for t in range(T):
            n = torch.tensor([t + 1], dtype=torch.int32, device="cuda")
            bsa.q4_window_decode(q, cache, n, 1, k_new=k[t][None, None], v_new=v[t][None, None])
    assert bsa.stream_status() == 0
    return cache


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_hair_below_a_tie(d, append):
    """Minimum -3.75 and maximum 3.75 give s = 1/2, and 0 is a tie: +-2^-40 are on
    either side of it, though fp32 takes both differences for 3.75."""
    x = torch.zeros(6, d)
    x[:, 0::32], x[:, 1::32] = -3.75, 3.75
    x[0, 2::32], x[0, 3::32] = -2.0 ** -40, 2.0 ** -40
    x[1, 2::32], x[1, 3::32] = -2.0 ** -100, 0.0
    x[2, 4::32] = -3.0                                 # ties that fp32 holds
    x[3:] *= -1
    x[4, 0::32] = 40.0                                 # other scales
    x[5] = x[0] * 2.0 ** -12
    x = x.to(torch.bfloat16)
    code = o.quantise(x[:1])[0]
    assert code[0, 2] == 7 and code[0, 3] == 8
    _check_rows(_written(x, -x, append), 0, 0, slice(0, 6), x, -x)


@pytest.mark.parametrize("d", [64, 128])
def test_values_of_all_sizes_in_one_group(d):
    g = torch.Generator().manual_seed(51)
    x = torch.randn(4000, d, generator=g) * 2.0 ** torch.randint(-60, 12, (4000, d), generator=g)
    x[::2] = torch.round(x[::2] * 4) / 4 + torch.where(torch.rand(2000, d, generator=g) < 0.3, -2.0 ** -50, 0.0)
    x = x.to(torch.bfloat16)
    _check_rows(_written(x, x.flip(0), False), 0, 0, slice(0, 4000), x, x.flip(0))


@pytest.mark.parametrize("append", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_a_group_of_infinities_is_limited_like_one_of_them(d, append):
    x = torch.randn(4, d, generator=torch.Generator().manual_seed(52))
    x[0, :32] = float("inf")
    x[1, 32:64] = -float("inf")
    x[2, :32], x[2, 5] = float("inf"), -float("inf")
    x[3, :32], x[3, 7] = -float("inf"), 1.0
    x = x.to(torch.bfloat16)
    cache = _written(x, -x, append)
    k, v = bsa.q4_read(cache, torch.zeros(1, dtype=torch.int32, device="cuda"), 4)
    top = torch.tensor(65504.0).to(torch.bfloat16)     # rounds to 2^16
    assert bool((k[0, 0, 0, :32].cpu() == top).all()) and bool((k[0, 0, 1, 32:64].cpu() == -top).all())
    assert bool((v[0, 0, 0, :32].cpu() == -top).all()) and bool((v[0, 0, 1, 32:64].cpu() == top).all())
    assert bool(torch.isfinite(k).all()) and bool(torch.isfinite(v).all())
    _check_rows(cache, 0, 0, slice(0, 4), x, -x)
