"""The 4-bit cache on the GPU against its fp64 oracle: codes and parameters bit
for bit, values read back to bf16's rounding, and which rows are touched."""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

pytestmark = pytest.mark.gpu


def _rows(shape, seed, kind="plain"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "offset":
        x = x + 3 * torch.randn(shape[1], 1, shape[3], generator=g)
    elif kind == "tiny":
        x = x * 1e-5
    elif kind == "grid":
        x = torch.round(x * 8) / 8           # many ties between two codes
    elif kind == "flat":
        x = x[..., :1].expand(shape).clone()  # constant groups
    elif kind == "wide":
        x = x * 1e5                          # past fp16's range
    return x.to(torch.bfloat16)


def _np(t):
    return t.cpu().numpy()


def _check_rows(cache, b, h, rows, k, v):
    """Cached rows equal the oracle's quantisation of k, v [n, d]."""
    for x, codes, params, is_key in ((k, cache.k_codes, cache.k_params, True),
                                     (v, cache.v_codes, cache.v_params, False)):
        want, s, m = o.quantise(x)
        got = _np(codes)[b, h][rows]
        np.testing.assert_array_equal(got, o.pack(want, is_key))
        par = _np(params)[b, h][rows]
        np.testing.assert_array_equal(par[..., 0], s)
        np.testing.assert_array_equal(par[..., 1], m)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,T,L", [(1, 1, 1, 1), (2, 3, 1, 40), (3, 2, 65, 90), (1, 5, 257, 300)])
@pytest.mark.parametrize("kind", ["plain", "offset", "tiny", "grid", "flat", "wide"])
def test_write_and_read(B, H, T, L, d, kind):
    k, v = _rows((B, H, T, d), 1, kind), _rows((B, H, T, d), 2, kind)
    cache = bsa.q4_cache(B, H, L, d)
    for t in cache:
        t.fill_(3)  # rows outside the ranges keep this
    start = torch.tensor([(7 * b) % (L - T + 1) for b in range(B)], dtype=torch.int32)
    lens = torch.tensor([T - (b * 3) % (T + 1) for b in range(B)], dtype=torch.int32)
    bsa.q4_write(cache, k.cuda(), v.cuda(), start.cuda(), lens=lens.cuda())
    kr, vr = bsa.q4_read(cache, start.cuda(), T, lens=lens.cuda())
    assert bsa.stream_status() == 0
    for b in range(B):
        s, n = int(start[b]), int(lens[b])
        for h in range(H):
            _check_rows(cache, b, h, slice(s, s + n), k[b, h, :n], v[b, h, :n])
            others = np.r_[0:s, s + n:L]
            for t in cache:
                assert (_np(t)[b, h][others] == 3).all()
            for got, x in ((kr, k), (vr, v)):
                want = o.values(*o.quantise(x[b, h, :n]))
                got = got[b, h].float().cpu().numpy()
                # one rounding of the fp32 sum (2^-24 of the value) and one to bf16 (2^-8)
                np.testing.assert_allclose(got[:n], want, rtol=2.0 ** -8 + 2.0 ** -20, atol=1e-30)
                assert (got[n:] == 0).all()


def test_strided_and_shared_inputs():
    B, H, T, d, L = 2, 3, 50, 128, 64
    k = _rows((B, T, H, d), 3).transpose(1, 2)                       # sequence-major
    v = _rows((1, H, T, 2 * d), 4)[..., d:].expand(B, H, T, d)       # a slice, shared by the batch
    start = torch.tensor([0, 14], dtype=torch.int32, device="cuda")
    cache = bsa.q4_cache(B, H, L, d)
    kc = k.transpose(1, 2).cuda().transpose(1, 2)
    vc = _rows((1, H, T, 2 * d), 4).cuda()[..., d:].expand(B, H, T, d)
    bsa.q4_write(cache, kc, vc, start)
    assert bsa.stream_status() == 0
    for b in range(B):
        for h in range(H):
            s = int(start[b])
            _check_rows(cache, b, h, slice(s, s + T), k[b, h], v[b, h])


def test_nan_and_infinity_stay_in_their_group():
    k = _rows((1, 1, 4, 64), 5)
    k[0, 0, 1, 3] = float("nan")
    k[0, 0, 2, 40] = float("inf")
    v = _rows((1, 1, 4, 64), 6)
    cache = bsa.q4_cache(1, 1, 4, 64)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.q4_write(cache, k.cuda(), v.cuda(), start)
    got = bsa.q4_read(cache, start, 4)[0].float().cpu().numpy()[0, 0]
    want = o.values(*o.quantise(k[0, 0]))
    assert np.isnan(got[1, :32]).all() and np.isfinite(got[1, 32:]).all()
    assert np.isfinite(got[2]).all()
    np.testing.assert_allclose(got, want, rtol=2.0 ** -8 + 2.0 ** -20)


def test_bad_ranges_are_reported_and_leave_the_cache():
    B, L, T, d = 5, 32, 8, 64
    k = _rows((B, 2, T, d), 7).cuda()
    cache = bsa.q4_cache(B, 2, L, d)
    start = torch.tensor([25, -1, 0, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # b = 3 is good
    lens = torch.tensor([8, 8, 9, 0, 8], dtype=torch.int32, device="cuda")
    bsa.q4_write(cache, k, k, start, lens=lens)
    assert bsa.stream_status() == bsa.STATUS_BAD_SEQ_LEN
    assert all(int(t.count_nonzero()) == 0 for t in cache)
    out = (torch.full_like(k, 5), torch.full_like(k, 5))
    bsa.q4_read(cache, start, T, lens=lens, out=out)
    assert bsa.stream_status() == bsa.STATUS_BAD_SEQ_LEN
    assert float(out[0].abs().sum()) == 0 and float(out[1].abs().sum()) == 0


def test_rows_past_two_to_the_31_bytes():
    """A cache whose last rows lie past 2^31 bytes of codes."""
    B, H, L, d = 1, 4, 8_400_000, 128
    cache = bsa.Q4Cache(*(torch.empty(s, dtype=t, device="cuda") for s, t in (
        ((B, H, L, d // 2), torch.uint8), ((B, H, L, d // 32, 2), torch.float16),
        ((B, H, L, d // 2), torch.uint8), ((B, H, L, d // 32, 2), torch.float16))))
    k = _rows((B, H, 3, d), 8)
    start = torch.tensor([L - 3], dtype=torch.int32, device="cuda")
    bsa.q4_write(cache, k.cuda(), k.cuda(), start)
    kr, vr = bsa.q4_read(cache, start, 3)
    want = o.values(*o.quantise(k))
    np.testing.assert_allclose(kr.float().cpu().numpy(), want, rtol=2.0 ** -8 + 2.0 ** -20)
    np.testing.assert_allclose(vr.float().cpu().numpy(), want, rtol=2.0 ** -8 + 2.0 ** -20)
    q = torch.randn(B, H, d).to(torch.bfloat16)
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    got, lse = bsa.q4_window_decode(q.cuda(), cache, n, window=3)
    assert bsa.stream_status() == 0
    O, _ = o.decode(q, want, want, [3], lambda b, h, t: np.arange(3), d ** -0.5)
    np.testing.assert_allclose(got.float().cpu().numpy(), O, rtol=2.0 ** -7, atol=2.0 ** -8)


def test_out_may_be_a_sequence_that_makes_its_items():
    """What `out` gives is held for the call, also where nothing else holds it."""
    cache = bsa.q4_cache(1, 2, 40, 64)
    x = torch.randn(1, 2, 40, 64, device="cuda").to(torch.bfloat16)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    bsa.q4_write(cache, x, -x, zero)

    class Pair:
        def __len__(self):
            return 2

        def __getitem__(self, i):
            return torch.empty(1, 2, 40, 64, dtype=torch.bfloat16, device="cuda")

    got, want = bsa.q4_read(cache, zero, 40, out=Pair()), bsa.q4_read(cache, zero, 40)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
