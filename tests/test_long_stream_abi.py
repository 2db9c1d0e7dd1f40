"""Host-side argument checks of the long-stream entry points (no GPU: every call
fails a check made before any CUDA call, so the fake pointers are never used),
and the oracle's packing."""
import ctypes

import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from block_sparse_attention_38_b200 import long_stream as ls
from oracle import long_stream as o

P = 4096
P8 = 4104  # 8 mod 16
NAN = float("nan")


def _cache(**kw):
    f = dict(k_codes=P, k_params=P, v_codes=P, v_params=P, B=2, H=3, L=96, d=64)
    f.update(kw)
    return ls._Cache(*(f[n] for n, _ in ls._Cache._fields_))


BAD_CACHE = [dict(k_codes=None), dict(k_params=None), dict(v_codes=None), dict(v_params=None), dict(B=0),
             dict(H=0), dict(L=0), dict(d=0), dict(k_codes=P8), dict(v_params=P8)]


def _ids(kw):
    return ",".join(f"{k}={v}" for k, v in kw.items())


def _write(cache=None, k=None, v=None, start=P, T=4):
    view = lambda x: None if x == "null" else ls._View(*(x or (P, 64, 64, 64)))  # noqa: E731
    return bsa.library().bsa_q4_write(cache or _cache(), view(k), view(v), start, None, T, None)


@pytest.mark.parametrize("kw", BAD_CACHE, ids=_ids)
def test_cache_arguments(kw):
    lib, c = bsa.library(), _cache(**kw)
    assert _write(cache=c) == bsa.ERR_INVALID_ARG
    assert lib.bsa_q4_read(c, P, None, 4, P, P, None) == bsa.ERR_INVALID_ARG
    assert lib.bsa_q4_window_decode(P, None, None, c, P, 6, 8, 0, 0.1, P, P, None) == bsa.ERR_INVALID_ARG
    assert lib.bsa_q4_decode(P, None, None, c, P, P, P, 6, 32, 0.1, P, P, None) == bsa.ERR_INVALID_ARG


def test_unsupported_head_size():
    lib, c = bsa.library(), _cache(d=96)
    assert _write(cache=c) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_q4_read(c, P, None, 4, P, P, None) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_q4_window_decode(P, None, None, c, P, 6, 8, 0, 0.1, P, P, None) == bsa.ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(k="null"), dict(v="null"), dict(start=None), dict(T=0), dict(T=-1), dict(k=(None, 64, 64, 64)),
    dict(k=(P8, 64, 64, 64)), dict(v=(P, 4, 64, 64)), dict(v=(P, 64, 60, 64)), dict(v=(P, 64, 64, 65)),
    dict(k=(P, -64, 64, 64))], ids=_ids)
def test_write_arguments(kw):
    assert _write(**kw) == bsa.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(start=None), dict(T=0), dict(k=None), dict(v=P8)], ids=_ids)
def test_read_arguments(kw):
    a = dict(start=P, T=4, k=P, v=P)
    a.update(kw)
    assert bsa.library().bsa_q4_read(_cache(), a["start"], None, a["T"], a["k"], a["v"], None) == bsa.ERR_INVALID_ARG


BAD_STEP = [dict(q=None), dict(q=P8), dict(kn=P), dict(vn=P), dict(kn=P8, vn=P), dict(seq=None), dict(H=0),
            dict(H=4), dict(scale=NAN), dict(scale=float("inf")), dict(O=None), dict(O=P8), dict(LSE=None),
            dict(LSE=P + 2)]


@pytest.mark.parametrize("kw", BAD_STEP + [dict(window=0), dict(sinks=-1)], ids=_ids)
def test_window_step_arguments(kw):
    a = dict(q=P, kn=None, vn=None, seq=P, H=6, window=8, sinks=2, scale=0.1, O=P, LSE=P)
    a.update(kw)
    lib = bsa.library()
    assert lib.bsa_q4_window_decode(a["q"], a["kn"], a["vn"], _cache(), a["seq"], a["H"], a["window"], a["sinks"],
                                    a["scale"], a["O"], a["LSE"], None) == bsa.ERR_INVALID_ARG
    assert lib.bsa_window_decode(a["q"], a["kn"], a["vn"], P, P, a["seq"], 2, a["H"], 3, 96, 64, a["window"],
                                 a["sinks"], a["scale"], a["O"], a["LSE"], None) == bsa.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(kc=None), dict(vc=P8), dict(B=0), dict(Hkv=0), dict(L=0), dict(Hkv=5)], ids=_ids)
def test_bf16_step_arguments(kw):
    a = dict(kc=P, vc=P, B=2, Hkv=3, L=96)
    a.update(kw)
    assert bsa.library().bsa_window_decode(P, None, None, a["kc"], a["vc"], P, a["B"], 6, a["Hkv"], a["L"], 64, 8, 2,
                                           0.1, P, P, None) == bsa.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", BAD_STEP + [dict(rp=None), dict(ci=None), dict(bs=0), dict(bs=64)], ids=_ids)
def test_block_step_arguments(kw):
    a = dict(q=P, kn=None, vn=None, seq=P, H=6, rp=P, ci=P, bs=32, scale=0.1, O=P, LSE=P)
    a.update(kw)  # L = 96 is no multiple of 64
    assert bsa.library().bsa_q4_decode(a["q"], a["kn"], a["vn"], _cache(), a["rp"], a["ci"], a["seq"], a["H"],
                                       a["bs"], a["scale"], a["O"], a["LSE"], None) == bsa.ERR_INVALID_ARG


@pytest.mark.parametrize("L,bs", [(96, 16), (256, 256), (4097 * 32, 32)])
def test_block_step_unsupported(L, bs):
    assert bsa.library().bsa_q4_decode(P, None, None, _cache(L=L), P, P, P, 6, bs, 0.1, P, P,
                                       None) == bsa.ERR_UNSUPPORTED


def test_status_reader_rejects_null():
    assert bsa.library().bsa_stream_status(None, 0) == bsa.ERR_INVALID_ARG


def test_binding_refuses_cpu_tensors_and_other_shapes():
    c = bsa.q4_cache(1, 2, 32, 64, device="cpu")
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    n = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: bsa.q4_write(c, x, x, n), lambda: bsa.q4_read(c, n, 3),
                 lambda: bsa.q4_window_decode(q, c, n, 8),
                 lambda: bsa.q4_decode(q, c, n, n, n, 32),
                 lambda: bsa.window_decode(q, x, x, n, 8),
                 lambda: bsa.q4_write(c._replace(k_params=c.k_params[..., 0]), x, x, n)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("is_key", [True, False])
def test_packing_is_a_permutation_and_inverts(d, is_key):
    assert sorted(o.nibble_of(c, d, is_key) for c in range(d)) == list(range(d))
    codes = np.random.default_rng(0).integers(0, 16, (5, d)).astype(np.uint8)
    np.testing.assert_array_equal(o.unpack(o.pack(codes, is_key), is_key), codes)


def test_quantising_by_hand():
    x = np.zeros((1, 64))
    x[0, :32] = np.arange(32) / 2.0      # 0 .. 15.5: scale 15.5 / 15 in fp16
    x[0, 32:] = -3.0                     # constant: scale 0
    code, s, m = o.quantise(x)
    assert s[0, 0] == np.float16(15.5 / 15) and m[0, 0] == 0
    assert code[0, 0] == 0 and code[0, 31] == 15 and code[0, 1] == 0 and code[0, 2] == 1
    assert s[0, 1] == 0 and m[0, 1] == -3 and (code[0, 32:] == 0).all()
    assert np.abs(o.values(code, s, m) - x).max() <= 0.5 * s[0, 0] + 15 * 2.0 ** -11 * s[0, 0]


# ------------------------------------------------------- sliding-window attention
def _v(data=P, b=64, h=64, n=64):
    return ls._View(data, b, h, n)


SIZES = dict(B=2, H=6, Hkv=3, N=40, d=64, window=8, sinks=2, scale=0.1, LSE=P)
BAD_SIZES = [dict(B=0), dict(H=0), dict(Hkv=0), dict(H=7), dict(N=0), dict(d=0), dict(window=0), dict(sinks=-1),
             dict(scale=NAN), dict(LSE=None), dict(LSE=P + 2)]
BAD_VIEWS = [_v(None), _v(P8), _v(b=4), _v(h=60), _v(n=65), _v(n=0), _v(n=32), _v(b=-64), _v(n=1 << 39)]


def _forward(bad=None, at=0, **kw):
    a = dict(SIZES, **kw)
    v = [_v() for _ in range(4)]
    if bad is not None:
        v[at] = bad
    return bsa.library().bsa_window_forward(v[0], v[1], v[2], None, a["B"], a["H"], a["Hkv"], a["N"], a["d"],
                                            a["window"], a["sinks"], a["scale"], v[3], a["LSE"], None)


def _backward(bad=None, at=0, ws=P, nbytes=1 << 30, **kw):
    a = dict(SIZES, **kw)
    v = [_v() for _ in range(8)]
    if bad is not None:
        v[at] = bad
    return bsa.library().bsa_window_backward(*v[:5], a["LSE"], None, a["B"], a["H"], a["Hkv"], a["N"], a["d"],
                                             a["window"], a["sinks"], a["scale"], *v[5:], ws, nbytes, None)


@pytest.mark.parametrize("kw", BAD_SIZES, ids=_ids)
def test_window_sizes(kw):
    assert _forward(**kw) == bsa.ERR_INVALID_ARG
    assert _backward(**kw) == bsa.ERR_INVALID_ARG


@pytest.mark.parametrize("bad", range(len(BAD_VIEWS)))
def test_window_views(bad):
    for at in range(4):
        assert _forward(BAD_VIEWS[bad], at) == bsa.ERR_INVALID_ARG
    for at in range(8):
        assert _backward(BAD_VIEWS[bad], at) == bsa.ERR_INVALID_ARG


def test_window_unsupported_and_workspace():
    wide = [ls._View(P, 96, 96, 96) for _ in range(8)]
    lib = bsa.library()
    assert lib.bsa_window_forward(*wide[:3], None, 2, 6, 3, 40, 96, 8, 2, 0.1, wide[3], P, None) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_window_backward(*wide[:5], P, None, 2, 6, 3, 40, 96, 8, 2, 0.1, *wide[5:], P, 1 << 30,
                                   None) == bsa.ERR_UNSUPPORTED
    need = bsa.window_backward_workspace_bytes(2, 6, 3, 40, 64, 8, 2)
    assert _backward(nbytes=need - 1) == bsa.ERR_BUFFER_TOO_SMALL
    assert _backward(ws=None) == _backward(ws=P8) == bsa.ERR_INVALID_ARG


def test_workspace_sizes():
    size = bsa.window_backward_workspace_bytes
    assert size(1, 1, 1, 1, 64, 1) >= 4
    assert size(1, 4, 2, 4096, 128, 256, 4) > size(1, 4, 2, 4096, 128, 256, 0) >= 4 * 4 * 4096
    assert size(1, 4, 2, 4096, 128, 4096, 4) == size(1, 4, 2, 4096, 128, 4096, 0)  # no far queries
    # sinks cost two rows-times-channels sums for each chunk, whatever the length
    assert size(1, 1, 1, 1 << 20, 128, 128, 4) < 4 * (1 << 20) + (2 + 32) * 2 * 128 * 128 * 4
    for bad in ((1, 3, 2, 8, 64, 1), (1, 1, 1, 8, 96, 1), (1, 1, 1, 8, 64, 0), (0, 1, 1, 8, 64, 1)):
        with pytest.raises(ValueError):
            size(*bad)


def test_binding_refuses_cpu_and_broadcast_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        bsa.window_forward(x, x, x, 2)
    with pytest.raises(ValueError):
        bsa.window_forward(torch.zeros(1, 3, 3, 64, dtype=torch.bfloat16), x, x, 2)
    with pytest.raises(ValueError):
        bsa.window_backward(x, x, x, x, x, torch.zeros(1, 2, 3), 2)


def test_row_numbers_stay_within_an_int():
    lib, big = bsa.library(), (1 << 30) + 1
    c = _cache(L=big)
    assert _write(cache=c) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_q4_read(c, P, None, 4, P, P, None) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_q4_read(_cache(), P, None, big, P, P, None) == bsa.ERR_UNSUPPORTED
    assert _write(T=(1 << 31) - 1) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_q4_window_decode(P, None, None, c, P, 6, 8, 0, 0.1, P, P, None) == bsa.ERR_UNSUPPORTED
    assert lib.bsa_window_decode(P, None, None, P, P, P, 2, 6, 3, big, 64, 8, 2, 0.1, P, P, None) == bsa.ERR_UNSUPPORTED
