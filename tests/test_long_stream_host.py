"""What the long-stream calls decide on the host (no GPU: nothing is launched, and fake
pointers are never used)."""
import pytest

import block_sparse_attention_38_b200 as bsa
from block_sparse_attention_38_b200 import long_stream as ls

P = 4096  # never used as a pointer


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,N,window,sinks", [
    (1, 8, 1, 4096, 128, 4), (1, 64, 1, 7552, 1, 1), (1, 8, 1, 7552, 128, 4), (2, 9, 3, 777, 300, 3),
    (1, 32, 8, 8192, 1024, 4), (1, 4, 1, 4100, 130, 300), (1, 1, 1, 1 << 20, 128, 4), (1, 16, 2, 2048, 512, 0)])
def test_backward_workspace_is_no_more_than_its_parts(B, H, Hkv, N, window, sinks, d):
    """A row's D, 4 bytes, and fp32 sums of dK and dV: where fewer than 60 key tiles leave
    their heads' sums in parts, as many as make 60 items, and no more than a tile has
    heads; and of sink tiles in up to 32 chunks.  Tiles without sinks have no chunks."""
    tiles = -(-N // 128)
    tile = 2 * 128 * d * 4
    group = H // Hkv
    items = B * Hkv * tiles
    parts = min(group, -(-60 // items)) if items < 60 else 1
    sunk = -(-min(sinks, N) // 128)
    most = B * H * N * 4 + 256 + B * Hkv * tile * ((tiles if parts > 1 else sunk) * parts + sunk * 32)
    assert B * H * N * 4 <= bsa.window_backward_workspace_bytes(B, H, Hkv, N, d, window, sinks) <= most


# strides in units of d = 64 of [B, H, N] = [2, 6, 40]
OVERLAPPING = [(2, 1, 1), (240, 1, 1), (1, 1, 6), (40, 40, 1), (240, 1, 5), (239, 40, 1), (120, 1, 2)]


@pytest.mark.parametrize("strides", OVERLAPPING, ids=str)
def test_outputs_whose_rows_overlap_are_refused(strides):
    lib, sizes = bsa.library(), (2, 6, 6, 40, 64, 8, 2, 0.1)
    bad, good = (ls._View(P, *(64 * s for s in x)) for x in (strides, (240, 40, 1)))
    assert lib.bsa_window_forward(good, good, good, None, *sizes, bad, P, None) == bsa.ERR_INVALID_ARG
    for at in range(3):
        grads = [bad if i == at else good for i in range(3)]
        assert lib.bsa_window_backward(*[good] * 5, P, None, *sizes, *grads, P, 1 << 30, None) == bsa.ERR_INVALID_ARG
