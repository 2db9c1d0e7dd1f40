"""What the long-stream calls raise on a GPU."""
import pytest
import torch

import block_sparse_attention_38_b200 as bsa

pytestmark = pytest.mark.gpu


def test_an_output_that_does_not_fit_raises_torch_s_own_error():
    """2^30 rows of 128 bf16 are 256 GiB, more than the device has; nothing is launched."""
    cache = bsa.q4_cache(1, 1, 8, 128)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(torch.OutOfMemoryError):
        bsa.q4_read(cache, start, 1 << 30)
    k, _ = bsa.q4_read(cache, start, 8)
    assert float(k.abs().sum()) == 0 and bsa.stream_status() == 0
