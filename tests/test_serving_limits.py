"""Sizes and views at the limits of the serving entry points: what is refused and
what is not, before any CUDA call."""
import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests.test_serving_abi import A, INVALID, NO_DEVICE, UNSUPPORTED, call_append, call_decode


def test_products_of_sizes_past_64_bits_are_refused():
    """Page strides and table lengths whose extents in bytes would wrap around."""
    for P, stride in ((4096, 1 << 52), (1 << 20, 1 << 44), (3, 1 << 51), (1 << 30, 1 << 33)):
        assert call_append(P=P, page_stride=stride) == UNSUPPORTED
        assert call_decode(P=P, page_stride=stride) == UNSUPPORTED
    for kv4 in (False, True):
        # tables that run into the cache however long they are
        for rows in (1 << 30, 1 << 31, 1 << 55, 1 << 57, 1 << 62):
            assert call_append(kv4, cos=6 * A - 4096, max_pos=rows) == INVALID, rows
            assert call_append(kv4, sin=6 * A - 4096, max_pos=rows) == INVALID, rows


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_sizes_within_the_limits_are_accepted():
    far = dict(kp=1 << 58, vp=1 << 59)
    assert call_append(P=4, page_stride=1 << 50, **far) == NO_DEVICE
    assert call_decode(P=4, page_stride=1 << 50, **far) == NO_DEVICE
    assert call_append(P=1, page_stride=1 << 52, **far) == NO_DEVICE
    assert call_append(max_pos=1 << 62, cos=20 * A, sin=30 * A) == NO_DEVICE  # rows that no int32 position names
