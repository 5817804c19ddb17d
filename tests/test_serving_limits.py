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


def decode_slices(H=4, Nq=1, D=64, B=3, gap=0, order="bnh", **kw):
    """q and o as neighbouring slices of one tensor [B, Nq, 2 H + 4, D] (or head-major within a batch)."""
    row = (2 * H + 4) * D
    st = [Nq * row, D, row] if order == "bnh" else [Nq * row, Nq * D, D]
    o = A + 2 * (H * (D if order == "bnh" else Nq * D) + gap)
    return call_decode(q=A, o=o, strides=st * 2, B=B, H=H, Hkv=2, Nq=Nq, D=D, lse=1 << 50, kp=1 << 51, vp=1 << 52,
                       table=1 << 53, lens=1 << 54, ws=1 << 55, **kw)


def test_decode_refuses_an_output_in_its_query():
    for order in ("bnh", "bhn"):
        for Nq in (1, 3):
            room = 4 * 64 * (1 if order == "bnh" else Nq)  # behind o, before the next token's or batch's q
            for gap in (-8, -64, room + 8):
                assert decode_slices(Nq=Nq, gap=gap, order=order) == INVALID, (order, Nq, gap)


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_decode_takes_an_output_beside_its_query_in_one_tensor():
    for order in ("bnh", "bhn"):
        for Nq in (1, 3):
            for B in (1, 3):
                for gap in (0, 8, 4 * 64):
                    assert decode_slices(Nq=Nq, B=B, gap=gap * (1 if order == "bnh" else Nq), order=order) == NO_DEVICE
    # head-major q, token-major o, each in its own part of a batch's block of one tensor
    assert call_decode(q=A, o=A + 2 * 1024, strides=[2048, 192, 64, 2048, 64, 256], B=5, H=4, Nq=3,
                       lse=1 << 50) == NO_DEVICE
    assert call_decode(q=A, o=A + 2 * 760, strides=[2048, 192, 64, 2048, 64, 256], B=5, H=4, Nq=3,
                       lse=1 << 50) == INVALID


def test_decode_workspace_without_kv_heads_is_enough_for_any():
    for H in (1, 6, 8, 40, 64):
        for Nq in (1, 2, 5):
            for D in (64, 128):
                most = max(fattn.decode_workspace_bytes(2, H, Nq, D, Hkv) for Hkv in range(1, H + 1) if H % Hkv == 0)
                assert fattn.decode_workspace_bytes(2, H, Nq, D) == most
