"""The serving operators at the edges of what their contracts allow, against plain
64-bit forms (tests/serving_ref.py)."""

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import serving_ref as R
from tests.test_packed_gpu import check_packed, make

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}

def ok():
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 0


# 1e-60 is 0 in 32 bits; 1e-42 is not, but far below the smallest normal number
@pytest.mark.parametrize("scale", [0.0, 1e-60, 1e-42])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp16", 128), ("bf16", 64)])
def test_scale_zero_is_the_mean_of_the_visible_values(dtype, D, causal, scale):
    """Every visible key weighs the same: O is their values' mean, LSE ln of their number."""
    q, k, v, cu = make([1, 127, 129, 300, 256, 5], 4, 2, D, DT[dtype], D, gaps=(2, 3))
    o, lse = fattn.fwd_packed(q, k, v, cu, causal=causal, scale=scale)
    ok()
    check_packed(q, k, v, cu, causal, scale, o, lse, "packed")
    for N in (1, 127, 129, 300):
        g = torch.Generator().manual_seed(N)
        q, k, v = (torch.randn(1, h, N, D, generator=g).to(DT[dtype]).cuda() for h in (4, 2, 2))
        o, lse = fattn.fwd(q, k, v, causal=causal, scale=scale)
        ok()
        one = torch.tensor([0, N], dtype=torch.int32)
        check_packed(*(t[0].transpose(0, 1) for t in (q, k, v)), one, causal, scale, o[0].transpose(0, 1), lse[0], "dense")
