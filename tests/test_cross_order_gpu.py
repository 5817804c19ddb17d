"""Calls that follow one another on a stream without a wait, over the same tensors and
workspaces: each sees what the call before it left, and nothing older."""
import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests.test_cross_gpu import make, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", [(2, 4, 2, 150, 300), (8, 19, 19, 500, 100), (8, 19, 19, 500, 300), (8, 16, 16, 60, 1500),
                                  (1, 32, 4, 3, 4000), (2, 2, 1, 40, 20000)])
def test_gradients_in_a_row(case, D):
    """Two sets of inputs, lengths and statistics take turns in the same buffers (query tiles and key blocks one
    each, in runs, in parts; fp16, whose statistics have a scale): every call gives the bits that it gives alone."""
    B, H, Hkv, Nq, Nk = case
    sets = [make(B, H, Hkv, Nq, Nk, D, torch.float16, s, [max(0, Nk - 37 * (b + s)) for b in range(B)], fill=0.5, q_std=0.5 + s)
            for s in (0, 1)]
    sets[1][3].mul_(3.0)
    outs, alone = [], []
    for q, k, v, do, t in sets:
        outs.append(fattn.fwd_cross(q, k, v, t))
        alone.append(fattn.bwd_cross(q, k, v, *outs[-1], do, t))
        ok()
    q, k, v, do, t = (torch.empty_like(x) for x in sets[0])
    o, lse = (torch.empty_like(x) for x in outs[0])
    ws = torch.empty(fattn.bwd_cross_workspace_bytes(B, H, Nq, Nk, D, Hkv), dtype=torch.uint8, device="cuda")
    got = []
    for i in range(8):
        for x, y in zip((q, k, v, do, t, o, lse), sets[i % 2] + tuple(outs[i % 2])):
            x.copy_(y)
        got.append(fattn.bwd_cross(q, k, v, o, lse, do, t, workspace=ws))
    ok()
    for i, grads in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(alone[i % 2], grads))
