"""Queries of no heads beside keys that have some: what belongs to the keys is computed."""
import math

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import serving_ref as R
from tests.test_cross_gpu import ok

pytestmark = pytest.mark.gpu


def test_rotate_turns_the_keys():
    g = torch.Generator().manual_seed(1)
    kv = torch.randn(2, 70, 6, 64, generator=g).half().cuda()
    q, k = kv[:, :, :0].transpose(1, 2), kv[:, :, 1:4].transpose(1, 2)
    pos = torch.randint(0, 99, (3, 2, 70), generator=g, dtype=torch.int32).cuda()
    cos, sin = (x.cuda() for x in R.tables(99, 64))
    axes = bytes(i % 3 for i in range(32))
    for more in (dict(axes=axes, pos=pos), dict(axes=None, pos=pos[0].contiguous(), inverse=True, interleaved=True)):
        want, _ = fattn.rotate(k, cos=cos, sin=sin, **more)
        qo, ko = fattn.rotate(q, cos=cos, sin=sin, k=k, k_out=torch.full((2, 3, 70, 64), math.nan).half().cuda(), **more)
        ok()
        assert qo.shape == (2, 0, 70, 64) and torch.equal(ko, want)


def test_gradients_of_the_keys_are_zeros():
    q = torch.empty(2, 0, 5, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(2, 3, 130, 64, device="cuda").bfloat16()
    o, lse = fattn.fwd_cross(q, k, k)
    assert o.shape == q.shape and lse.shape == (2, 0, 5)
    dq, dk, dv = fattn.bwd_cross(q, k, k, o, lse, o, dk=torch.full_like(k, math.nan), dv=torch.full_like(k, math.nan))
    ok()
    assert dq.shape == q.shape and (dk == 0).all() and (dv == 0).all()
