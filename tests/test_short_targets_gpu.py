"""So many short sequences or entries that a warp takes one for itself (two for every CTA
that the device holds): cross attention of few rows, decode behind a shared prefix."""
import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests.test_cross_gpu import check_fwd
from tests.test_cross_gpu import make as make_cross
from tests.test_shared_gpu import check, make, ok, spare_for

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def lengths(B, most, seed):
    """Empty, of one token, around whole units, long among short; mostly short."""
    g = torch.Generator().manual_seed(seed)
    some = [0, 1, 2, 15, 16, 17, 95, 96, 97, 127, 128, 129, 191, 192, 193, 255, 256, 257, most]
    short = torch.randint(0, 60, (B,), generator=g).tolist()
    at = torch.randint(0, 4 * len(some), (B,), generator=g).tolist()
    return [min(some[i] if i < len(some) else n, most) for i, n in zip(at, short)]


@pytest.mark.parametrize("share,Nq", [(1, 1), (4, 2), (4, 4), (2, 13)])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 64), ("fp16", 128)])
def test_cross(dtype, D, share, Nq):
    """1, 8, 16 and 26 rows a K/V head."""
    Hkv, Nk = 4, 600
    B = sms() + 7
    assert B * Hkv >= 4 * sms()
    lens = lengths(B, Nk, D + Nq)
    q, k, v, _, t = make_cross(B, share * Hkv, Hkv, Nq, Nk, D, DT[dtype], Nq, lens)
    o, lse = fattn.fwd_cross(q, k, v, t)
    ok()
    check_fwd(q, k, v, lens, fattn._default_scale(D), o, lse)


@pytest.mark.parametrize("prefix", [0, 1, 100, 128, 200])
@pytest.mark.parametrize("once", [False, True])
@pytest.mark.parametrize("share,Nq", [(1, 1), (4, 2), (8, 2)])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 64), ("fp16", 128)])
def test_behind_a_prefix(dtype, D, share, Nq, once, prefix):
    """1, 8 and 16 rows; the prefix read by every sequence (in at most two units), and once."""
    Hkv, page = 16, 16
    B = sms() // 4 + 3
    assert B * Hkv >= 4 * sms()
    lens = lengths(B, 300, prefix + Nq)
    args, rows = make(B, share * Hkv, Hkv, D, DT[dtype], page, prefix, lens, Nq, prefix + B + D,
                      spare=spare_for(B, Hkv, D, page, once))
    o, lse = fattn.decode_shared(**args)
    ok()
    check(args, rows, fattn._default_scale(D), o, lse, "%s %d" % (once, prefix))


@pytest.mark.parametrize("once", [False, True])
def test_few_sequences_of_many_heads(once):
    """32 sequences at most are dealt out by every warp for itself."""
    Hkv = -(-4 * sms() // 30)
    lens = lengths(30, 300, 3)
    args, rows = make(30, Hkv, Hkv, 64, torch.float16, 32, 150, lens, 1, 4, spare=spare_for(30, Hkv, 64, 32, once))
    o, lse = fattn.decode_shared(**args)
    ok()
    check(args, rows, 0.125, o, lse)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N", [(2, 3, 200), (1, 5, 256), (8, 8, 1000), (2, 3, 129)])
def test_many_rows_have_the_dense_forwards_bits(B, H, N, D):
    """Queries and keys of one length, a head a K/V head, keys not cut into parts.  (bf16: in
    fp16 the weights are held 2^7 times their size, whose exponents round differently.)"""
    g = torch.Generator().manual_seed(N)
    q, k, v = (torch.randn(B, H, N, D, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    assert fattn.cross_workspace_bytes(B, H, N, N, D, H) == 16
    o, lse = fattn.fwd(q, k, v)
    o2, lse2 = fattn.fwd_cross(q, k, v)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
