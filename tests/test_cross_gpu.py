"""Cross attention (fwd_cross, bwd_cross) against plain 64-bit forms."""
import math

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import more_ref as M
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def ok():
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 0


def make(B, H, Hkv, Nq, Nk, D, dt, seed, lens=None, fill=math.nan, q_std=1.5):
    """q and the gradient as [B, Nq, H, D] seen as [B, H, Nq, D]; k and v slices of
    one projection of the states; `fill` lies behind each entry's keys."""
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(B, Nq, H, D, generator=g) * q_std).to(dt)
    kv = torch.randn(B, Nk, 2 * Hkv, D, generator=g).to(dt)
    do = torch.randn(B, Nq, H, D, generator=g).to(dt)
    lens = [Nk] * B if lens is None else lens
    for b, n in enumerate(lens):
        kv[b, n:] = fill
    q, kv, do = q.cuda(), kv.cuda(), do.cuda()
    return (q.transpose(1, 2), kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2), do.transpose(1, 2),
            torch.tensor(lens, dtype=torch.int32).cuda())


def check_fwd(q, k, v, lens, scale, o, lse, what=""):
    dt, D = q.dtype, q.shape[-1]
    ro, rl, av, worst = M.cross(q.cpu(), k.cpu(), v.cpu(), lens, scale)
    # (bf16 divides by the sum of the rounded weights: twice the rounding, as for packed prompts)
    bo, bl = R.attend_bounds(ro, torch.where(torch.isinf(rl), 0.0, rl), av, worst, D, dt, 2 * R.u_of(dt))
    R.check(o, ro, bo, what + " O")
    M.check_rows_without_keys(o.cpu(), lse.cpu(), lens)
    some = torch.tensor([n > 0 for n in lens])
    if some.any():
        R.check(lse.cpu()[some], rl[some], bl[some], what + " LSE")


# (B, H, Hkv, Nq, Nk, lens): both sides of 32 rows a K/V head (the streaming kernel and the tensor-core
# forward), keys around tile borders, rows around tile borders, heads stacked in one tile, entries without keys.
FORWARD = [
    (2, 4, 2, 1, 1, [1, 0]), (3, 8, 2, 1, 300, [300, 17, 0]), (2, 8, 1, 4, 129, [129, 128]),   # <= 32 rows
    (1, 4, 4, 33, 1, None), (2, 4, 1, 9, 40, [40, 0]), (2, 6, 2, 43, 257, [257, 128]),          # stacked heads
    (3, 2, 2, 127, 500, [500, 0, 129]), (1, 2, 1, 128, 128, None), (2, 2, 2, 129, 127, [127, 1]),
    (1, 3, 1, 257, 1000, [999]), (2, 4, 2, 300, 260, [256, 260]), (1, 1, 1, 700, 64, None),
    (4, 8, 8, 64, 2500, [2500, 1, 0, 1300]),                                                    # keys cut into parts
]


@pytest.mark.parametrize("case", FORWARD)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 64), ("fp16", 128)])
def test_forward(dtype, D, case):
    """NaN lies behind every entry's keys."""
    B, H, Hkv, Nq, Nk, lens = case
    q, k, v, _, t = make(B, H, Hkv, Nq, Nk, D, DT[dtype], Nq + Nk, lens)
    o, lse = fattn.fwd_cross(q, k, v, t)
    ok()
    check_fwd(q, k, v, lens or [Nk] * B, fattn._default_scale(D), o, lse, str(case))


@pytest.mark.parametrize("Nq", [1, 40, 300])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_forward_layouts(dtype, D, Nq):
    """Contiguous tensors, no lengths, outputs by strides, no lse: the same bits."""
    q, k, v, _, _ = make(2, 4, 2, Nq, 333, D, DT[dtype], 5)
    o, lse = fattn.fwd_cross(q, k, v)
    out = torch.full((2, Nq, 7, D), 7.0, dtype=q.dtype, device="cuda")
    o2, l2 = fattn.fwd_cross(q.contiguous(), k.contiguous(), v.contiguous(), out=out[:, :, 2:6].transpose(1, 2))
    o3, l3 = fattn.fwd_cross(q, k, v, return_lse=False)
    ok()
    assert torch.equal(o, o2) and torch.equal(o, o3) and torch.equal(lse, l2) and l3 is None
    assert (out[:, :, :2] == 7).all() and (out[:, :, 6:] == 7).all()
    check_fwd(q, k, v, [333, 333], fattn._default_scale(D), o, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_equals_the_dense_forward(D):
    """Nq = Nk, one head a K/V head: fwd's bits."""
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(2, 3, 520, D, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    o, lse = fattn.fwd(q, k, v)
    ws = fattn.cross_workspace_bytes(2, 3, 520, 520, D, 3)
    o2, lse2 = fattn.fwd_cross(q, k, v)
    ok()
    if ws <= 16:
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    else:  # keys cut into parts: sums in another order
        assert (o.float() - o2.float()).abs().max() <= 2 ** -7 * o.float().abs().max() and (lse - lse2).abs().max() <= 1e-5


def test_many_entries_and_lengths():
    """More entries than a CTA's warps list at once, each with a length of its own."""
    g = torch.Generator().manual_seed(2)
    for Nq in (1, 20):
        lens = torch.randint(0, 200, (300,), generator=g).tolist()
        q, k, v, _, t = make(300, 4, 2, Nq, 200, 64, torch.float16, 3, lens)
        o, lse = fattn.fwd_cross(q, k, v, t)
        ok()
        check_fwd(q, k, v, lens, 0.125, o, lse)


def test_large_scores_and_scale_zero():
    for Nq in (2, 200):
        q, k, v, _, t = make(2, 4, 2, Nq, 700, 128, torch.bfloat16, 4, [700, 300], q_std=30.0)
        for scale in (fattn._default_scale(128), 0.0):
            o, lse = fattn.fwd_cross(q, k, v, t, scale=scale)
            ok()
            check_fwd(q, k, v, [700, 300], scale, o, lse)


@pytest.mark.parametrize("Nq", [1, 100])
def test_lengths_out_of_range_are_cut_and_reported(Nq):
    q, k, v, do, _ = make(2, 2, 1, Nq, 150, 64, torch.float16, 6)
    bad, good = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([-5, 151], [0, 150]))
    want, lw = fattn.fwd_cross(q, k, v, good)
    ok()
    got, lg = fattn.fwd_cross(q, k, v, bad)
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 1
    assert torch.equal(want, got) and torch.equal(lw, lg)
    a = fattn.bwd_cross(q, k, v, want, lw, do, good)
    ok()
    b = fattn.bwd_cross(q, k, v, want, lw, do, bad)
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 1
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_keys_at_all():
    """Nk = 0, and every kv_len 0: zeros, whatever the outputs held."""
    for Nq in (1, 70):
        q = torch.randn(2, 4, Nq, 64, device="cuda").half()
        k = torch.empty(2, 2, 0, 64, device="cuda").half()
        o, lse = fattn.fwd_cross(q, k, k, out=torch.full_like(q, math.nan))
        dq, dk, dv = fattn.bwd_cross(q, k, k, o, lse, q, dq=torch.full_like(q, math.nan))
        ok()
        assert (o == 0).all() and (lse == -math.inf).all() and (dq == 0).all() and dk.shape == k.shape
    q = torch.empty(2, 4, 0, 64, device="cuda").half()
    k = torch.randn(2, 2, 130, 64, device="cuda").half()
    o, lse = fattn.fwd_cross(q, k, k)
    dq, dk, dv = fattn.bwd_cross(q, k, k, o, lse, q, dk=torch.full_like(k, math.nan), dv=torch.full_like(k, math.nan))
    ok()
    assert (dk == 0).all() and (dv == 0).all()


BACKWARD = [
    (1, 1, 1, 1, 1, None), (2, 4, 2, 1, 130, [130, 0]), (2, 4, 1, 17, 40, [40, 3]), (1, 2, 2, 128, 128, None),
    (2, 2, 1, 129, 257, [257, 128]), (2, 6, 2, 43, 300, [129, 300]), (1, 2, 2, 300, 127, [126]), (3, 2, 2, 260, 64, [64, 0, 33]),
    (1, 4, 4, 70, 900, [900]), (1, 8, 2, 600, 200, None),
    (2, 6, 2, 2, 200, [200, 64]), (1, 10, 2, 25, 130, None), (2, 12, 2, 30, 90, [90, 17]), (1, 7, 1, 20, 300, None),  # stacked heads
    (3, 8, 1, 1, 129, [129, 0, 128]), (1, 24, 1, 11, 70, None),
]


@pytest.mark.parametrize("case", BACKWARD)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 64), ("fp16", 128)])
def test_backward(dtype, D, case):
    B, H, Hkv, Nq, Nk, lens = case
    dt = DT[dtype]
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, D, dt, Nq + 3 * Nk, lens)
    scale = fattn._default_scale(D)
    lens = lens or [Nk] * B
    o, lse = fattn.fwd_cross(q, k, v, t)
    dq, dk, dv = (torch.full(x.shape, math.nan, dtype=dt, device="cuda") for x in (q, k, v))
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, dq=dq, dk=dk, dv=dv)
    ok()
    args = [x.cpu() for x in (q, k, v, do)]
    ref = M.cross_grads(*args, lens, scale)
    bounds = M.cross_grad_bounds(*args, lens, scale, dt, ref)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, bounds):
        R.check(x, r, b, "%s %s" % (name, case))
    for b, n in enumerate(lens):
        assert (got[1][b, :, n:] == 0).all() and (got[2][b, :, n:] == 0).all()
        if n == 0:
            assert (got[0][b] == 0).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_backward_many_blocks(dtype, D):
    """So many key blocks and query tiles that none is cut into parts; entries without keys, of one key, of a tile."""
    dt, lens = DT[dtype], [300, 0, 1, 128, 299, 129, 300, 257, 64, 300]
    q, k, v, do, t = make(10, 8, 8, 260, 300, D, dt, 77, lens)
    o, lse = fattn.fwd_cross(q, k, v, t)
    dq, dk, dv = (torch.full(x.shape, math.nan, dtype=dt, device="cuda") for x in (q, k, v))
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, dq=dq, dk=dk, dv=dv)
    ok()
    args, scale = [x.cpu() for x in (q, k, v, do)], fattn._default_scale(D)
    ref = M.cross_grads(*args, lens, scale)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, M.cross_grad_bounds(*args, lens, scale, dt, ref)):
        R.check(x, r, b, name)


@pytest.mark.parametrize("case", [(1, 8, 1, 900, 100, [70]), (1, 32, 4, 3, 4000, None), (2, 2, 1, 130, 2000, [2000, 1])])
def test_backward_cut_into_parts(case):
    """Few key blocks of many query tiles, few query tiles of many key tiles (more parts than an entry has tiles)."""
    B, H, Hkv, Nq, Nk, lens = case
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, 64, torch.bfloat16, 78, lens)
    lens = lens or [Nk] * B
    o, lse = fattn.fwd_cross(q, k, v, t)
    need = fattn.bwd_cross_workspace_bytes(B, H, Nq, Nk, 64, Hkv)
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    again = fattn.bwd_cross(q, k, v, o, lse, do, t)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    args = [x.cpu() for x in (q, k, v, do)]
    ref = M.cross_grads(*args, lens, 0.125)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, M.cross_grad_bounds(*args, lens, 0.125, torch.bfloat16, ref)):
        R.check(x, r, b, name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", [(8, 19, 19, 1403, 100, [100, 0, 1, 64, 99, 33, 17, 65]), (4, 76, 38, 700, 128, [128, 127, 0, 2]),
                                  (3, 60, 20, 450, 5, None), (8, 19, 19, 900, 300, [300, 0, 128, 129, 1, 257, 256, 100]),
                                  (4, 76, 38, 500, 200, None), (6, 30, 10, 333, 640, [640, 512, 513, 0, 385, 5])])
def test_backward_of_many_query_tiles(D, case):
    """A CTA takes a run of query tiles: over keys of one tile and of several, of entries with all, some and no keys."""
    B, H, Hkv, Nq, Nk, lens = case
    dt = torch.float16 if D == 64 else torch.bfloat16
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, D, dt, Nq + D, lens)
    lens = lens or [Nk] * B
    o, lse = fattn.fwd_cross(q, k, v, t)
    dq, dk, dv = (torch.full(x.shape, math.nan, dtype=dt, device="cuda") for x in (q, k, v))
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, dq=dq, dk=dk, dv=dv)
    again = fattn.bwd_cross(q, k, v, o, lse, do, t)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    args, scale = [x.cpu() for x in (q, k, v, do)], fattn._default_scale(D)
    ref = M.cross_grads(*args, lens, scale)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, M.cross_grad_bounds(*args, lens, scale, dt, ref)):
        R.check(x, r, b, name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", [(8, 16, 16, 85, 1500, [1500, 0, 1, 128, 129, 777, 1499, 640]), (3, 16, 8, 1, 4000, [4000, 3, 2561]),
                                  (9, 18, 9, 60, 1000, None), (1, 100, 10, 12, 2700, [2690])])
def test_backward_of_many_key_blocks(D, case):
    """Queries of one tile, whole or stacked heads: a CTA takes a run of key blocks, some behind an entry's keys."""
    B, H, Hkv, Nq, Nk, lens = case
    dt = torch.float16 if D == 64 else torch.bfloat16
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, D, dt, Nq + D, lens)
    lens = lens or [Nk] * B
    o, lse = fattn.fwd_cross(q, k, v, t)
    dq, dk, dv = (torch.full(x.shape, math.nan, dtype=dt, device="cuda") for x in (q, k, v))
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, dq=dq, dk=dk, dv=dv)
    again = fattn.bwd_cross(q, k, v, o, lse, do, t)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    args, scale = [x.cpu() for x in (q, k, v, do)], fattn._default_scale(D)
    ref = M.cross_grads(*args, lens, scale)
    for name, x, r, b in zip(("dq", "dk", "dv"), got, ref, M.cross_grad_bounds(*args, lens, scale, dt, ref)):
        R.check(x, r, b, name)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("case", [(8, 19, 19, 1000, 100), (8, 19, 19, 1000, 300), (8, 16, 16, 60, 1500)])
@pytest.mark.parametrize("fill", [math.nan, 0.0])
def test_captured_gradients(fill, D, case):
    """Runs of query tiles and of key blocks, captured and replayed over new contents and lengths, gradients of odd
    strides: the same bits (with `fill` = NaN most entries come to see keys that are NaN)."""
    B, H, Hkv, Nq, Nk = case
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, D, torch.bfloat16, Nq + Nk, [Nk - i for i in range(B)], fill)
    o, lse = fattn.fwd_cross(q, k, v, t)
    rows = torch.zeros(B, Nq, H + 1, D, dtype=torch.bfloat16, device="cuda")
    cols = torch.zeros(2, B, Nk, Hkv + 2, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(fattn.bwd_cross_workspace_bytes(B, H, Nq, Nk, D, Hkv), dtype=torch.uint8, device="cuda")
    out = dict(dq=rows[:, :, 1:].transpose(1, 2), dk=cols[0, :, :, 2:].transpose(1, 2), dv=cols[1, :, :, :Hkv].transpose(1, 2))
    fattn.bwd_cross(q, k, v, o, lse, do, t, workspace=ws, **out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.fwd_cross(q, k, v, t, out=o, lse=lse)
        fattn.bwd_cross(q, k, v, o, lse, do, t, workspace=ws, **out)
    for step in range(3):
        do.copy_(torch.roll(do, 1, 2))
        t.copy_(torch.roll(t, 1) if step else torch.tensor([0] + [Nk] * (B - 1), dtype=torch.int32))
        graph.replay()
        ws.fill_(255)
        graph.replay()
        want_o, want_lse = fattn.fwd_cross(q, k, v, t)
        want = fattn.bwd_cross(q, k, v, want_o, want_lse, do, t)
        ok()
        assert all(torch.equal(x.view(torch.int16), out[name].view(torch.int16)) for x, name in zip(want, ("dq", "dk", "dv")))
    assert (rows[:, :, 0] == 0).all() and (cols[0, :, :, :2] == 0).all() and (cols[1, :, :, Hkv:] == 0).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_backward_layouts_and_repeats(dtype, D):
    """Gradients as slices of a projection's gradient, contiguous inputs, a second run: the same bits."""
    dt = DT[dtype]
    q, k, v, do, t = make(2, 4, 2, 150, 333, D, dt, 8, [333, 200])
    o, lse = fattn.fwd_cross(q, k, v, t)
    a = fattn.bwd_cross(q, k, v, o, lse, do, t)
    grad = torch.full((2, 333, 6, D), 7.0, dtype=dt, device="cuda")
    b = fattn.bwd_cross(q.contiguous(), k.contiguous(), v.contiguous(), o.contiguous(), lse, do.contiguous(), t,
                        dk=grad[:, :, 1:3].transpose(1, 2), dv=grad[:, :, 3:5].transpose(1, 2))
    ok()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert (grad[:, :, 0] == 7).all() and (grad[:, :, 5] == 7).all()


@pytest.mark.parametrize("D", [64, 128])
def test_backward_other_groups_never_leak(D):
    """NaN in the queries and gradients of one K/V head's group reaches no other group's gradients."""
    for Nq, share in ((3, 4), (40, 3), (130, 2)):
        q, k, v, do, t = make(2, 3 * share, 3, Nq, 200, D, torch.float16, Nq, [200, 150], fill=0.0)
        o, lse = fattn.fwd_cross(q, k, v, t)
        want = fattn.bwd_cross(q, k, v, o, lse, do, t)
        q2, do2 = q.clone(), do.clone()
        q2[:, share:2 * share] = math.nan
        do2[:, share:2 * share] = math.inf
        got = fattn.bwd_cross(q2, k, v, o, lse, do2, t)
        ok()
        for x, y, per in zip(want, got, (share, 1, 1)):
            for g in (0, 2):
                assert torch.equal(x[:, g * per:(g + 1) * per], y[:, g * per:(g + 1) * per])


def test_backward_equals_the_dense_backward():
    g = torch.Generator().manual_seed(9)
    q, k, v, do = (torch.randn(2, h, 400, 64, generator=g).half().cuda() for h in (4, 2, 2, 4))
    o, lse = fattn.fwd(q, k, v)
    a = fattn.bwd(q, k, v, o, lse, do)
    b = fattn.bwd_cross(q, k, v, o, lse, do)
    ok()
    ref = M.cross_grads(*(x.cpu() for x in (q, k, v, do)), [400, 400], 0.125)
    bounds = M.cross_grad_bounds(*(x.cpu() for x in (q, k, v, do)), [400, 400], 0.125, torch.float16, ref)
    for x, y, r, e in zip(a, b, ref, bounds):
        R.check(x, r, e, "dense")
        R.check(y, r, e, "cross")


def test_captured_and_on_another_stream():
    """A training step's forward and backward in one graph, replayed on other inputs and lengths."""
    q, k, v, do, t = make(2, 4, 2, 140, 300, 64, torch.float16, 10, [300, 10], fill=0.5)
    out, lse = torch.empty_like(q), torch.empty(2, 4, 140, device="cuda")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws = torch.empty(max(16, fattn.cross_workspace_bytes(2, 4, 140, 300, 64, 2)), dtype=torch.uint8, device="cuda")
    wb = torch.empty(fattn.bwd_cross_workspace_bytes(2, 4, 140, 300, 64, 2), dtype=torch.uint8, device="cuda")

    def step():
        fattn.fwd_cross(q, k, v, t, out=out, lse=lse, workspace=ws)
        fattn.bwd_cross(q, k, v, out, lse, do, t, dq=dq, dk=dk, dv=dv, workspace=wb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed, lens in ((11, [150, 300]), (12, [0, 129])):
        q2, k2, v2, do2, _ = make(2, 4, 2, 140, 300, 64, torch.float16, seed, fill=0.5)
        for a, b in ((q, q2), (k, k2), (v, v2), (do, do2), (t, torch.tensor(lens, dtype=torch.int32))):
            a.copy_(b)
        graph.replay()
        ok()
        got = [x.clone() for x in (out, lse, dq, dk, dv)]
        o2, l2 = fattn.fwd_cross(q, k, v, t, stream=s)
        want = (o2, l2) + fattn.bwd_cross(q, k, v, o2, l2, do, t, stream=s)
        ok()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_two_streams_at_once():
    """Calls on two streams, workspaces of their own, give what they give alone."""
    sets = [make(3, 8, 2, Nq, 1500, 64, torch.float16, 60 + Nq, [1500, 700, 20], fill=0.5) for Nq in (70, 33)]
    alone = []
    for q, k, v, do, t in sets:
        o, lse = fattn.fwd_cross(q, k, v, t)
        alone.append((o, lse) + fattn.bwd_cross(q, k, v, o, lse, do, t))
    ok()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, (q, k, v, do, t) in zip(streams, sets):
            s.wait_stream(torch.cuda.current_stream())
            o, lse = fattn.fwd_cross(q, k, v, t, stream=s)
            got.append((o, lse) + fattn.bwd_cross(q, k, v, o, lse, do, t, stream=s))
        ok()
        for a, b in zip(alone, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("Nq", [1, 40])
def test_tensors_past_32_bits(Nq):
    """17 million keys (4.4 GB each of K and V): the last one outweighs all others, so
    that O is its value, its value's gradient the sum of dO, and dQ and dK vanish."""
    D, Nk = 128, 17_000_001
    g = torch.Generator().manual_seed(61)
    k, v = (torch.zeros(1, 1, Nk, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q, do = (torch.randn(1, 1, Nq, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    q[..., 0] = 64.0
    k[0, 0, -1, 0] = 16.0                     # a score of 1024 / sqrt(128) = 90.5 and more
    v[0, 0, -1] = torch.randn(D, generator=g).to(torch.bfloat16).cuda()
    v[0, 0, -2] = 1000.0                      # weighs e^-90
    o, lse = fattn.fwd_cross(q, k, v)
    dk, dv = torch.full_like(k, math.nan), torch.full_like(v, math.nan)
    dq, _, _ = fattn.bwd_cross(q, k, v, o, lse, do, dk=dk, dv=dv)
    ok()
    assert torch.equal(o, v[:, :, -1:].expand_as(o))
    want = do.double().sum(2)[0, 0]
    assert ((dv[0, 0, -1].double() - want).abs() <= 2.0 ** -8 * (want.abs() + do.double().abs().sum(2)[0, 0])).all()
    for start in range(0, Nk - 1, 1 << 22):
        part = slice(start, min(start + (1 << 22), Nk - 1))
        assert dv[0, 0, part].abs().max() <= 1e-30 and dk[0, 0, part].abs().max() <= 1e-30
    # dS of the last key is P (dP - Delta), both the sum of dO O: fp32 sums of D exact
    # products, each off by at most D 2^-23 of the sum of magnitudes
    small = 2 * D * 2.0 ** -23 * (do.double().abs() * o.double().abs()).sum(-1).max().item() * 16 * D ** -0.5
    assert dq.double().abs().max().item() <= small and dk[0, 0, -1].isfinite().all()


def test_refusals_of_the_binding():
    q, k, v, do, t = make(2, 4, 2, 5, 30, 64, torch.float16, 62)
    o, lse = fattn.fwd_cross(q, k, v, t)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:, :, :-1]), dict(v=v.bfloat16()), dict(kv_lens=t.long()),
                dict(kv_lens=t[:1]), dict(out=o[..., :32]), dict(lse=lse.double()), dict(k=k.cpu()),
                dict(q=q.transpose(2, 3)), dict(workspace=torch.empty(8))):
        args = dict(dict(q=q, k=k, v=v, kv_lens=t), **bad)
        with pytest.raises(ValueError):
            fattn.fwd_cross(**args)
    for bad in (dict(o=o.float()), dict(dout=do[:1]), dict(lse=lse[..., :-1]), dict(dq=torch.empty_like(k)),
                dict(dk=torch.empty_like(q)), dict(kv_lens=t.cpu())):
        with pytest.raises(ValueError):
            fattn.bwd_cross(**dict(dict(q=q, k=k, v=v, o=o, lse=lse, dout=do, kv_lens=t), **bad))
    for f, args in ((fattn.fwd_cross, dict(q=q, k=k, v=v, out=q)),
                    (fattn.fwd_cross, dict(q=q, k=k, v=v, scale=-1.0)),
                    (fattn.fwd_cross, dict(q=q, k=k, v=v, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))),
                    (fattn.fwd_cross, dict(q=q[:1].expand(2, -1, -1, -1), k=k, v=v)),
                    (fattn.bwd_cross, dict(q=q, k=k, v=v, o=o, lse=lse, dout=do, dq=do))):
        with pytest.raises(fattn.FattnError) as e:
            f(**args)
        assert e.value.code == 1
    ok()
