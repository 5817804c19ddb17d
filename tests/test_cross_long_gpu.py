"""Cross attention in fp16 over keys so many that a weight is a subnormal number of the
type: against 64-bit forms, with bounds relative to the weights and to the gradients."""
import math

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -11  # half a step of fp16, relative


def ok():
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 0


def pieces(B, Hkv, share, Nq, rows_at_once):
    """(b, K/V head, query rows of all heads that share it): so many rows that 64-bit scores fit."""
    for b in range(B):
        for g in range(Hkv):
            for i in range(0, share * Nq, rows_at_once):
                yield b, g, slice(i, min(i + rows_at_once, share * Nq))


def check(got, ref, bound, what):
    over = ((got.double() - ref).abs() / bound).max().item()
    assert got.isfinite().all() and over <= 1, "%s: %.3g of the bound" % (what, over)


def check_gradients(q, k, v, do, lens, scale, got, what):
    """From the kernels' arithmetic.  P, of up to 1, is held 2^14 times its size in fp16:
    off by U of itself, and by half a subnormal step, 2^-25, of what is held.  dS is held
    2^E times its size, where 2^E times B = 2 max|dO_i| max|v_j| (2-norms over the K/V
    head's rows and seen keys, of which |dP - Delta| is at most that) lies above 2^14: off
    by U and by 2^-25 2^-E < 2^-39 B; dP is an fp32 sum of D products.  Delta = dO . O by the forward's error of O: its
    weights' rounding U (and `eps`) of sum p |v|, O's own
    rounding.  exp2, the LSE and the fp32 sums: `eps` of P, and twice (in s and in the LSE)
    (D + 1) 2^-23 of the largest sum of |q k|, as in serving_ref.  Results are rounded once."""
    B, H, Nq, D = q.shape
    Hkv = k.shape[1]
    share = H // Hkv
    sums = 1e-4 + (max(Nq * share, k.shape[2]) / 16.0 + 8.0) * 2.0 ** -24
    ref = [torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (q, k, v)]
    bound = [torch.zeros_like(x) for x in ref]
    qd, dod = (x.double().reshape(B, Hkv, share * Nq, D) for x in (q, do))
    rq, rb = (x.view(B, Hkv, share * Nq, D) for x in (ref[0], bound[0]))
    for b, g, rows in pieces(B, Hkv, share, Nq, max(1, (1 << 27) // max(k.shape[2], 1))):
        n = lens[b]
        if n == 0:
            continue
        kk, vv, qq, dd = k[b, g, :n].double(), v[b, g, :n].double(), qd[b, g, rows], dod[b, g, rows]
        eps = sums + 2 * (D + 1) * 2.0 ** -23 * scale * (qq.abs() @ kk.abs().T).max()
        p = torch.softmax(scale * qq @ kk.T, 1)
        dp = dd @ vv.T
        delta = (p * dp).sum(1, keepdim=True)
        o, av = p @ vv, p @ vv.abs()
        ddelta = (dd.abs() * ((U + eps) * av + 2 * U * o.abs() + 2.0 ** -25)).sum(1, keepdim=True)
        most = 2 * dod[b, g].norm(dim=1).max() * vv.norm(dim=1).max()
        ds = p * (dp - delta)
        ddp = D * 2.0 ** -23 * (dd.abs() @ vv.abs().T)
        w = (1.05 * U + eps) * ds.abs() + p * (ddelta + ddp + eps * (dp.abs() + delta.abs())) + 2.0 ** -39 * most
        rq[b, g, rows] = scale * ds @ kk
        rb[b, g, rows] = scale * w @ kk.abs()
        ref[1][b, g, :n] += scale * ds.T @ qq
        bound[1][b, g, :n] += scale * w.T @ qq.abs()
        ref[2][b, g, :n] += p.T @ dd
        bound[2][b, g, :n] += ((1.05 * U + eps) * p + 2.0 ** -39).T @ dd.abs()
        del p, dp, ddp, ds, w
    for name, x, r, e in zip(("dq", "dk", "dv"), got, ref, bound):
        check(x, r, e + U * (r.abs() + e) + 2.0 ** -25, "%s, %s" % (what, name))
    for b, n in enumerate(lens):
        assert (got[1][b, :, n:] == 0).all() and (got[2][b, :, n:] == 0).all()


def make(B, H, Hkv, Nq, Nk, D, lens, seed, q_std=0.02, k_std=1.0, v_std=1.0, do_std=1.0):
    """Rows and keys of a projection each; NaN behind an entry's keys."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    q, do = ((rand(B, Nq, H, D) * s).half().transpose(1, 2) for s in (q_std, do_std))
    kv = torch.empty(B, Nk, 2 * Hkv, D, dtype=torch.float16, device="cuda")
    for b in range(B):
        kv[b, :, :Hkv] = (rand(Nk, Hkv, D) * k_std).half()
        kv[b, :, Hkv:] = (rand(Nk, Hkv, D) * v_std).half()
        kv[b, lens[b]:] = math.nan
    t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    return q, kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2), do, t


# (B, H, Hkv, Nq, Nk, D, lens): one tile of query rows (runs of key blocks, dQ cut into parts), several tiles,
# runs of query tiles, key blocks in parts; an entry with few of its many keys, and with none.
LONG = [(1, 2, 1, 20, 120000, 64, [119999]), (2, 4, 2, 9, 100000, 128, [100000, 70001]), (1, 1, 1, 300, 100000, 64, [100000]),
        (1, 2, 2, 20000, 17000, 64, [16999]), (1, 2, 2, 20000, 17000, 128, [17000]), (1, 1, 1, 900, 17000, 128, [16500]),
        (3, 2, 2, 40, 60000, 64, [60000, 0, 77]), (1, 1, 1, 8, 1000003, 64, [1000003]), (1, 1, 1, 40, 4000000, 64, [4000000])]


@pytest.mark.parametrize("do_std", [1.0, 2.0 ** -7])
@pytest.mark.parametrize("case", LONG)
def test_gradients_of_small_weights(case, do_std):
    """Near-uniform weights: each is about 1 / Nk.  Gradients of a sum, and as small as a mean's."""
    B, H, Hkv, Nq, Nk, D, lens = case
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, D, lens, Nk + Nq, do_std=do_std)
    o, lse = fattn.fwd_cross(q, k, v, t)
    dq, dk, dv = (torch.full(x.shape, math.nan, dtype=x.dtype, device="cuda") for x in (q, k, v))
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, dq=dq, dk=dk, dv=dv)
    again = fattn.bwd_cross(q, k, v, o, lse, do, t)
    ok()
    assert all(torch.equal(x, y) for x, y in zip(got, again))
    check_gradients(q, k, v, do, lens, fattn._default_scale(D), got, str(case))


@pytest.mark.parametrize("case", [(1, 2, 1, 20, 20000, 64, [20000]), (1, 1, 1, 300, 20000, 128, [19999]),
                                  (1, 2, 2, 20000, 17000, 64, [17000]), (2, 1, 1, 900, 17000, 64, [17000, 3])])
def test_large_gradients(case):
    """A few keys have the weight of a row, and P (dP - Delta) is past fp16's range, the gradients are not."""
    B, H, Hkv, Nq, Nk, D, lens = case
    q, k, v, do, t = make(B, H, Hkv, Nq, Nk, D, lens, Nk + Nq, q_std=32.0, k_std=32.0, v_std=30.0, do_std=600.0 / math.sqrt(Nq))
    scale = 2.0 ** -10
    do[:, :, 0] *= math.sqrt(Nq)
    o, lse = fattn.fwd_cross(q, k, v, t, scale=scale)
    got = fattn.bwd_cross(q, k, v, o, lse, do, t, scale=scale)
    ok()
    check_gradients(q, k, v, do, lens, scale, got, str(case))


def test_an_entry_does_not_depend_on_the_others():
    """Nor on another K/V head's group: its gradients have the bits that they have alone."""
    q, k, v, do, t = make(3, 4, 2, 40, 40000, 64, [40000, 30000, 12], 5)
    o, lse = fattn.fwd_cross(q, k, v, t)
    want = fattn.bwd_cross(q, k, v, o, lse, do, t)
    q2, do2, v2 = q.clone(), do.clone(), v.clone()
    do2[0] *= 500.0
    do2[1, 2:] = math.inf
    v2[2] *= 100.0
    got = fattn.bwd_cross(q2, k, v2, o, lse, do2, t)
    ok()
    for x, y, per in zip(want, got, (2, 1, 1)):
        assert torch.equal(x[1, :per], y[1, :per])


def test_captured_over_other_contents():
    """Captured with a workspace that anything may lie in: eager's bits for each replay's inputs and lengths."""
    q, k, v, do, t = make(2, 2, 2, 150, 30000, 64, [30000, 30000], 6)
    o, lse = fattn.fwd_cross(q, k, v, t)
    ws = torch.full((fattn.bwd_cross_workspace_bytes(2, 2, 150, 30000, 64, 2),), 255, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(x) for x in (q, k, v)]
    names = ("dq", "dk", "dv")
    fattn.bwd_cross(q, k, v, o, lse, do, t, workspace=ws, **dict(zip(names, out)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fattn.bwd_cross(q, k, v, o, lse, do, t, workspace=ws, **dict(zip(names, out)))
    for factor, lens in ((64.0, [30000, 5]), (1 / 4096, [17, 29999]), (1.0, [30000, 0])):
        do.mul_(factor)
        t.copy_(torch.tensor(lens, dtype=torch.int32))
        fattn.fwd_cross(q, k, v, t, out=o, lse=lse)
        ws.fill_(255)
        graph.replay()
        graph.replay()
        want = fattn.bwd_cross(q, k, v, o, lse, do, t)
        ok()
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def weight_error(s, D, n):
    """P's one rounding, exponentials, scores (as in serving_ref), and the sum of n values
    near 1: n / 16 products add to an fp32 accumulator, each with an error of up to 2^-23 of
    what it holds then (the tensor cores cut), which grows evenly from 0 to the sum."""
    return U + 2.0 ** -20 + 2 * (D + 1) * 2.0 ** -23 * s + n / 16 * 2.0 ** -23 / 2


@pytest.mark.parametrize("D", [64, 128])
def test_forward_of_many_keys_beside_one(D):
    """One key outweighs each of 120000 others 2^14 to 2^18 times, which together weigh about as
    much: the weights of the others keep their bits (rows enough that keys are not cut)."""
    H, Nq, Nk = 2, 20000, 120001
    g = torch.Generator(device="cuda").manual_seed(7)
    k = torch.zeros(1, H, Nk, D, dtype=torch.float16, device="cuda")
    v = (1.0 + 0.1 * torch.randn(1, H, Nk, D, generator=g, device="cuda")).half()
    q = torch.zeros(1, H, Nq, D, dtype=torch.float16, device="cuda")
    k[:, :, 5, 0] = 1.0
    v[:, :, 5] = 0.0
    q[..., 0] = (9.7 + 2.8 * torch.rand(1, H, Nq, generator=g, device="cuda")).half()
    o, lse = fattn.fwd_cross(q, k, v, scale=1.0)
    ok()
    rows = torch.arange(0, Nq, 7, device="cuda")
    s = q[0, :, rows, 0].double()
    total = s.exp() + (Nk - 1)
    ref = v[0].double().sum(1)[:, None] / total[..., None]
    core = weight_error(s, D, Nk)[..., None] * ref.abs()
    check(o[0, :, rows], ref, core + U * (ref.abs() + core), "O")
    # (scores as in serving_ref; Nk / 128 tiles' sums are added one by one, each off by up to 2^-24 of a sum that grows evenly)
    bound = (D + 1) * 2.0 ** -23 * s + 2.0 ** -20 * (1 + total.log()) + Nk / 128 * 2.0 ** -24 / 2
    assert ((lse[0, :, rows].double() - total.log()).abs() <= bound).all()


def test_decode_behind_a_long_prefix_keeps_small_weights():
    """The same for a chunk of tokens behind a shared prefix, whose own keys weigh nothing."""
    H, Nq, D, page, P = 64, 650, 64, 64, 120000
    g = torch.Generator(device="cuda").manual_seed(8)
    pages = P // page
    kp = torch.zeros(pages + 11, 1, page, D, dtype=torch.float16, device="cuda")
    vp = (1.0 + 0.1 * torch.randn(pages + 11, 1, page, D, generator=g, device="cuda")).half()
    kp[0, 0, 5, 0], vp[0, 0, 5] = 1.0, 0.0
    kp[pages:, ..., 0] = -30.0
    q = torch.zeros(1, H, Nq, D, dtype=torch.float16, device="cuda")
    q[..., 0] = (9.7 + 2.8 * torch.rand(1, H, Nq, generator=g, device="cuda")).half()
    i32 = dict(dtype=torch.int32, device="cuda")
    o, lse = fattn.decode_shared(q, kp, vp, torch.arange(pages, **i32), torch.tensor([P], **i32),
                                 torch.arange(pages, pages + 11, **i32)[None], torch.tensor([Nq], **i32), scale=1.0)
    ok()
    s = q[0, :, :, 0].double()
    total = s.exp() + (P - 1)  # (an own key weighs e^-291 at most)
    ref = vp[:pages, 0].double().sum((0, 1)) / total[..., None]
    core = weight_error(s, D, P)[..., None] * ref.abs()
    check(o[0], ref, core + U * (ref.abs() + core), "O")
