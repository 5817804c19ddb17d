"""Attention of packed sequences (fwd_packed) against a plain 64-bit form, and
the serving operators run together as a model's steps use them."""
import math

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
INVALID = 1


def ok():
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 0


def make(lens, H, Hkv, D, dt, seed, gaps=(0, 0), q_std=1.0, fill=math.nan):
    """q, k, v as slices of one projection; rows of no sequence hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    T = sum(lens) + sum(gaps)
    x = torch.randn(T, H + 2 * Hkv, D, generator=g)
    x[:, :H] *= q_std
    x[:gaps[0]] = fill
    x[T - gaps[1]:] = fill
    x = x.to(dt).cuda()
    cu = [gaps[0]]
    for n in lens:
        cu.append(cu[-1] + n)
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], torch.tensor(cu, dtype=torch.int32).cuda()


def check_packed(q, k, v, cu, causal, scale, o, lse, what="", rows=None):
    """Every row (or `rows` random rows of each sequence) against the 64-bit form.

    P is at most 2^8 while the running max is stale; it is rounded once, and for
    bf16 the normaliser is the sum of the rounded P, for which |sum of p v's
    roundings| + |O| |sum of p's roundings| bounds the numerator and the
    normaliser together: twice u_of(dtype) of sum p|v| covers both types."""
    T, H, D = q.shape
    dt = q.dtype
    at = cu.tolist()
    g = torch.Generator().manual_seed(1)
    for a, b in zip(at[:-1], at[1:]):
        n = b - a
        if n == 0:
            continue
        pick = torch.arange(n) if rows is None or n <= rows else torch.cat(
            [torch.randperm(n, generator=g)[:rows], torch.tensor([0, 1, n - 2, n - 1])])
        qs = q[a:b].cpu().double().transpose(0, 1)[:, pick]
        ks, vs = (t[a:b].cpu().double().transpose(0, 1) for t in (k, v))
        ends = (pick + 1).tolist() if causal else [n] * len(pick)
        ro, rl, av, worst = R.attend(qs, ks, vs, scale, ends)
        bo, bl = R.attend_bounds(ro, rl, av, worst, D, dt, 2 * R.u_of(dt))
        w = "%s sequence of %d" % (what, n)
        R.check(o[a:b].cpu().transpose(0, 1)[:, pick], ro, bo, w + " O")
        R.check(lse[:, a:b].cpu()[:, pick], rl, bl, w + " LSE")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D,H,Hkv,lens", [
    ("bf16", 128, 4, 2, [1, 127, 128, 129, 0, 255, 256, 257, 300]),
    ("fp16", 64, 4, 1, [300, 1, 0, 0, 513, 64, 128, 65]),
    ("bf16", 64, 3, 3, [5]), ("fp16", 128, 8, 1, [2, 3, 700]), ("bf16", 128, 1, 1, [0, 1])])
def test_packed(dtype, D, H, Hkv, lens, causal):
    """NaN lies in every row of no sequence, and those rows of out and lse are left as they were."""
    q, k, v, cu = make(lens, H, Hkv, D, DT[dtype], D + H, gaps=(3, 130))
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((H, q.shape[0]), 7.0, device="cuda")
    o, l = fattn.fwd_packed(q, k, v, cu, causal=causal, out=out, lse=lse)
    ok()
    assert o is out and l is lse
    check_packed(q, k, v, cu, causal, fattn._default_scale(D), o, lse)
    a, b = cu[0].item(), cu[-1].item()
    assert (out[:a] == 7).all() and (out[b:] == 7).all() and (lse[:, :a] == 7).all() and (lse[:, b:] == 7).all()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp16", 128), ("bf16", 64)])
def test_packed_equals_the_dense_forward(dtype, D, causal):
    """One sequence of all tokens, head-major and token-major: the bits of fwd."""
    N, H, Hkv = 777, 6, 2
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(1, h, N, D, generator=g).to(DT[dtype]).cuda() for h in (H, Hkv, Hkv))
    o, lse = fattn.fwd(q, k, v, causal=causal)
    cu = torch.tensor([0, N], dtype=torch.int32).cuda()
    for major in ("head", "token"):
        p = [t[0].transpose(0, 1) for t in (q, k, v)]
        if major == "token":
            p = [t.contiguous() for t in p]
        out = torch.empty_like(q)[0].transpose(0, 1) if major == "head" else None
        o2, lse2 = fattn.fwd_packed(*p, cu, causal=causal, out=out)
        ok()
        assert torch.equal(o2.transpose(0, 1), o[0]) and torch.equal(lse2, lse[0])


@pytest.mark.parametrize("causal", [True, False])
def test_packed_many_sequences(causal):
    """More sequences than a CTA has threads, most of them empty or tiny, one long."""
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 9, (1500,), generator=g).tolist()
    lens[700] = 4099
    q, k, v, cu = make(lens, 2, 1, 64, torch.bfloat16, 5)
    o, lse = fattn.fwd_packed(q, k, v, cu, causal=causal)
    ok()
    check_packed(q, k, v, cu, causal, 0.125, o, lse, rows=200)


def test_packed_another_sequence_never_leaks():
    """NaN and infinities in one sequence reach none of the others, whatever shares its tiles."""
    lens = [100, 60, 200, 129]
    for D, dt in ((128, torch.bfloat16), (64, torch.float16)):
        q, k, v, cu = make(lens, 2, 2, D, dt, 6)
        at = cu.tolist()
        for causal in (True, False):
            o, lse = fattn.fwd_packed(q, k, v, cu, causal=causal)
            for b in range(len(lens)):
                for bad in (math.nan, math.inf):
                    kk, vv = k.clone(), v.clone()
                    kk[at[b]:at[b + 1]] = bad
                    vv[at[b]:at[b + 1]] = -bad
                    o2, lse2 = fattn.fwd_packed(q, kk, vv, cu, causal=causal)
                    ok()
                    keep = torch.ones(sum(lens), dtype=torch.bool)
                    keep[at[b]:at[b + 1]] = False
                    keep = keep.cuda()
                    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[:, keep], lse[:, keep])


@pytest.mark.parametrize("cu", [[-1, 5], [0, 6, 5, 8], [0, 9], [3, 2], [0, 4, 2 ** 31 - 1]])
def test_packed_bad_table_does_nothing_and_is_reported(cu):
    q, k, v, _ = make([8], 2, 1, 64, torch.float16, 7)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((2, 8), 7.0, device="cuda")
    fattn.fwd_packed(q, k, v, torch.tensor(cu, dtype=torch.int32).cuda(), out=out, lse=lse)
    torch.cuda.synchronize()
    assert fattn.get_device_status() == INVALID and fattn.get_device_status() == 0
    assert (out == 7).all() and (lse == 7).all()


def test_packed_empty():
    q, k, v, _ = make([8], 2, 1, 64, torch.float16, 8)
    zero = torch.zeros(1, dtype=torch.int32).cuda()
    o, lse = fattn.fwd_packed(q, k, v, zero)                       # no sequence
    o2, _ = fattn.fwd_packed(q, k, v, torch.zeros(4, dtype=torch.int32).cuda())  # three empty ones
    o3, _ = fattn.fwd_packed(q[:0], k[:0], v[:0], zero)            # no token
    ok()
    assert (o == 0).all() and (o2 == 0).all() and (lse == 0).all() and o3.shape[0] == 0
    o4, none = fattn.fwd_packed(q, k, v, torch.tensor([0, 8], dtype=torch.int32).cuda(), return_lse=False)
    ok()
    assert none is None and torch.isfinite(o4).all()


def test_packed_streams_and_graphs():
    """Two graphs with a workspace each, replayed at once with lengths that change between replays."""
    H, Hkv, D, T = 4, 2, 128, 900
    q, k, v, cu = make([T], H, Hkv, D, torch.bfloat16, 9)
    cu = torch.tensor([0, 100, 500, 500, T], dtype=torch.int32).cuda()
    out0, lse0 = fattn.fwd_packed(q, k, v, cu)
    ok()
    graphs, outs, keep = [], [], []
    for _ in range(2):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        oo, ll = torch.zeros_like(out0), torch.zeros_like(lse0)
        ws = torch.empty(fattn.packed_workspace_bytes(4, T), dtype=torch.uint8, device="cuda")
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                fattn.fwd_packed(q, k, v, cu, out=oo, lse=ll, workspace=ws, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        graphs.append((g, s))
        outs.append((oo, ll))
        keep.append(ws)
    for table in ([0, 100, 500, 500, T], [0, 1, 2, 3, T], [0, 300, 600, 600, 640]):
        cu.copy_(torch.tensor(table, dtype=torch.int32))
        for oo, ll in outs:
            oo.zero_()
            ll.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        ok()
        want, want_l = fattn.fwd_packed(q, k, v, cu)
        ok()
        for oo, ll in outs:
            assert torch.equal(oo, want) and torch.equal(ll, want_l)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype,D,H,Hkv", [("bf16", 128, 8, 2), ("fp16", 64, 4, 4)])
def test_prompts_then_steps(dtype, D, H, Hkv, kv4):
    """As a server runs them: the prompts' tokens are rotated and appended and
    attend to themselves, then three steps append one token a sequence and
    attend to the cache.  Every step is compared with attention over all rows
    so far as the cache holds them, in 64 bits, with q as the append rotated it."""
    dt, ps, steps = DT[dtype], 16, 3
    lens = [37, 1, 130, 16]
    B, T = len(lens), sum(lens)
    scale = fattn._default_scale(D)
    width = max(-(-(n + steps) // ps) for n in lens)
    P = B * width
    g = torch.Generator().manual_seed(10)
    table = torch.randperm(P, generator=g).to(torch.int32).view(B, width)
    cos, sin = (t.cuda() for t in R.tables(256, D))
    if kv4:
        cache = []
        for _ in range(2):
            cache += [torch.zeros(P, Hkv, ps, D // 2, dtype=torch.uint8, device="cuda"),
                      torch.full((P, Hkv, ps, D // 32, 2), math.nan, dtype=torch.float16, device="cuda")]
        app, att = fattn.cache_append_kv4, fattn.decode_kv4
    else:
        cache = [torch.full((P, Hkv, ps, D), math.nan, dtype=dt, device="cuda") for _ in range(2)]
        app, att = fattn.cache_append, fattn.decode

    def slots_of(b, j):
        return table[b].long()[j // ps] * ps + j % ps

    q, k, v, cu = make(lens, H, Hkv, D, dt, 11)
    j = [torch.arange(n) for n in lens]
    slots = torch.cat([slots_of(b, x) for b, x in enumerate(j)]).cuda()
    pos = torch.cat(j).to(torch.int32).cuda()
    held = {}
    if kv4:
        held = dict(v_out=torch.empty(T, Hkv, D, dtype=dt, device="cuda"), held=True)
    k_out = torch.empty(T, Hkv, D, dtype=dt, device="cuda")
    res = app(k, v, *cache, slots, pos=pos, cos=cos, sin=sin, q=q, k_out=k_out, **held)
    kk, vv = (res[1], res[2]) if kv4 else (res[1], v)
    o, lse = fattn.fwd_packed(res[0], kk, vv, cu)
    ok()
    check_packed(res[0], kk, vv, cu, True, scale, o, lse, "prompt")
    from tests.test_cache_gpu import check_decode
    for step in range(steps):
        q1, k1, v1, _ = make([B], H, Hkv, D, dt, 20 + step)
        now = torch.tensor(lens) + step
        slots = torch.stack([slots_of(b, now[b]) for b in range(B)]).cuda()
        qr = app(k1, v1, *cache, slots, pos=now.to(torch.int32).cuda(), cos=cos, sin=sin, q=q1)[0]
        seq = (now + 1).to(torch.int32).cuda()
        qd = qr.unsqueeze(2)
        o, lse = att(qd, *cache, table.cuda(), seq)
        ok()
        check_decode(kv4, qd, cache, table, seq, scale, o, lse, "step %d" % step)


def test_results_allocated_on_the_call_s_stream():
    """Without out, lse and workspace a call on another stream allocates them
    there: nothing enqueued on the current stream touches them meanwhile."""
    H, Hkv, D = 4, 2, 64
    q, k, v, cu = make([300, 5], H, Hkv, D, torch.float16, 12)
    want, want_l = fattn.fwd_packed(q, k, v, cu)
    pages = torch.zeros(20, Hkv, 16, D, dtype=torch.float16, device="cuda")
    vpages = torch.zeros_like(pages)
    slots = torch.arange(305).cuda()
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None]
    n = torch.tensor([305], dtype=torch.int32).cuda()
    fattn.cache_append(k, v, pages, vpages, slots)
    qd = q[-1:].unsqueeze(2)
    dec, dec_l = fattn.decode(qd, pages, vpages, table, n)
    ok()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    big = torch.empty(1 << 26, device="cuda")
    for _ in range(20):
        big.normal_()  # keeps the current stream busy, and its freed blocks in use
        junk = torch.full_like(want, 9.0)
        del junk
        o, l = fattn.fwd_packed(q, k, v, cu, stream=s)
        o2, l2 = fattn.decode(qd, pages, vpages, table, n, stream=s)
        s.synchronize()
        with torch.cuda.stream(s):
            assert torch.equal(o, want) and torch.equal(l, want_l)
            assert torch.equal(o2, dec) and torch.equal(l2, dec_l)
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 0
