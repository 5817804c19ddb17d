"""The serving operators at the edges of what their contracts allow, against plain
64-bit forms (tests/serving_ref.py)."""
import math

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import serving_ref as R
from tests.test_cache_gpu import append, check_decode, make_decode, new_cache, run_decode
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


def rows_at_the_ends(T, Hkv, D, dt, seed):
    """Rows whose groups of 32 reach the ends of fp16's range, in several ways."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, Hkv, D // 32, 32, generator=g) * 10.0 ** torch.randint(0, 4, (T, Hkv, D // 32, 1), generator=g)
    big = 1e5 if dt == torch.bfloat16 else 65504.0
    kinds = [(0.0, big), (-big, big), (0.0, math.inf), (-math.inf, math.inf), (None, 65504.0), (None, math.inf),
             (-60000.0, 65504.0), (60000.0, big), (-math.inf, None), (None, None)]
    pick = torch.randint(0, len(kinds), (T, Hkv, D // 32), generator=g)
    for i, (lo, hi) in enumerate(kinds):
        m = pick == i
        sub = x[m]
        if lo is not None and hi is not None:
            a, b = max(lo, -65504.0), min(hi, 65504.0)
            sub = a + (b - a) * torch.rand(sub.shape, generator=g)
        if lo is not None:
            sub[:, 3] = lo
        if hi is not None:
            sub[:, 7] = hi
        x[m] = sub
    return x.flatten(-2).to(dt)


@pytest.mark.parametrize("held", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp16", 128), ("bf16", 64)])
def test_kv4_values_at_the_ends_of_the_range_stay_finite(dtype, D, held):
    """What the append holds for elements at and past +-65504 may lie a little
    past it (the scale is rounded, to nearest): outputs in 16 bits and the
    attention over such rows are finite all the same, and right."""
    dt, T, Hkv, H, ps = DT[dtype], 160, 2, 8, 16
    v = rows_at_the_ends(T, Hkv, D, dt, D)
    k = rows_at_the_ends(T, Hkv, D, dt, D + 1)
    cache = new_cache(True, T // ps, Hkv, ps, D, dt, 0.0)
    k_out, v_out = (torch.empty(T, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
    fattn.cache_append_kv4(k.cuda(), v.cuda(), *cache, torch.arange(T).cuda(), k_out=k_out, v_out=v_out, held=held)
    ok()
    past = 0
    for which, x, out, c, s in (("k", k, k_out, *cache[:2]), ("v", v, v_out, *cache[2:])):
        c, s = (t.cpu().transpose(1, 2).flatten(0, 1) for t in (c, s))  # [T, Hkv, ..]
        assert torch.isfinite(s).all()
        if not held:
            assert torch.equal(out.cpu(), x)
            continue
        val = R.held(c, s, which)
        past += (val > 65519.0).sum().item()
        size = val.abs() + 16 * s[..., 0].double().repeat_interleave(32, -1)
        if dt == torch.float16:
            val = val.clamp(-65504, 65504)  # the nearest that fp16 has
        R.check(out, val, R.u_of(dt) * (1 + 2.0 ** -10) * val.abs() + 2.0 ** -23 * size + R.tiny(dt), which)
    assert past > 20 or not held
    # attention: keys of ordinary size first, then the extreme ones (weights decided by few keys: scores of some 100)
    g = torch.Generator().manual_seed(3)
    table = torch.arange(T // ps, dtype=torch.int32)[None].repeat(5, 1).cuda()
    lens = torch.tensor([T, 1, 17, 33, T - 5], dtype=torch.int32).cuda()
    for kk, scale in ((torch.randn(T, Hkv, D, generator=g).to(dt), 0.2), (k, 2.0 ** -17)):
        fattn.cache_append_kv4(kk.cuda(), v.cuda(), *cache, torch.arange(T).cuda())
        for Nq in (1, 3, 8):
            q = torch.randn(5, H, Nq, D, generator=g).to(dt).cuda()
            o, lse = fattn.decode_kv4(q, *cache, table, lens, scale=scale)
            ok()
            check_saturated(q, cache, table, lens, scale, o, lse)


def check_saturated(q, cache, table, lens, scale, o, lse):
    """check_decode's bounds, with outputs in fp16 cut to +-65504."""
    B, H, Nq, D = q.shape
    cache, table = [t.cpu() for t in cache], table.cpu()
    for b, n in enumerate(lens.tolist()):
        ends = [max(0, n - Nq + 1 + i) for i in range(Nq)]
        rows = [R.gather(t, table[b], n) for t in cache]
        k, v = R.held(rows[0], rows[1], "k"), R.held(rows[2], rows[3], "v")
        off = (rows[3][..., 1].double().abs() + 16 * rows[3][..., 0].double()).repeat_interleave(32, -1)
        ro, rl, av, worst = R.attend(q[b].cpu().double(), k, v, scale, ends)
        _, _, v_err, _ = R.attend(q[b].cpu().double(), k, 2.0 ** -11 * (v.abs() + off), scale, ends)
        bo, bl = R.attend_bounds(ro, rl, av, worst, D, q.dtype, 2.0 ** -11, v_err)
        if q.dtype == torch.float16:
            ro = ro.clamp(-65504, 65504)
        seen = torch.tensor([e > 0 for e in ends])
        R.check(o[b].cpu()[:, seen], ro[:, seen], bo[:, seen], "O of %d" % n)
        R.check(lse[b].cpu()[:, seen], rl[:, seen], bl[:, seen], "LSE of %d" % n)


def exact_codes(x, scales):
    """Codes of x (float64, exact) against the stored scales and zeros, from the definition."""
    s, z = (scales[..., i].double().repeat_interleave(32, -1) for i in range(2))
    q = torch.where(s > 0, (x - z) / torch.where(s > 0, s, 1.0), 0.0)
    return q.clamp(0, 15).round(), ((q - q.floor() - 0.5).abs() < 1e-5) & (q - q.floor() != 0.5)


@pytest.mark.parametrize("rot", [0, 16])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("fp16", 128), ("bf16", 64)])
def test_append_kv4_codes_where_differences_are_not_exact(dtype, D, rot):
    """Elements beside a zero of quite another size: x - zero takes more than 24
    bits and lies next to a border of two codes.  Every code of a row that does
    not turn is the exact quotient's rounding."""
    dt, T, ps = DT[dtype], 320, 16
    g = torch.Generator().manual_seed(D + rot)
    e = 2.0 ** -torch.randint(17, 25, (T, 1, D // 32, 1), generator=g).double()       # tiny, exact in both types
    step = 2.0 ** torch.randint(-2, 3, (T, 1, D // 32, 1), generator=g).double()
    k = torch.randint(0, 15, (T, 1, D // 32, 32), generator=g).double()
    # even tokens: a tiny zero under multiples of half steps; odd ones: a zero of -13/2 steps under tiny elements
    low = torch.where(torch.randint(0, 2, e.shape, generator=g) > 0, e, -e)
    x = (k + 0.5) * step
    x[..., 0], x[..., 1] = low[..., 0], 15 * step[..., 0]
    y = torch.where(torch.randint(0, 2, k.shape, generator=g) > 0, e, -e) * torch.randint(1, 4, k.shape, generator=g)
    y[..., 0], y[..., 1] = -6.5 * step[..., 0], 8.5 * step[..., 0]
    x[1::2] = y[1::2]
    x = x.flatten(-2).to(dt)
    cache = new_cache(True, T // ps, 1, ps, D, dt, 0.0)
    kw = {}
    if rot:
        cos, sin = (t.cuda() for t in R.tables(64, rot))
        kw = dict(pos=torch.zeros(T, dtype=torch.int32).cuda(), cos=cos, sin=sin)  # position 0: the turn changes nothing
    fattn.cache_append_kv4(x.cuda(), x.cuda(), *cache, torch.arange(T).cuda(), **kw)
    ok()
    near = 0
    for which, codes, scales in (("k", *cache[:2]), ("v", *cache[2:])):
        codes, scales = (t.cpu().transpose(1, 2).flatten(0, 1) for t in (codes, scales))
        want, close = exact_codes(x.double(), scales)
        near += close.sum().item()
        assert torch.equal(R.unpack(codes, which).double(), want), which
    assert near > 1000


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_kv4_pairs_far_past_the_range(interleaved):
    """Pairs of some 10^7 that turn until one of them lies within +-65504: its
    fp32 error is that of the pair's size, hundreds of times the range's own.
    Codes, scales and zeros are those of the rotation in 64 bits."""
    T, D, ps = 4000, 64, 16
    g = torch.Generator().manual_seed(31)
    cos, sin = R.tables(4096, D)
    pos = torch.randint(1, 4096, (T,), generator=g, dtype=torch.int32)
    c, s = cos.double()[pos.long()], sin.double()[pos.long()]
    b = (1 + torch.rand(T, D // 2, generator=g).double()) * 2.0 ** 24 * c     # along (sin, cos): turns to (0, 1)
    a = b * s / c
    k = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    k = k[:, None].to(torch.bfloat16)
    cache = new_cache(True, T // ps, 1, ps, D, torch.bfloat16, 0.0)
    fattn.cache_append_kv4(k.cuda(), k.cuda(), *cache, torch.arange(T).cuda(), pos=pos.cuda(), cos=cos.cuda(),
                           sin=sin.cuda(), interleaved=interleaved)
    ok()
    x = R.rotate(k, pos, cos, sin, interleaved)[0].clamp(-65504, 65504).unflatten(-1, (-1, 32))
    assert (x.abs() < 60000).sum() > T * D // 8
    lo, hi = x.amin(-1), x.amax(-1)
    scale, zero = ((hi - lo) / 15).float().half().double(), lo.float().half().double()
    got = cache[1].cpu().double().transpose(1, 2).reshape(T, 1, D // 32, 2)
    assert torch.equal(got[..., 0], scale) and torch.equal(got[..., 1], zero)
    q = (x - zero[..., None]) / torch.where(scale > 0, scale, 1.0)[..., None]
    want = torch.where(scale[..., None] > 0, q, 0.0).clamp(0, 15).round().flatten(-2)
    codes = R.unpack(cache[0].cpu().transpose(1, 2).reshape(T, 1, D // 2), "k").double()
    assert torch.equal(codes, want)


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_rows_without_keys_beside_values_that_are_not_finite(kv4):
    """More new tokens than the sequence has: the rows before its first key are O
    = 0, LSE = -inf, whatever its values hold; alone, joined and cut between CTAs."""
    B, H, Hkv, Nq, D, ps = 700, 4, 2, 6, 64, 16
    for lens in ([2], [3] * B, [4, 9000, 1]):  # few keys; a warp each; beside a sequence that is cut
        q, cache, table, seq = make_decode(kv4, lens, H, Hkv, Nq, D, ps, "fp16", 40)
        for t in cache[2:] if kv4 else cache[1:]:
            if t.dtype == torch.float16:
                t.fill_(math.nan)
        o, lse = run_decode(kv4, q, cache, table, seq)
        ok()
        for b, n in enumerate(lens[:40]):
            empty = max(0, Nq - n)
            assert (o[b, :, :empty] == 0).all() and (lse[b, :, :empty] == -math.inf).all()
            assert torch.isnan(o[b, :, empty:]).all() and torch.isfinite(lse[b, :, empty:]).all()


@pytest.mark.parametrize("kv4", [False, True])
def test_captured_steps_read_what_they_append(kv4):
    """A graph of several steps, each an append followed at once by the attention
    over it, and a prompt's append followed by the packed attention of its rows:
    the kernels of a replay start while the one before them ends.  Two graphs
    with caches of their own replay at once; tokens, slots, positions and lengths
    change between replays.  Results and caches are those of calls that wait."""
    B, H, Hkv, D, ps, width, steps, T = 3, 8, 2, 128, 16, 8, 4, 200
    dt = torch.bfloat16
    cos, sin = (t.cuda() for t in R.tables(256, D))
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(50)).to(torch.int32).view(B, width)
    table_d = table.cuda()

    class Side:
        def __init__(self):
            self.cache = new_cache(kv4, B * width, Hkv, ps, D, dt, 0.0)
            self.prompt = new_cache(kv4, -(-T // ps), Hkv, ps, D, dt, 0.0)
            self.x = torch.zeros(steps, B, H + 2 * Hkv, D, dtype=dt, device="cuda")
            self.slots = torch.zeros(steps, B, dtype=torch.int64, device="cuda")
            self.pos = torch.zeros(steps, B, dtype=torch.int32, device="cuda")
            self.lens = torch.ones(steps, B, dtype=torch.int32, device="cuda")
            self.px = torch.zeros(T, H + 2 * Hkv, D, dtype=dt, device="cuda")
            self.pslots = torch.arange(T, device="cuda")
            self.ppos = torch.arange(T, dtype=torch.int32, device="cuda")
            self.cu = torch.tensor([0, 60, 61, T], dtype=torch.int32, device="cuda")
            self.qr = torch.zeros(steps, B, H, D, dtype=dt, device="cuda")
            self.o = torch.zeros(steps, B, H, 1, D, dtype=dt, device="cuda")
            self.lse = torch.zeros(steps, B, H, 1, device="cuda")
            self.pk = torch.zeros(T, Hkv, D, dtype=dt, device="cuda")
            self.pv = torch.zeros(T, Hkv, D, dtype=dt, device="cuda")
            self.po = torch.zeros(T, H, D, dtype=dt, device="cuda")
            self.plse = torch.zeros(H, T, device="cuda")
            self.ws = torch.empty(fattn.decode_workspace_bytes(B, H, 1, D, Hkv), dtype=torch.uint8, device="cuda")
            self.pws = torch.empty(fattn.packed_workspace_bytes(3, T), dtype=torch.uint8, device="cuda")

        def run(self, wait=lambda: None):
            turn = dict(cos=cos, sin=sin)
            pq, pk, pv = self.px[:, :H], self.px[:, H:H + Hkv], self.px[:, H + Hkv:]
            append(kv4, pk, pv, self.prompt, self.pslots, pos=self.ppos, q=pq, q_out=pq, k_out=self.pk, v_out=self.pv,
                   held=True, **turn)
            wait()
            fattn.fwd_packed(pq, self.pk, self.pv if kv4 else pv, self.cu, out=self.po, lse=self.plse,
                             workspace=self.pws)
            wait()
            for i in range(steps):
                x = self.x[i]
                append(kv4, x[:, H:H + Hkv], x[:, H + Hkv:], self.cache, self.slots[i], pos=self.pos[i], q=x[:, :H],
                       q_out=self.qr[i], **turn)
                wait()
                run_decode(kv4, self.qr[i].unsqueeze(2), self.cache, table_d, self.lens[i], out=self.o[i],
                           lse=self.lse[i], workspace=self.ws)
                wait()

        def outputs(self):
            return [self.qr, self.o, self.lse, self.pk, self.pv, self.po, self.plse, *self.cache, *self.prompt]

    sides, want = [Side(), Side()], Side()
    sides[0].run()  # (modules are loaded before a capture)
    for t in sides[0].outputs():
        t.zero_()
    graphs = []
    for side in sides:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                side.run()
        torch.cuda.current_stream().wait_stream(s)
        graphs.append((g, s))
    g = torch.Generator().manual_seed(51)
    at = torch.tensor([0, 17, 100])
    for t in want.outputs():
        t.zero_()
    for side in sides:
        for t in side.outputs():
            t.zero_()
    for _ in range(5):
        x = torch.randn(steps, B, H + 2 * Hkv, D, generator=g).to(dt)
        px = torch.randn(T, H + 2 * Hkv, D, generator=g).to(dt)
        pslots = torch.randperm(T, generator=g)
        for side in sides + [want]:
            side.x.copy_(x)
            side.px.copy_(px)
            side.pslots.copy_(pslots)
            for i in range(steps):
                j = at + i
                side.slots[i] = (table[torch.arange(B), j // ps].long() * ps + j % ps).cuda()
                side.pos[i] = j.to(torch.int32).cuda()
                side.lens[i] = (j + 1).to(torch.int32).cuda()
        torch.cuda.synchronize()
        for graph, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        ok()
        want.run(wait=torch.cuda.synchronize)
        ok()
        for side in sides:
            for i, (a, b) in enumerate(zip(side.outputs(), want.outputs())):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
        check_decode(kv4, want.qr[-1].unsqueeze(2), want.cache, table_d, want.lens[-1], fattn._default_scale(D),
                     sides[0].o[-1], sides[0].lse[-1])
        at = at + steps


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("Nq", [1, 3])
def test_decode_output_beside_its_query_in_one_tensor(kv4, Nq):
    B, H, Hkv, D = 3, 8, 2, 64
    q, cache, table, lens = make_decode(kv4, [100, 3, 33], H, Hkv, Nq, D, 32, "fp16", 60)
    want, want_l = run_decode(kv4, q, cache, table, lens)
    both = torch.full((B, Nq, 2 * H + 1, D), 7.0, dtype=q.dtype, device="cuda")
    both[:, :, :H] = q.transpose(1, 2)
    out = both[:, :, H:2 * H].transpose(1, 2)
    o, lse = run_decode(kv4, both[:, :, :H].transpose(1, 2), cache, table, lens, out=out)
    ok()
    assert o is out and torch.equal(o, want) and torch.equal(lse, want_l)
    assert torch.equal(both[:, :, :H].transpose(1, 2), q) and (both[:, :, 2 * H:] == 7).all()
    with pytest.raises(fattn.FattnError):
        run_decode(kv4, both[:, :, :H].transpose(1, 2), cache, table, lens, out=both[:, :, H - 1:2 * H - 1].transpose(1, 2))


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_inputs_made_on_another_stream(captured, kv4):
    """Tokens that another stream makes, late: the append waits for the event and for
    the kernel before it on its own stream, eager and in a graph with a fork and a join."""
    B, H, Hkv, D, ps, n = 4, 8, 2, 64, 16, 90
    dt = torch.float16
    q, cache, table, lens = make_decode(kv4, [n] * B, H, Hkv, 1, D, ps, "fp16", 61)
    j = torch.full((B,), n - 1)
    slots = (table.cpu().long()[torch.arange(B), j // ps] * ps + j % ps).cuda()
    src = torch.zeros(B, H + 2 * Hkv, D, dtype=dt, device="cuda")
    x = torch.zeros_like(src)
    slow = torch.zeros(1 << 27, device="cuda")
    o, lse = torch.zeros(B, H, 1, D, dtype=dt, device="cuda"), torch.zeros(B, H, 1, device="cuda")
    ws = torch.empty(fattn.decode_workspace_bytes(B, H, 1, D, Hkv), dtype=torch.uint8, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step(kv_cache, out, l):
        append(kv4, x[:, H:H + Hkv], x[:, H + Hkv:], kv_cache, slots, stream=torch.cuda.current_stream())
        run_decode(kv4, x[:, :H].unsqueeze(2), kv_cache, table, lens, out=out, lse=l, workspace=ws,
                   stream=torch.cuda.current_stream())

    def both():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            slow.add_(1.0)          # some 150 us
            x.copy_(src)
        append(kv4, src[:, H:H + Hkv], src[:, H + Hkv:], cache, slots, stream=main)  # a kernel right before the join
        main.wait_stream(side)
        step(cache, o, lse)

    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        both()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                both()
        g = torch.Generator(device="cuda").manual_seed(62)
        for _ in range(4):
            src.copy_(torch.randn(src.shape, generator=g, device="cuda"))
            x.fill_(9.0)
            other = [t.clone() for t in cache]
            if captured:
                graph.replay()
            else:
                both()
            torch.cuda.synchronize()
            assert torch.equal(x, src)
            want, want_l = torch.zeros_like(o), torch.zeros_like(lse)
            step(other, want, want_l)
            ok()
            assert torch.equal(o, want) and torch.equal(lse, want_l)
            for a, b in zip(cache, other):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv4", [False, True])
def test_decode_lse_has_the_accuracy_of_32_bits(kv4, D, dtype):
    """Over sequences of one key the LSE is the score itself.  4 bits: partial sums
    are some three times the score (codes about 7.5, taken off again by the
    zeros); with a dozen roundings of 2^-24 at most each, the root mean square
    of the error is 3 * sqrt(12 / 3) * 2^-24 = 3.6e-7 of the score's, below 2^-21."""
    B, H, Hkv, ps = 300, 16, 4, 16
    q, cache, table, lens = make_decode(kv4, [1] * B, H, Hkv, 1, D, ps, dtype, 70, q_std=3.0)
    scale = 0.125
    _, lse = run_decode(kv4, q, cache, table, lens, scale=scale)
    ok()
    if kv4:
        rows = [t[table[:, 0].long(), :, 0].cpu() for t in cache]
        k = R.held(rows[0], rows[1], "k")                    # [B, Hkv, D]
    else:
        k = cache[0][table[:, 0].long(), :, 0].cpu().double()
    want = (q.cpu().double()[:, :, 0] * k.repeat_interleave(H // Hkv, 1)).sum(-1) * scale
    err = lse.cpu().double()[..., 0] - want
    assert err.pow(2).mean().sqrt() <= 2.0 ** -21 * want.pow(2).mean().sqrt()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv4", [False, True])
def test_decode_small_weights_keep_their_bits(kv4, dtype):
    """One key in sixteen outweighs the others 2^17 times, but has the value 0: what
    is left is the others' weights, each rounded to a 16-bit type once."""
    n, H, Hkv, D, ps = 600, 4, 2, 64, 16
    dt = DT[dtype]
    q, cache, table, lens = make_decode(kv4, [n], H, Hkv, 1, D, ps, dtype, 80)
    q.zero_()
    q[..., 0] = 1.0
    # the score below the large one's, as a number of the type, whose weight lies worst between the multiples of 2^-24
    xs = torch.arange(11.0, 13.0, 1.0 / 128).to(torch.bfloat16 if dtype == "bf16" else torch.float16).double()
    w = torch.exp(-xs) * 2.0 ** 24
    x = xs[((w - w.floor() - 0.5).abs() + (w > 160) + (w < 60)).argmin()].item()
    for j in range(n):
        large, at = j % 16 == 5, (table[0, j // ps], slice(None), j % ps)
        if kv4:
            cache[1][at] = cache[3][at] = 0.0
            cache[1][at][..., 1] = 0.0 if large else -x
            cache[3][at][..., 1] = 0.0 if large else 1.0
        else:
            cache[0][at] = 0.0 if large else -x
            cache[1][at] = 0.0 if large else 1.0
    o, lse = run_decode(kv4, q, cache, table, lens, scale=1.0)
    ok()
    check_decode(kv4, q, cache, table, lens, 1.0, o, lse)
