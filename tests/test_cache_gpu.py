"""Appending to a paged cache and attention over it, 16 and 4 bits, against
plain 64-bit forms (tests/serving_ref.py)."""
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


def new_cache(kv4, P, Hkv, ps, D, dt, fill):
    """Cache tensors on the GPU, every element set (fill: 16-bit value)."""
    if not kv4:
        return [torch.full((P, Hkv, ps, D), fill, dtype=dt, device="cuda") for _ in range(2)]
    out = []
    for _ in range(2):
        out += [torch.full((P, Hkv, ps, D // 2), 0xA7, dtype=torch.uint8, device="cuda"),
                torch.full((P, Hkv, ps, D // 32, 2), fill, dtype=torch.float16, device="cuda")]
    return out


def append(kv4, k, v, cache, slots, **kw):
    if kv4:
        return fattn.cache_append_kv4(k, v, *cache, slots, **kw)
    kw.pop("v_out", None)
    kw.pop("held", None)
    return fattn.cache_append(k, v, *cache, slots, **kw)


def qkv_slices(T, H, Hkv, D, dt, seed, std=1.0):
    """q, k, v as slices of one projection's output, on the GPU."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H + 2 * Hkv, D, generator=g) * std).to(dt).cuda()
    return x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]


def check_quantised(x, mag, codes, scales, which, what):
    """codes, scales [.., Hkv, D/2], [.., Hkv, D/32, 2] on the CPU hold x (float64)."""
    ex = 3 * 2.0 ** -24 * mag  # error of the fp32 values that were quantised
    xg, eg = x.unflatten(-1, (-1, 32)), ex.unflatten(-1, (-1, 32)).amax(-1)
    lo, hi = xg.amin(-1), xg.amax(-1)
    s, z = scales[..., 0].double(), scales[..., 1].double()
    u16, t16 = 2.0 ** -11, R.tiny(torch.float16)
    assert ((z - lo).abs() <= u16 * (lo.abs() + eg) + eg + t16).all(), what
    step = (hi - lo) / 15
    es = 2 * eg / 15 + 2.0 ** -22 * step
    assert ((s - step).abs() <= u16 * (step + es) + es + t16).all(), what
    c = R.unpack(codes, which).double().unflatten(-1, (-1, 32))
    sd = torch.where(s > 0, s, 1.0)[..., None]
    want = torch.where(s[..., None] > 0, (xg - z[..., None]) / sd, 0.0).clamp(0, 15)
    # code = rint of an fp32 quotient: half a step, the input's error in steps, fp32 roundings of values up to ~16
    slack = 0.5 + (eg[..., None] / sd) + 2.0 ** -18
    assert ((c - want).abs() <= slack).all(), what


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype,D,H,Hkv,T,ps,rot", [
    ("bf16", 128, 4, 2, 67, 16, 128), ("fp16", 64, 8, 1, 33, 48, 32), ("bf16", 64, 5, 5, 1, 16, 64),
    ("fp16", 128, 3, 1, 3, 32, 16), ("bf16", 128, 40, 8, 9, 64, 64), ("fp16", 64, 1, 1, 130, 16, 0),
    ("fp16", 64, 2, 1, 20001, 16, 64), ("bf16", 128, 1, 1, 9001, 32, 128)])  # the most tokens that a block takes
def test_append(dtype, D, H, Hkv, T, ps, rot, kv4, interleaved):
    dt = DT[dtype]
    P = -(-T // ps) + 2
    q, k, v = qkv_slices(T, H, Hkv, D, dt, T + D)
    g = torch.Generator().manual_seed(5)
    slots = torch.randperm(P * ps, generator=g)[:T]
    if T > 2:
        slots[1] = -1          # a padded token
        slots[T - 1] = -7
    pos = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32)
    cos, sin = R.tables(5000, rot)
    cache = new_cache(kv4, P, Hkv, ps, D, dt, 3.5)
    before = [t.cpu().clone() for t in cache]
    k_out, v_out = (torch.full((T, Hkv, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    q_out = torch.full((T, H, D), 7.0, dtype=dt, device="cuda")
    rotation = dict(pos=pos.cuda(), cos=cos.cuda(), sin=sin.cuda(), interleaved=interleaved) if rot else {}
    append(kv4, k, v, cache, slots.cuda(), q=q, q_out=q_out, k_out=k_out, v_out=v_out, **rotation)
    ok()
    live = slots >= 0
    qr, qm = R.rotate(q.cpu(), pos, cos, sin, interleaved)
    kr, km = R.rotate(k.cpu(), pos, cos, sin, interleaved)
    R.check(q_out[live.cuda()], qr[live], R.rotated_bound(qr, qm, dt)[live], "q_out")
    R.check(k_out[live.cuda()], kr[live], R.rotated_bound(kr, km, dt)[live], "k_out")
    for t in (q_out, k_out) + ((v_out,) if kv4 else ()):
        assert (t.cpu()[~live] == 7.0).all()  # a padded token's rows are left as they were
    pg, at = slots[live] // ps, slots[live] % ps
    after = [t.cpu() for t in cache]
    if not kv4:
        assert torch.equal(after[0][pg, :, at], k_out.cpu()[live])
        assert torch.equal(after[1][pg, :, at], v.cpu()[live])
    else:
        assert torch.equal(v_out.cpu()[live], v.cpu()[live])
        check_quantised(kr[live], km[live], after[0][pg, :, at], after[1][pg, :, at], "k", "K")
        check_quantised(v.cpu().double()[live], torch.zeros_like(v.cpu().double()[live]), after[2][pg, :, at],
                        after[3][pg, :, at], "v", "V")
        # the values that the cache stands for
        append(kv4, k, v, cache, slots.cuda(), q=q, q_out=q_out, k_out=k_out, v_out=v_out, held=True, **rotation)
        ok()
        for n, out, c, sc in (("k", k_out, after[0], after[1]), ("v", v_out, after[2], after[3])):
            val = R.held(c[pg, :, at], sc[pg, :, at], n)
            size = val.abs() + 16 * sc[pg, :, at][..., 0].double().repeat_interleave(32, -1)
            R.check(out[live.cuda()], val, R.u_of(dt) * (1 + 2.0 ** -10) * val.abs() + 2.0 ** -23 * size + R.tiny(dt), n)
    for b, a in zip(before, after):  # every other slot is left as it was
        a = a.clone()
        a[pg, :, at] = b[pg, :, at]
        assert torch.equal(a, b)


def test_append_in_place_without_q_and_head_major():
    T, H, Hkv, D, ps = 21, 6, 3, 128, 16
    dt = torch.bfloat16
    q, k, v = qkv_slices(T, H, Hkv, D, dt, 3)
    cos, sin = (t.cuda() for t in R.tables(64, D))
    pos, slots = torch.arange(T, dtype=torch.int32).cuda(), torch.arange(T).cuda()
    c1, c2, c3 = (new_cache(False, 2, Hkv, ps, D, dt, 0.0) for _ in range(3))
    q_ref, k_ref = fattn.cache_append(k, v, *c1, slots, pos=pos, cos=cos, sin=sin, q=q,
                                      k_out=torch.empty(T, Hkv, D, dtype=dt, device="cuda"))
    # without q
    assert fattn.cache_append(k, v, *c2, slots, pos=pos, cos=cos, sin=sin) == (None, None)
    # head-major inputs, and q and k turned in place
    qh, kh, vh = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    out = fattn.cache_append(kh, vh, *c3, slots, pos=pos, cos=cos, sin=sin, q=qh, q_out=qh, k_out=kh)
    ok()
    assert out[0] is qh and torch.equal(qh, q_ref) and torch.equal(kh, k_ref)
    for a, b, c in zip(c1, c2, c3):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("kv4", [False, True])
def test_append_index_out_of_range_is_skipped_and_reported(kv4):
    T, Hkv, D, ps, P = 6, 2, 64, 16, 2
    dt = torch.float16
    _, k, v = qkv_slices(T, 1, Hkv, D, dt, 4)
    cos, sin = (t.cuda() for t in R.tables(8, D))
    for slots, pos in (([0, 1, P * ps, 3, 1 << 40, 5], [0, 1, 2, 3, 4, 5]),
                       ([0, 1, 2, 3, 4, 5], [0, 1, 8, 3, -1, 5])):
        cache = new_cache(kv4, P, Hkv, ps, D, dt, 2.0)
        before = [t.clone() for t in cache]
        append(kv4, k, v, cache, torch.tensor(slots).cuda(), cos=cos, sin=sin,
               pos=torch.tensor(pos, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert fattn.get_device_status() == INVALID
        assert fattn.get_device_status() == 0
        for a, b in zip(cache, before):
            written = (a != b).flatten(3).any(-1).any(1)  # [P, ps]
            assert written.flatten().nonzero().flatten().tolist() == [0, 1, 3, 5]


def test_append_kv4_special_values():
    D, ps = 64, 16
    x = torch.randn(5, 1, D, generator=torch.Generator().manual_seed(6))
    x[0] = 0.0                       # a constant row: scale 0
    x[1, 0, :32] = -3.25
    x[2, 0, 3] = math.nan
    x[3, 0, 5] = math.inf
    x[4, 0, :32] = math.nan
    x = x.to(torch.bfloat16).cuda()
    cache = new_cache(True, 1, 1, ps, D, torch.bfloat16, 0.0)
    slots = torch.arange(5).cuda()
    k_out, v_out = torch.empty_like(x), torch.empty_like(x)
    fattn.cache_append_kv4(x, x, *cache, slots, k_out=k_out, v_out=v_out, held=True)
    ok()
    for out in (k_out, v_out):
        assert torch.isfinite(out).all()
        assert (out[0] == 0).all() and (out[1, 0, :32] == -3.25).all()
        row = x[2, 0].double().cpu()
        fine = torch.cat([row[:3], row[4:32]])
        assert abs(out[2, 0, 3].item() - fine.min().item()) <= 2.0 ** -8 * abs(fine.min().item())
        step = (fine.max() - fine.min()).item() / 15
        assert (torch.cat([out[2, 0, :3], out[2, 0, 4:32]]).double().cpu() - fine).abs().max() <= 0.6 * step
        assert out[3, 0, 5].item() == 65536.0  # 65504 rounded to bf16
        assert (out[4, 0, :32] == 0).all()
    for t in (cache[1], cache[3]):
        assert torch.isfinite(t).all()


# ---------------------------------------------------------------------------
# Attention over the cache
# ---------------------------------------------------------------------------
def make_decode(kv4, lens, H, Hkv, Nq, D, ps, dtype, seed, q_std=2.0, spare=2):
    """Inputs on the GPU.  Slots behind each sequence's last token hold NaN, and
    table entries behind its last page are out of range: none may be used."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    need = [-(-n // ps) for n in lens]
    P = sum(need) + spare
    W = max(max(need), 1)
    perm = torch.randperm(P, generator=g)
    table = torch.full((B, W), 1 << 30, dtype=torch.int32)
    table[:, ::2] = -1
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    q = (torch.randn(B, H, Nq, D, generator=g) * q_std).to(dt)
    used = torch.zeros(P, ps, dtype=torch.bool)
    for b, n in enumerate(lens):
        j = torch.arange(n)
        used[table[b].long()[j // ps], j % ps] = True
    hidden = ~used[:, None, :, None]
    if kv4:
        cache = []
        for which in "kv":
            cache.append(R.pack(torch.randint(0, 16, (P, Hkv, ps, D), generator=g), which))
            s = 0.05 + 0.4 * torch.rand(P, Hkv, ps, D // 32, generator=g)
            z = -7.5 * s + 0.3 * torch.randn(s.shape, generator=g)
            cache.append(torch.stack([s, z], -1).half().masked_fill(hidden[..., None], math.nan))
    else:
        cache = [torch.randn(P, Hkv, ps, D, generator=g).to(dt).masked_fill(hidden, math.nan) for _ in range(2)]
    return q.cuda(), [t.cuda() for t in cache], table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def run_decode(kv4, q, cache, table, lens, **kw):
    return (fattn.decode_kv4 if kv4 else fattn.decode)(q, *cache, table, lens, **kw)


def check_decode(kv4, q, cache, table, lens, scale, o, lse, what=""):
    B, H, Nq, D = q.shape
    dt = q.dtype
    cache, table = [t.cpu() for t in cache], table.cpu()
    for b, n in enumerate(lens.tolist()):
        ends = [max(0, n - Nq + 1 + i) for i in range(Nq)]
        v_err = 0.0
        if kv4:
            rows = [R.gather(t, table[b], n) for t in cache]
            k, v = R.held(rows[0], rows[1], "k"), R.held(rows[2], rows[3], "v")
            # V enters as an fp16 number: off by 2^-11 of the value, and its
            # offset within the conversion (|zero| + 16 scale) by 2^-11 of that
            off = (rows[3][..., 1].double().abs() + 16 * rows[3][..., 0].double()).repeat_interleave(32, -1)
            verr = 2.0 ** -11 * (v.abs() + off)
        else:
            k, v = (R.gather(t, table[b], n).double() for t in cache)
            verr = None
        ro, rl, av, worst = R.attend(q[b].cpu().double(), k, v, scale, ends)
        if kv4:
            _, _, v_err, _ = R.attend(q[b].cpu().double(), k, verr, scale, ends)
        u_p = 2.0 ** -11 if kv4 else R.u_of(dt)
        bo, bl = R.attend_bounds(ro, rl, av, worst, D, dt, u_p, v_err)
        empty = torch.tensor([e == 0 for e in ends])
        got_l = lse[b].cpu().double()
        assert (o[b].cpu()[:, empty] == 0).all() and (got_l[:, empty] == -math.inf).all(), what
        if (~empty).any():
            R.check(o[b][:, (~empty).cuda()], ro[:, ~empty], bo[:, ~empty], "%s O, sequence %d of %d" % (what, b, n))
            R.check(got_l[:, ~empty], rl[:, ~empty], bl[:, ~empty], "%s LSE, sequence %d of %d" % (what, b, n))


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 127, 129, 300, 1000]


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype,D,H,Hkv,Nq,ps", [
    ("bf16", 128, 8, 2, 1, 16), ("fp16", 64, 4, 4, 1, 32), ("bf16", 64, 6, 2, 2, 48), ("fp16", 128, 16, 1, 1, 64),
    ("bf16", 128, 32, 1, 1, 16), ("fp16", 64, 8, 1, 4, 128), ("bf16", 64, 10, 1, 7, 16), ("fp16", 128, 5, 1, 1, 80)])
def test_decode(dtype, D, H, Hkv, Nq, ps, kv4):
    q, cache, table, lens = make_decode(kv4, LENS, H, Hkv, Nq, D, ps, dtype, D + H + Nq)
    scale = fattn._default_scale(D)
    o, lse = run_decode(kv4, q, cache, table, lens)
    ok()
    check_decode(kv4, q, cache, table, lens, scale, o, lse)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("B,H,Hkv,n", [(1, 8, 1, 20011), (1, 32, 8, 4097), (200, 4, 2, 70), (2, 64, 1, 3000)])
def test_decode_work_splits(B, H, Hkv, n, kv4):
    """Few long sequences (the keys are split over the GPU) and many short ones."""
    lens = [max(1, n - 13 * b) for b in range(B)]
    q, cache, table, lens = make_decode(kv4, lens, H, Hkv, 1, 128, 64, "bf16", B + n, q_std=1.0)
    o, lse = run_decode(kv4, q, cache, table, lens, scale=0.25)
    ok()
    check_decode(kv4, q, cache, table, lens, 0.25, o, lse)
    o2, lse2 = run_decode(kv4, q, cache, table, lens, scale=0.25)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # the same call, the same bits


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_scores_of_any_size(kv4):
    """Scores far from zero, rising along the keys (every key moves the running
    max), equal scores, and scale 0."""
    D, ps, n = 64, 16, 700
    q, cache, table, lens = make_decode(kv4, [n], 4, 2, 1, D, ps, "fp16", 9)
    if kv4:
        cache[0].fill_(0)
        ramp = torch.arange(n, device="cuda").half() * 0.25 - 90
        for j in range(-(-n // ps)):
            part = ramp[j * ps:(j + 1) * ps]
            cache[1][table[0, j], :, :len(part), :, 1] = part[None, :, None]
            cache[1][table[0, j], :, :len(part), :, 0] = 0
    else:
        for j in range(n):
            cache[0][table[0, j // ps], :, j % ps] = 0.25 * j - 90
    for scale in (0.125, 1.0, 0.0):
        for sign in (1.0, -1.0):
            qq = (q.abs() * sign).contiguous()
            o, lse = run_decode(kv4, qq, cache, table, lens, scale=scale)
            ok()
            check_decode(kv4, qq, cache, table, lens, scale, o, lse, "scale %g" % (scale * sign))


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_tables_out_of_range(kv4):
    """A page out of range among those a sequence uses: its keys take no part;
    a length outside the table: cut to it.  Both are reported."""
    D, ps = 128, 16
    q, cache, table, lens = make_decode(kv4, [64, 48], 4, 2, 1, D, ps, "bf16", 10)
    good, _ = run_decode(kv4, q, cache, table, lens)
    ok()
    for bad_page in (-1, cache[0].shape[0], 1 << 30):
        t = table.clone()
        t[0, 1] = bad_page
        o, lse = run_decode(kv4, q, cache, t, lens)
        torch.cuda.synchronize()
        assert fattn.get_device_status() == INVALID and fattn.get_device_status() == 0
        assert torch.equal(o[1], good[1])
        # the keys of the other three pages, in an order of its own
        t4 = torch.stack([table[0, 0], table[0, 2], table[0, 3]])[None].contiguous()
        one = torch.tensor([48], dtype=torch.int32).cuda()
        check_decode(kv4, q[:1], cache, t4, one, fattn._default_scale(D), o[:1], lse[:1], "page %d" % bad_page)
    for bad_len in (-5, 4 * ps + 1, 2 ** 31 - 1):
        l = lens.clone()
        l[0] = bad_len
        o, lse = run_decode(kv4, q, cache, table, l)
        torch.cuda.synchronize()
        assert fattn.get_device_status() == INVALID and fattn.get_device_status() == 0
        assert torch.equal(o[1], good[1])
        if bad_len < 0:
            assert (o[0] == 0).all() and (lse[0] == -math.inf).all()
        else:
            assert torch.equal(o[0], good[0])


def test_decode_strides_and_page_stride():
    """q as a slice of a projection, o token-major, K and V pages in one tensor."""
    B, H, Hkv, Nq, D, ps = 3, 8, 2, 2, 64, 32
    dt = torch.float16
    q, cache, table, lens = make_decode(False, [100, 3, 33], H, Hkv, Nq, D, ps, "fp16", 11)
    o, lse = fattn.decode(q, *cache, table, lens)
    both = torch.stack(cache, 1).contiguous()  # [P, 2, Hkv, ps, D]
    proj = torch.zeros(B, Nq, H + 2 * Hkv, D, dtype=dt, device="cuda")
    proj[:, :, :H] = q.transpose(1, 2)
    out = torch.zeros(B, Nq, H, D, dtype=dt, device="cuda")
    o2, lse2 = fattn.decode(proj[:, :, :H].transpose(1, 2), both[:, 0], both[:, 1], table, lens,
                            out=out.transpose(1, 2))
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(out.transpose(1, 2), o)
    o3, none = fattn.decode(q, *cache, table, lens, return_lse=False)
    assert none is None and torch.equal(o3, o)
    # an append into the shared tensor, through its page stride
    _, k, v = qkv_slices(2, 1, Hkv, D, dt, 12)
    slots = torch.tensor([5, ps * (both.shape[0] - 1) + 1]).cuda()
    before = both.clone()
    fattn.cache_append(k, v, both[:, 0], both[:, 1], slots)
    ok()
    for t in range(2):
        p, at = slots[t].item() // ps, slots[t].item() % ps
        assert torch.equal(both[p, 0, :, at], k[t]) and torch.equal(both[p, 1, :, at], v[t])
        both[p, :, :, at] = before[p, :, :, at]
    assert torch.equal(both.nan_to_num(9.0), before.nan_to_num(9.0))


@pytest.mark.parametrize("kv4", [False, True])
def test_offsets_past_32_bits(kv4):
    """A pool of more than 2^32 bytes per tensor (16 bits: more than 2^31
    elements): the last pages are written and read where they are."""
    Hkv, ps, D = 8, 64, 128
    P = (1 << 32) // (Hkv * ps * (D // 2 if kv4 else 2 * D)) + 40
    if kv4:
        cache = []
        for _ in range(2):
            cache += [torch.empty(P, Hkv, ps, D // 2, dtype=torch.uint8, device="cuda"),
                      torch.empty(P, Hkv, ps, D // 32, 2, dtype=torch.float16, device="cuda")]
    else:
        cache = [torch.empty(P, Hkv, ps, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    n = 150
    pages = torch.tensor([P - 1, 3, P - 7], dtype=torch.int32)
    q, k, v = qkv_slices(n, 16, Hkv, D, torch.bfloat16, 13)
    j = torch.arange(n)
    slots = pages.long()[j // ps] * ps + j % ps
    append(kv4, k, v, cache, slots.cuda())
    qd = q[-1:].unsqueeze(2).contiguous()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    o, lse = run_decode(kv4, qd, cache, pages[None].cuda(), lens, scale=0.1)
    ok()
    small = new_cache(kv4, 3, Hkv, ps, D, torch.bfloat16, 0.0)
    append(kv4, k, v, small, j.cuda())
    table = torch.arange(3, dtype=torch.int32)[None].cuda()
    o2, lse2 = run_decode(kv4, qd, small, table, lens, scale=0.1)
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_decode(kv4, qd, small, table, lens, 0.1, o, lse)


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_more_sequences_than_threads(kv4):
    """The prefix sums over sequences run in pieces; many are empty, one is long."""
    g = torch.Generator().manual_seed(17)
    lens = torch.randint(0, 40, (700,), generator=g)
    lens[torch.randperm(700, generator=g)[:200]] = 0
    lens[601] = 3000
    q, cache, table, lens = make_decode(kv4, lens.tolist(), 4, 2, 1, 64, 16, "fp16", 18)
    o, lse = run_decode(kv4, q, cache, table, lens)
    ok()
    check_decode(kv4, q, cache, table, lens, 0.125, o, lse)


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_workspace_contents_are_ignored(kv4):
    """Whatever the workspace holds on entry, also what calls of other shapes
    left in it, the result is the same."""
    n = [2000, 0, 300, 5000]
    q, cache, table, lens = make_decode(kv4, n, 8, 2, 1, 128, 32, "bf16", 19)
    want, want_l = run_decode(kv4, q, cache, table, lens)
    ws = torch.empty(fattn.decode_workspace_bytes(4, 64, 4, 128, 2), dtype=torch.uint8, device="cuda")
    other = make_decode(kv4, [700, 900], 64, 2, 4, 128, 16, "bf16", 20)
    for fill in (0, 1, 0x5B, 0xFF, None, None):
        if fill is None:  # a call of another shape, with the same workspace, right before
            run_decode(kv4, *other, workspace=ws)
        else:
            ws.fill_(fill)
        for _ in range(2):
            o, lse = run_decode(kv4, q, cache, table, lens, workspace=ws)
            ok()
            assert torch.equal(o, want) and torch.equal(lse, want_l)
    g = torch.Generator(device="cuda").manual_seed(21)
    for _ in range(3):
        ws.random_(0, 256, generator=g)
        o, lse = run_decode(kv4, q, cache, table, lens, workspace=ws)
        ok()
        assert torch.equal(o, want) and torch.equal(lse, want_l)


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_non_finite_query_stays_in_its_row(kv4):
    q, cache, table, lens = make_decode(kv4, [100, 260], 8, 2, 2, 64, 16, "fp16", 22)
    want, want_l = run_decode(kv4, q, cache, table, lens)
    for bad in (math.nan, math.inf):
        q2 = q.clone()
        q2[0, 3, 1, 5] = bad
        q2[1, 6, 0, :] = bad
        o, lse = run_decode(kv4, q2, cache, table, lens)
        ok()
        keep = torch.ones(q.shape[:3], dtype=torch.bool, device="cuda")
        keep[0, 3, 1] = keep[1, 6, 0] = False
        assert torch.equal(o[keep], want[keep]) and torch.equal(lse[keep], want_l[keep])
        assert torch.isnan(o[~keep]).all()


def test_decode_padded_batch_and_shared_pages():
    """Rows of a padded batch have length 0; sequences may share pages."""
    H, Hkv, D, ps = 8, 4, 128, 16
    q, cache, table, lens = make_decode(False, [120, 64, 0, 0], H, Hkv, 1, D, ps, "bf16", 23)
    table[2:] = table[0]
    table[1, :2] = table[0, :2]
    table[1, 2:4] = table[0, 4:6]
    o, lse = fattn.decode(q, *cache, table, lens)
    ok()
    check_decode(False, q, cache, table, lens, fattn._default_scale(D), o, lse)


@pytest.mark.parametrize("kv4", [False, True])
def test_streams_and_graphs(kv4):
    """A step on another stream, captured and replayed with lengths and tables
    that change between replays; two graphs with a workspace each."""
    H, Hkv, D, ps, B = 8, 2, 128, 16, 3
    q, cache, table, lens = make_decode(kv4, [200, 7, 90], H, Hkv, 1, D, ps, "bf16", 14)
    _, k, v = qkv_slices(B, 1, Hkv, D, torch.bfloat16, 15)
    slots = torch.tensor([-1] * B).cuda()
    o = torch.zeros_like(q)
    lse = torch.zeros(B, H, 1, device="cuda")
    wss = [torch.empty(fattn.decode_workspace_bytes(B, H, 1, D, Hkv), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(stream=None, ws=None, out=o, l=lse):
        append(kv4, k, v, cache, slots, stream=stream)
        return run_decode(kv4, q, cache, table, lens, out=out, lse=l, workspace=ws, stream=stream)

    step(ws=wss[0])
    ok()
    first = o.clone()
    outs = [(torch.zeros_like(o), torch.zeros_like(lse)) for _ in range(2)]
    graphs = []
    for ws, (oo, ll) in zip(wss, outs):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                step(stream=s, ws=ws, out=oo, l=ll)
        torch.cuda.current_stream().wait_stream(s)
        graphs.append((g, s))
    for lengths in ([200, 7, 90], [1, 7, 33], [0, 3, 80]):
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in graphs:   # both at once, on their own streams
                with torch.cuda.stream(s):
                    g.replay()
        ok()
        want, want_l = step()
        ok()
        for oo, ll in outs:
            assert torch.equal(oo, want) and torch.equal(ll, want_l)
        check_decode(kv4, q, cache, table, lens, fattn._default_scale(D), *outs[0])
    lens.copy_(torch.tensor([200, 7, 90], dtype=torch.int32))
    step()
    assert torch.equal(o, first)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_kv4_ties_round_to_even(dtype):
    """Values on a coarse grid, where (x - zero) / scale is often exactly k + 1/2:
    every code is the exact quotient's rounding, ties to even."""
    D, ps, T = 128, 16, 160
    g = torch.Generator().manual_seed(16)
    x = torch.randint(-1024, 1025, (T, 1, D), generator=g).float() / 256
    # ranges of 15 * 2^k grid steps: scales that are powers of two
    for i in range(T // 2):
        lo = x[i, 0].view(4, 32).amin(-1, keepdim=True)
        span = torch.randint(0, 31, (4, 32), generator=g).float() * 2.0 ** -(1 + i % 4)
        x[i, 0] = (lo + span.clamp(max=30 * 2.0 ** -(1 + i % 4))).flatten()
        x[i, 0, ::32] = lo.flatten()
        x[i, 0, 1::32] = lo.flatten() + 30 * 2.0 ** -(1 + i % 4)
    x = x.to(DT[dtype])
    cache = new_cache(True, T // ps, 1, ps, D, DT[dtype], 0.0)
    fattn.cache_append_kv4(x.cuda(), x.cuda(), *cache, torch.arange(T).cuda())
    ok()
    ties = 0
    for which, codes, scales in (("k", cache[0], cache[1]), ("v", cache[2], cache[3])):
        c = R.unpack(codes.cpu().transpose(1, 2).reshape(T, 1, D // 2), which).double()
        s = scales.cpu().double().transpose(1, 2).reshape(T, 1, D // 32, 2).repeat_interleave(32, dim=2)
        q = (x.double() - s[..., 1]) / s[..., 0]
        q = torch.where(s[..., 0] > 0, q, 0.0).clamp(0, 15)
        ties += ((q - q.floor()) == 0.5).sum().item()
        assert torch.equal(c, q.round())
    assert ties > 1000


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype,D,H,Hkv,Nq,ps", [("bf16", 128, 8, 8, 1, 16), ("fp16", 64, 16, 1, 1, 32),
                                                ("bf16", 64, 32, 2, 2, 48), ("fp16", 128, 40, 1, 2, 16),
                                                ("bf16", 128, 16, 1, 1, 64), ("fp16", 64, 6, 6, 3, 16)])
def test_decode_short_sequences(dtype, D, H, Hkv, Nq, ps, kv4):
    """Many short sequences (where there are enough, a warp takes each), some of
    the next longer kind among them."""
    g = torch.Generator().manual_seed(24)
    B = 660 // Hkv + 1
    lens = torch.randint(0, 300, (B,), generator=g)
    lens[::7] = torch.randint(200, 700, (len(lens[::7]),), generator=g)
    lens[3] = lens[4] = 0
    lens[50] = 40
    q, cache, table, lens = make_decode(kv4, lens.tolist(), H, Hkv, Nq, D, ps, dtype, 25)
    table[50, 0] = -1  # a page out of range: that sequence alone changes
    o, lse = run_decode(kv4, q, cache, table, lens)
    torch.cuda.synchronize()
    assert fattn.get_device_status() == INVALID
    keep = torch.arange(B) != 50
    check_decode(kv4, q[keep.cuda()], cache, table[keep.cuda()], lens[keep.cuda()], fattn._default_scale(D),
                 o[keep.cuda()], lse[keep.cuda()])
    assert torch.isfinite(o[50]).all()


@pytest.mark.parametrize("D,rot,dtype,interleaved", [(128, 128, "bf16", False), (64, 32, "fp16", True),
                                                     (64, 64, "bf16", False)])
def test_append_kv4_rotated_codes_are_the_definitions(D, rot, dtype, interleaved):
    """Of 50000 groups and more, some hundred lie so close to a rounding's border
    that fp32 cannot tell its side: all their codes, scales and zeros are those
    of the rotation in 64 bits (scale and zero as fp16 of the nearest fp32)."""
    T, Hkv, ps = 8000, 2, 16
    g = torch.Generator().manual_seed(27)
    k = (torch.randn(T, Hkv, D, generator=g) * 2.0 ** torch.randint(-9, 10, (T, 1, 1), generator=g)).to(DT[dtype])
    k[5] = 0.0
    k[6, 1, : D // 2] = 0.0
    k[7] = 1.0
    pos = torch.randint(0, 4096, (T,), generator=g, dtype=torch.int32)
    cos, sin = R.tables(4096, rot)
    cache = new_cache(True, T // ps, Hkv, ps, D, DT[dtype], 0.0)
    fattn.cache_append_kv4(k.cuda(), k.cuda(), *cache, torch.arange(T).cuda(), pos=pos.cuda(), cos=cos.cuda(),
                           sin=sin.cuda(), interleaved=interleaved)
    ok()
    x = R.rotate(k, pos, cos, sin, interleaved)[0].unflatten(-1, (-1, 32))
    lo, hi = x.amin(-1), x.amax(-1)
    scale, zero = ((hi - lo) / 15).float().half().double(), lo.float().half().double()
    got = cache[1].cpu().double().transpose(1, 2).reshape(T, Hkv, D // 32, 2)
    assert torch.equal(got[..., 0], scale) and torch.equal(got[..., 1], zero)
    q = (x - zero[..., None]) / torch.where(scale > 0, scale, 1.0)[..., None]
    want = torch.where(scale[..., None] > 0, q, 0.0).clamp(0, 15).round().flatten(-2)
    codes = R.unpack(cache[0].cpu().transpose(1, 2).reshape(T, Hkv, D // 2), "k").double()
    assert torch.equal(codes, want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_kv4_rotated_infinities_take_the_ends(interleaved):
    """An infinite element makes both of its rotated pair infinite: they stand for
    fp16's ends, beside which the group's other elements keep their codes."""
    T, D, ps = 320, 64, 16
    g = torch.Generator().manual_seed(28)
    k = torch.randn(T, 1, D, generator=g) * 2.0 ** torch.randint(0, 16, (T, 1, 1), generator=g)
    k[torch.arange(T), 0, torch.randint(0, D, (T,), generator=g)] = math.inf
    k[::2] = -k[::2]
    k = k.to(torch.bfloat16)
    pos = torch.randint(1, 512, (T,), generator=g, dtype=torch.int32)
    cos, sin = R.tables(512, D)
    assert (cos[1:] != 0).all() and (sin[1:] != 0).all()
    cache = new_cache(True, T // ps, 1, ps, D, torch.bfloat16, 0.0)
    fattn.cache_append_kv4(k.cuda(), k.cuda(), *cache, torch.arange(T).cuda(), pos=pos.cuda(), cos=cos.cuda(),
                           sin=sin.cuda(), interleaved=interleaved)
    ok()
    x = R.rotate(k, pos, cos, sin, interleaved)[0].clamp(-65504, 65504).unflatten(-1, (-1, 32))
    assert (x.abs() == 65504).flatten(1).sum(1).ge(2).all()
    lo, hi = x.amin(-1), x.amax(-1)
    scale, zero = ((hi - lo) / 15).float().half().double(), lo.float().half().double()
    got = cache[1].cpu().double().transpose(1, 2).reshape(T, 1, D // 32, 2)
    assert torch.equal(got[..., 0], scale) and torch.equal(got[..., 1], zero)
    want = ((x - zero[..., None]) / scale[..., None]).clamp(0, 15).round().flatten(-2)
    codes = R.unpack(cache[0].cpu().transpose(1, 2).reshape(T, 1, D // 2), "k").double()
    assert torch.equal(codes, want)
