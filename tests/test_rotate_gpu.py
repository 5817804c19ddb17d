"""Rotation by positions with several axes: rotate, its gradient, and the appends
with axes, against plain 64-bit forms."""
import math

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import more_ref as M
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
MAX_POS = 700


def ok():
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 0


def axes_of(kind, rot, A):
    n = rot // 2
    if kind == "in turn":
        return bytes(i % A for i in range(n))
    each = n // A
    return fattn.rotary_axes([n - each * (A - 1)] + [each] * (A - 1))


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D,rot,A,kind", [("bf16", 128, 128, 3, "sections"), ("fp16", 64, 64, 2, "in turn"),
                                                ("bf16", 64, 32, 3, "in turn"), ("fp16", 128, 16, 8, "in turn"),
                                                ("fp16", 128, 48, 1, "sections"), ("bf16", 64, 64, 3, "sections")])
@pytest.mark.parametrize("B,H,Hkv,N", [(1, 1, 1, 1), (2, 8, 2, 67), (3, 5, 5, 129)])
def test_rotate(B, H, Hkv, N, dtype, D, rot, A, kind, interleaved, inverse):
    """From slices of a projection into contiguous tensors."""
    dt, g = DT[dtype], torch.Generator().manual_seed(N + rot)
    qkv = torch.randn(B, N, H + 2 * Hkv, D, generator=g).to(dt)
    pos = torch.randint(0, MAX_POS, (A, B, N), generator=g, dtype=torch.int32)
    cos, sin = R.tables(MAX_POS, rot)
    axes = axes_of(kind, rot, A)
    x = qkv.cuda()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    qo, ko = fattn.rotate(q, pos.cuda(), cos.cuda(), sin.cuda(), axes=axes, interleaved=interleaved, inverse=inverse, k=k)
    ok()
    assert qo.is_contiguous() and ko.is_contiguous() and torch.equal(x.cpu(), qkv)
    for got, src in ((qo, q), (ko, k)):
        y, mag = M.rotated(src.cpu(), pos, axes, cos, sin, interleaved, inverse)
        R.check(got, y, R.rotated_bound(y, mag, dt), "rotate")
        assert torch.equal(got[..., rot:], src[..., rot:])


def test_in_place_slices_and_one_axis():
    """In place on a projection's slices, into its gradient's layout, without k, with one axis: the same bits."""
    B, N, H, Hkv, D = 2, 70, 4, 2, 64
    g = torch.Generator().manual_seed(1)
    x = torch.randn(B, N, H + 2 * Hkv, D, generator=g).half().cuda()
    cos, sin = (t.cuda() for t in R.tables(MAX_POS, D))
    pos = torch.randint(0, MAX_POS, (B, N), generator=g, dtype=torch.int32).cuda()
    q, k = x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hkv].transpose(1, 2)
    qo, ko = fattn.rotate(q, pos, cos, sin, k=k)
    q1, none = fattn.rotate(q, pos, cos, sin)
    q3, _ = fattn.rotate(q, pos[None].expand(3, -1, -1).contiguous(), cos, sin, axes=bytes(i % 3 for i in range(32)))
    ok()
    assert none is None and torch.equal(q1, qo) and torch.equal(q3, qo)
    y = torch.full_like(x, 7.0)
    fattn.rotate(q, pos, cos, sin, k=k, q_out=y[:, :, :H].transpose(1, 2), k_out=y[:, :, H:H + Hkv].transpose(1, 2))
    v = x[:, :, H + Hkv:].clone()
    fattn.rotate(q, pos, cos, sin, k=k, q_out=q, k_out=k)
    ok()
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(x[:, :, H + Hkv:], v)
    assert torch.equal(y[:, :, :H + Hkv], x[:, :, :H + Hkv]) and (y[:, :, H + Hkv:] == 7).all()


def test_cache_appends_rotation_is_this_one():
    """The same rows through cache_append turn to the same bits."""
    T, H, Hkv, D = 90, 4, 2, 128
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(T, h, D, generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    cos, sin = (t.cuda() for t in R.tables(MAX_POS, D))
    pos = torch.randint(0, MAX_POS, (3, T), generator=g, dtype=torch.int32).cuda()
    kp, vp = (torch.zeros(6, Hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for axes in (axes_of("sections", D, 3), axes_of("in turn", D, 3)):
        for inter in (False, True):
            k_out = torch.empty_like(k)
            a, b = fattn.cache_append(k, v, kp, vp, torch.arange(T).cuda(), pos=pos, cos=cos, sin=sin, axes=axes, q=q,
                                      k_out=k_out, interleaved=inter)
            c, d = fattn.rotate(q.transpose(0, 1)[None], pos[:, None].contiguous(), cos, sin, axes=axes, interleaved=inter,
                                k=k.transpose(0, 1)[None])
            ok()
            assert torch.equal(a, c[0].transpose(0, 1)) and torch.equal(b, d[0].transpose(0, 1))


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,D,rot,A,kind,T", [("bf16", 128, 128, 3, "sections", 70), ("fp16", 64, 64, 2, "in turn", 700),
                                                  ("fp16", 128, 64, 3, "in turn", 1), ("bf16", 64, 16, 4, "in turn", 33)])
def test_append_with_axes(dtype, D, rot, A, kind, T, interleaved, kv4):
    """One axis of equal positions gives the form without axes bit for bit; several, the 64-bit form."""
    dt, H, Hkv, page = DT[dtype], 4, 2, 16
    g = torch.Generator().manual_seed(T + D)
    q, k, v = (torch.randn(T, h, D, generator=g).to(dt).cuda() for h in (H, Hkv, Hkv))
    cos, sin = R.tables(MAX_POS, rot)
    axes = axes_of(kind, rot, A)
    pos = torch.randint(0, MAX_POS, (A, T), generator=g, dtype=torch.int32)
    pages = T // page + 2
    slots = torch.randperm(pages * page, generator=g)[:T].cuda()

    def run(pos, axes):
        k_out = torch.empty_like(k)
        kw = dict(pos=pos.contiguous().cuda(), cos=cos.cuda(), sin=sin.cuda(), interleaved=interleaved, q=q, k_out=k_out, axes=axes)
        if not kv4:
            pool = [torch.zeros(pages, Hkv, page, D, dtype=dt, device="cuda") for _ in range(2)]
            q_out, _ = fattn.cache_append(k, v, *pool, slots, **kw)
        else:
            pool = []
            for _ in range(2):
                pool += [torch.zeros(pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda"),
                         torch.zeros(pages, Hkv, page, D // 32, 2, dtype=torch.float16, device="cuda")]
            q_out, _, _ = fattn.cache_append_kv4(k, v, *pool, slots, held=False, **kw)
        ok()
        return [q_out, k_out] + pool
    same = run(pos[:1].expand(A, -1), axes)
    plain = run(pos[0], None)
    assert all(torch.equal(a, b) for a, b in zip(same, plain))
    got = run(pos, axes)
    for x, src in ((got[0], q), (got[1], k)):
        y, mag = M.rotated(src.cpu().transpose(0, 1)[None], pos[:, None], axes, cos, sin, interleaved)
        R.check(x.cpu().transpose(0, 1)[None], y, R.rotated_bound(y, mag, dt), "append")
    at = slots.cpu()
    if not kv4:
        assert torch.equal(got[2][at // page, :, at % page], got[1]) and torch.equal(got[3][at // page, :, at % page], v)
    else:  # codes stand for the turned row within half a step (and the scale's own rounding)
        y, mag = M.rotated(k.cpu().transpose(0, 1)[None], pos[:, None], axes, cos, sin, interleaved)
        y = y[0].transpose(0, 1)
        sc = got[3].cpu()[at // page, :, at % page].double()
        held = R.held(got[2].cpu()[at // page, :, at % page], got[3].cpu()[at // page, :, at % page], "k")
        step = sc[..., 0].repeat_interleave(32, -1)
        # half a step, zero and 15 scales off by their fp16 roundings, fp32 roundings of the pair
        off = 0.5 * step + 2.0 ** -11 * (15 * step + sc[..., 1].abs().repeat_interleave(32, -1)) + 2.0 ** -20 * (1 + mag[0].transpose(0, 1))
        R.check(held, y, off, "codes")


@pytest.mark.parametrize("bad", [-1, MAX_POS])
def test_positions_out_of_range(bad):
    """On any axis: the token's rows are left as they were, and it is reported."""
    g = torch.Generator().manual_seed(3)
    D, N = 64, 50
    cos, sin = (t.cuda() for t in R.tables(MAX_POS, D))
    q = torch.randn(1, 3, N, D, generator=g).half().cuda()
    axes = axes_of("sections", D, 3)
    for ax in range(3):
        pos = torch.randint(0, MAX_POS, (3, 1, N), generator=g, dtype=torch.int32).cuda()
        want, _ = fattn.rotate(q, pos, cos, sin, axes=axes)
        ok()
        pos[ax, 0, 17] = bad
        out = torch.full_like(q, 7.0)
        fattn.rotate(q, pos, cos, sin, axes=axes, q_out=out)
        torch.cuda.synchronize()
        assert fattn.get_device_status() == 1
        keep = torch.arange(N) != 17
        assert (out[:, :, 17] == 7).all() and torch.equal(out[:, :, keep], want[:, :, keep])
        k, v = (torch.randn(N, 2, D, generator=g).half().cuda() for _ in range(2))
        kp, vp = (torch.full((4, 2, 16, D), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
        fattn.cache_append(k, v, kp, vp, torch.arange(N).cuda(), pos=pos[:, 0].contiguous(), cos=cos, sin=sin, axes=axes)
        torch.cuda.synchronize()
        assert fattn.get_device_status() == 1
        assert (kp[1, :, 1] == 7).all() and (vp[1, :, 1] == 7).all() and torch.equal(vp[1, :, 2], v[18])


def test_the_gradient():
    """sum(g * rotate(q)) moves with q as rotate(g, inverse) says: the adjoint, in 64 bits from the 16-bit outputs."""
    g = torch.Generator().manual_seed(4)
    D, N = 128, 40
    cos, sin = R.tables(MAX_POS, D)
    axes = axes_of("in turn", D, 3)
    pos = torch.randint(0, MAX_POS, (3, 1, N), generator=g, dtype=torch.int32)
    q, up = (torch.randn(1, 2, N, D, generator=g).half() for _ in range(2))
    a, _ = fattn.rotate(q.cuda(), pos.cuda(), cos.cuda(), sin.cuda(), axes=axes)
    b, _ = fattn.rotate(up.cuda(), pos.cuda(), cos.cuda(), sin.cuda(), axes=axes, inverse=True)
    ok()
    left, right = (up.double() * a.cpu().double()).sum(-1), (b.cpu().double() * q.double()).sum(-1)
    # each output element is off by half a unit of its last place (and a few of fp32's)
    bound = 1.01 * 2.0 ** -11 * ((up.double() * a.cpu().double()).abs().sum(-1) + (b.cpu().double() * q.double()).abs().sum(-1)) + 1e-6
    assert ((left - right).abs() <= bound).all()


def test_training_step_on_a_graph():
    """rotate, fwd, bwd and rotate's gradient captured as one graph, replayed on other inputs."""
    B, H, Hkv, N, D = 2, 4, 2, 130, 64
    g = torch.Generator().manual_seed(5)
    cos, sin = (t.cuda() for t in R.tables(MAX_POS, D))
    axes = axes_of("sections", D, 3)
    x = torch.randn(B, N, H + 2 * Hkv, D, generator=g).half().cuda()
    pos = torch.randint(0, MAX_POS, (3, B, N), generator=g, dtype=torch.int32).cuda()
    do = torch.randn(B, H, N, D, generator=g).half().cuda()
    grad = torch.zeros_like(x)

    def step(grad):
        q, k = fattn.rotate(x[:, :, :H].transpose(1, 2), pos, cos, sin, axes=axes, k=x[:, :, H:H + Hkv].transpose(1, 2))
        v = x[:, :, H + Hkv:].transpose(1, 2).contiguous()
        o, lse = fattn.fwd(q, k, v, causal=True)
        dq, dk, dv = fattn.bwd(q, k, v, o, lse, do, causal=True)
        fattn.rotate(dq, pos, cos, sin, axes=axes, inverse=True, k=dk, q_out=grad[:, :, :H].transpose(1, 2),
                     k_out=grad[:, :, H:H + Hkv].transpose(1, 2))
        grad[:, :, H + Hkv:] = dv.transpose(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(grad)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(grad)
    for seed in (6, 7):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(x.shape, generator=g).half())
        pos.copy_(torch.randint(0, MAX_POS, pos.shape, generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.zeros_like(x)
        step(want)
        ok()
        assert torch.equal(grad, want) and torch.isfinite(grad).all() and (grad != 0).any()


def test_tensors_past_32_bits():
    """17 million tokens (4.4 GB of q): the first and the last rows."""
    N, D = 17_000_001, 128
    q = torch.zeros(1, 1, N, D, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(6)
    rows = [0, 1, 2 ** 24 - 1, 2 ** 24, N - 2, N - 1]
    q[0, 0, rows] = torch.randn(len(rows), D, generator=g).to(torch.bfloat16).cuda()
    cos, sin = R.tables(MAX_POS, D)
    pos = torch.randint(0, MAX_POS, (3, 1, N), generator=g, dtype=torch.int32)
    axes = axes_of("sections", D, 3)
    got, _ = fattn.rotate(q, pos.cuda(), cos.cuda(), sin.cuda(), axes=axes)
    ok()
    y, mag = M.rotated(q[:, :, rows].cpu(), pos[:, :, rows], axes, cos, sin, False)
    R.check(got[:, :, rows], y, R.rotated_bound(y, mag, torch.bfloat16), "far rows")
    assert (got[0, 0, 2:2 ** 24 - 1] == 0).all() and (got[0, 0, 2 ** 24 + 1:N - 2] == 0).all()


def test_refusals_of_the_binding():
    D = 64
    q, k = (torch.randn(2, h, 9, D, device="cuda").half() for h in (4, 2))
    cos, sin = (t.cuda() for t in R.tables(MAX_POS, D))
    pos = torch.zeros(3, 2, 9, dtype=torch.int32, device="cuda")
    axes = axes_of("in turn", D, 3)
    good = dict(q=q, pos=pos, cos=cos, sin=sin, axes=axes, k=k)
    fattn.rotate(**good)
    for bad in (dict(q=q.float()), dict(pos=pos[0]), dict(pos=pos.long()), dict(axes=axes[:-1]), dict(cos=cos.double()),
                dict(sin=sin[:, :-1]), dict(k=k[:, :, :-1]), dict(q_out=q[:, :, :-1]), dict(pos=pos[:0]), dict(axes=None)):
        with pytest.raises((ValueError, fattn.FattnError)):
            fattn.rotate(**dict(good, **bad))
    with pytest.raises(fattn.FattnError):      # a pair on an axis that pos does not have
        fattn.rotate(**dict(good, axes=bytes([3]) * 32))
    with pytest.raises((ValueError, TypeError)):
        fattn.rotate(**dict(good, axes="0" * 32))
    with pytest.raises((ValueError, TypeError)):
        fattn.rotate(**dict(good, axes=[300] * 32))
    kp = torch.zeros(2, 2, 16, D, dtype=torch.float16, device="cuda")
    rows = dict(k=k[0].transpose(0, 1), v=k[1].transpose(0, 1), k_pages=kp, v_pages=kp.clone(), slots=torch.arange(9).cuda(), cos=cos,
                sin=sin)
    fattn.cache_append(**rows, pos=pos[:, 0].contiguous(), axes=axes)
    for bad in (dict(pos=pos[0, 0], axes=axes), dict(pos=pos[:, 0].contiguous()), dict(pos=pos[:, 0].contiguous(), axes=axes[1:])):
        with pytest.raises(ValueError):
            fattn.cache_append(**rows, **bad)
    ok()
