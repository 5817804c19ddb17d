"""Decode attention behind a shared prefix (decode_shared) against a plain 64-bit
form, and its use in a server's steps."""
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


def make(B, H, Hkv, D, dt, page, prefix, lens, Nq, seed, spare=0, fill=math.nan, q_std=2.0):
    """A pool whose pages are dealt out at random; `fill` lies in every slot that holds no token."""
    g = torch.Generator().manual_seed(seed)
    shared = -(-prefix // page)
    need = [-(-n // page) for n in lens]
    pages = shared + sum(need) + 2
    perm = torch.randperm(pages, generator=g)
    kp, vp = (torch.full((pages, Hkv, page, D), fill, dtype=dt) for _ in range(2))
    table = torch.full((B, max(max(need), 1) + 1), -1, dtype=torch.int32)
    at = shared

    def put(rows, pages_of):
        for x, pool in zip(rows, (kp, vp)):
            for j in range(x.shape[1]):
                pool[pages_of[j // page], :, j % page] = x[:, j]
    rows = [[torch.randn(Hkv, n, D, generator=g).to(dt) for _ in range(2)] for n in [prefix] + list(lens)]
    put(rows[0], perm[:shared])
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        put(rows[1 + b], perm[at:at + n])
        at += n
    q = (torch.randn(B, H, Nq, D, generator=g) * q_std).to(dt)
    pt = torch.cat([perm[:shared].int(), torch.full((spare,), -1, dtype=torch.int32)])
    return dict(q=q.cuda(), k_pages=kp.cuda(), v_pages=vp.cuda(), prefix_table=pt.cuda(),
                prefix_len=torch.tensor([prefix], dtype=torch.int32).cuda(), block_table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32).cuda()), rows


def check(args, rows, scale, o, lse, what=""):
    q = args["q"].cpu()
    dt, D = q.dtype, q.shape[-1]
    pk, pv = (x.double() for x in rows[0])
    for b in range(q.shape[0]):
        ok_, ov = (x.double() for x in rows[1 + b])
        ro, rl, av, worst = M.shared(q[b].double(), pk, pv, ok_, ov, scale)
        # the weights are rounded once; in bf16 the prefix's part is divided by the sum of its rounded weights
        bo, bl = R.attend_bounds(ro, torch.where(torch.isinf(rl), 0.0, rl), av, worst, D, dt, 2 * R.u_of(dt))
        R.check(o[b], ro, bo, "%s O of %d" % (what, b))
        none = torch.isinf(rl)
        assert (lse[b].cpu()[none] == -math.inf).all()
        R.check(lse[b].cpu()[~none], rl[~none], bl[~none], "%s LSE of %d" % (what, b))


def spare_for(B, Hkv, D, page, once):
    """Unused entries behind the prefix's pages: so many that the prefix could be long enough to be read once for all."""
    return (170 << 20) // ((B - 1) * Hkv * 4 * D * page) + 1 if once and B > 1 else 2


CASES = [
    # B, H, Hkv, page, prefix, own lengths, Nq
    (1, 4, 2, 16, 1, [1], 1), (3, 8, 2, 16, 130, [5, 17, 1], 1), (2, 4, 1, 48, 257, [50, 0], 1), (4, 4, 4, 80, 128, [3, 90, 2, 1], 2),
    (5, 16, 4, 64, 1000, [1, 2, 64, 65, 129], 1), (3, 6, 2, 128, 700, [4, 300, 3], 3), (2, 8, 1, 32, 2500, [33, 700], 4),
    (70, 8, 2, 16, 300, [1 + i % 40 for i in range(70)], 1), (2, 2, 2, 16, 0, [20, 3], 1), (1, 8, 2, 64, 500, [200], 130),
    (3, 3, 1, 16, 90, [0, 0, 2], 2),
]


@pytest.mark.parametrize("once", [False, True])
@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 64), ("fp16", 128)])
def test_shared(dtype, D, case, once):
    """Read by every sequence for itself, and once for all (which the table's width decides)."""
    B, H, Hkv, page, prefix, lens, Nq = case
    args, rows = make(B, H, Hkv, D, DT[dtype], page, prefix, lens, Nq, prefix + B, spare=spare_for(B, Hkv, D, page, once))
    o, lse = fattn.decode_shared(**args)
    ok()
    check(args, rows, fattn._default_scale(D), o, lse, str(case))


@pytest.mark.parametrize("once", [False, True])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_as_decode_over_the_joined_tables(dtype, D, once):
    """A prefix of whole pages: decode with the prefix's pages in every table computes the same."""
    args, rows = make(6, 8, 2, D, DT[dtype], 32, 960, [1, 40, 200, 7, 32, 64], 2, 3, spare=spare_for(6, 2, D, 32, once))
    o, lse = fattn.decode_shared(**args)
    B = 6
    table = torch.cat([args["prefix_table"][None, :30].expand(B, -1), args["block_table"]], 1).contiguous()
    o2, lse2 = fattn.decode(args["q"], args["k_pages"], args["v_pages"], table, args["seq_lens"] + 960)
    ok()
    check(args, rows, fattn._default_scale(D), o, lse)
    check(args, rows, fattn._default_scale(D), o2, lse2)


def test_no_prefix_is_decode():
    args, rows = make(3, 4, 2, 64, torch.float16, 16, 0, [20, 3, 100], 1, 4)
    args["prefix_table"] = args["prefix_table"][:0]
    o, lse = fattn.decode_shared(**args)
    o2, lse2 = fattn.decode(args["q"], args["k_pages"], args["v_pages"], args["block_table"], args["seq_lens"])
    ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("once", [False, True])
def test_layouts_workspace_contents_and_repeats(once):
    """q and o by strides, K and V pages in one tensor, workspaces of any contents, no lse: the same bits."""
    args, rows = make(5, 8, 2, 128, torch.bfloat16, 16, 600, [1, 30, 2, 99, 16], 2, 5, fill=0.25,
                      spare=spare_for(5, 2, 128, 16, once))
    o, lse = fattn.decode_shared(**args)
    kv = torch.stack([args["k_pages"], args["v_pages"]], 1)
    q = torch.empty(5, 2, 11, 128, dtype=torch.bfloat16, device="cuda")
    q[:, :, 2:10] = args["q"].transpose(1, 2)
    out = torch.empty_like(q)
    need = fattn.decode_shared_workspace_bytes(5, 8, 2, 128, 2)
    for fill in (0, 255, 0x5b):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        more = dict(args, q=q[:, :, 2:10].transpose(1, 2), k_pages=kv[:, 0], v_pages=kv[:, 1])
        for _ in range(2):
            o2, l2 = fattn.decode_shared(**more, out=out[:, :, 2:10].transpose(1, 2), workspace=ws)
        ok()
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    o3, l3 = fattn.decode_shared(**args, return_lse=False)
    ok()
    assert torch.equal(o, o3) and l3 is None


def test_lengths_and_pages_out_of_range():
    args, rows = make(2, 4, 2, 64, torch.float16, 16, 160, [5, 9], 1, 6, fill=0.0)
    full = fattn.decode_shared(**args)
    ok()
    got = fattn.decode_shared(**dict(args, prefix_len=torch.tensor([161], dtype=torch.int32).cuda()))
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 1 and torch.equal(got[0], full[0]) and torch.equal(got[1], full[1])
    none = fattn.decode_shared(**dict(args, prefix_len=torch.tensor([0], dtype=torch.int32).cuda()))
    ok()
    got = fattn.decode_shared(**dict(args, prefix_len=torch.tensor([-3], dtype=torch.int32).cuda()))
    torch.cuda.synchronize()
    assert fattn.get_device_status() == 1 and torch.equal(got[0], none[0])
    for bad in (-1, -2, -2 ** 31, args["k_pages"].shape[0], 2 ** 31 - 1):  # its keys and values are zeros
        table = args["prefix_table"].clone()
        table[4] = bad
        got = fattn.decode_shared(**dict(args, prefix_table=table))
        torch.cuda.synchronize()
        assert fattn.get_device_status() == 1
        zeroed = [[x.clone() for x in rows[0]]] + rows[1:]
        for x in zeroed[0]:
            x[:, 64:80] = 0
        check(args, zeroed, 0.125, *got, "page %d" % bad)


def test_pages_of_a_long_prefix_out_of_range():
    """The same where the prefix's keys are read once, a tile and more behind the bad page."""
    args, rows = make(70, 8, 4, 64, torch.float16, 16, 2600, [3 + i % 7 for i in range(70)], 1, 8, fill=0.0)
    full = fattn.decode_shared(**args)
    ok()
    check(args, rows, 0.125, *full)
    for at, bad in ((0, -1), (9, -2 ** 31), (100, 10 ** 6), (162, -2)):
        table = args["prefix_table"].clone()
        table[at] = bad
        got = fattn.decode_shared(**dict(args, prefix_table=table))
        torch.cuda.synchronize()
        assert fattn.get_device_status() == 1
        zeroed = [[x.clone() for x in rows[0]]] + rows[1:]
        for x in zeroed[0]:
            x[:, 16 * at:16 * at + 16] = 0
        check(args, zeroed, 0.125, *got, "page %d of %d" % (bad, at))
    for n, want in ((2601, 2600), (-1, 0)):
        got = fattn.decode_shared(**dict(args, prefix_len=torch.tensor([n * 16 if n > 0 else n], dtype=torch.int32).cuda()))
        torch.cuda.synchronize()
        assert fattn.get_device_status() == 1
        assert want == 0 or got[0].isfinite().all()


@pytest.mark.parametrize("once", [False, True])
def test_long_pool(once):
    """Pages past 2^32 bytes of the pool."""
    D, Hkv, page = 128, 8, 128
    pages = 9000  # 2.4 GB each of K and V
    args, rows = make(2, 8, Hkv, D, torch.bfloat16, page, 300, [10, 140], 1, 7, spare=spare_for(2, Hkv, D, page, once))
    kp, vp = (torch.zeros(2 * pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = args["k_pages"].shape[0]
    kp[-n:], vp[-n:] = args["k_pages"], args["v_pages"]
    up = 2 * pages - n
    args = dict(args, k_pages=kp, v_pages=vp, prefix_table=args["prefix_table"] + up, block_table=args["block_table"] + up)
    o, lse = fattn.decode_shared(**args)
    ok()
    check(args, rows, fattn._default_scale(D), o, lse)


@pytest.mark.parametrize("once", [False, True])
def test_two_graphs_and_streams(once):
    """Two captured steps with workspaces of their own, replayed together with other lengths."""
    sets = [make(4, 8, 2, 64, torch.float16, 16, 400, [33, 33, 33, 33], 1, 20 + i, fill=0.5,
                 spare=spare_for(4, 2, 64, 16, once)) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs, spaces = [], [], []
    for (args, _), s in zip(sets, streams):
        ws = torch.empty(fattn.decode_shared_workspace_bytes(4, 8, 1, 64, 2), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(args["q"]), torch.empty(4, 8, 1, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            fattn.decode_shared(**args, out=out, lse=lse, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            fattn.decode_shared(**args, out=out, lse=lse, workspace=ws)
        graphs.append(g)
        outs.append((out, lse))
        spaces.append(ws)
    for lens, prefix in (([1, 2, 30, 4], 399), ([32, 3, 7, 20], 17), ([5, 5, 5, 5], 0)):
        for (args, _), _ in zip(sets, streams):
            args["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
            args["prefix_len"].fill_(prefix)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        ok()
        for (args, _), (out, lse) in zip(sets, outs):
            o2, l2 = fattn.decode_shared(**args)
            ok()
            assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_a_server_with_images_and_an_encoder(dtype, D):
    """The operators together: a prefix with an image (positions with three axes)
    and the requests' own tokens enter the cache, a step attends behind the shared
    prefix, and then over an encoder's states."""
    dt = DT[dtype]
    H, Hkv, page, P, B = 8, 2, 16, 200, 3
    g = torch.Generator().manual_seed(30)
    cos, sin = R.tables(512, D)
    axes = fattn.rotary_axes((D // 2 - 2 * (3 * D // 16), 3 * D // 16, 3 * D // 16))
    assert len(axes) == D // 2
    lens = [1, 18, 40]
    pages = 40
    kp, vp = (torch.full((pages, Hkv, page, D), math.nan, dtype=dt, device="cuda") for _ in range(2))
    perm = torch.randperm(pages, generator=g)
    shared = -(-P // page)
    need = [-(-n // page) for n in lens]
    table = torch.zeros(B, max(need), dtype=torch.int32)
    at = shared
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n].int()
        at += n
    n = torch.arange(P)
    pos = torch.stack([torch.where(n < 100, n, 100), torch.where(n < 100, n, 100 + (n - 100) // 10),
                       torch.where(n < 100, n, 100 + n % 10)]).int()

    def tokens(count):
        return [torch.randn(count, h, D, generator=g).to(dt) for h in (H, Hkv, Hkv)]

    def append(q, k, v, slots, pos):
        return fattn.cache_append(k.cuda(), v.cuda(), kp, vp, slots.cuda(), pos=pos.contiguous().cuda(), cos=cos.cuda(),
                                  sin=sin.cuda(), axes=axes, q=q.cuda())[0]

    def turned(x, pos):  # [T, h, D] -> the cache's values
        y, _ = M.rotated(x.transpose(0, 1)[None], pos[:, None], axes, cos, sin, False)
        return y[0].to(dt)  # [h, T, D]
    _, pk, pv = tokens(P)
    append(torch.zeros(P, H, D, dtype=dt), pk, pv, perm[n // page] * page + n % page, pos)
    rows = [[turned(pk, pos), pv.transpose(0, 1)]]
    q_rot, q_turned = [], []
    for b, m in enumerate(lens):
        i = torch.arange(m)
        q, k, v = tokens(m)
        p = (300 + i).int().expand(3, -1)
        out = append(q, k, v, table[b].long()[i // page] * page + i % page, p)
        q_rot.append(out[-1])
        rows.append([turned(k, p), v.transpose(0, 1)])
    args = dict(q=torch.stack(q_rot)[:, :, None], k_pages=kp, v_pages=vp, prefix_table=perm[:shared].int().cuda(),
                prefix_len=torch.tensor([P], dtype=torch.int32).cuda(), block_table=table.cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32).cuda())
    o, lse = fattn.decode_shared(**args)
    states = torch.randn(B, 77, 2 * Hkv, D, generator=g).to(dt).cuda()
    k, v = states[:, :, :Hkv].transpose(1, 2), states[:, :, Hkv:].transpose(1, 2)
    o2, lse2 = fattn.fwd_cross(o, k, v, torch.tensor([77, 0, 5], dtype=torch.int32).cuda())
    ok()
    # (the cache's own rounding against turned()'s: one unit in few elements)
    for mine, r in zip((kp, vp), zip(*[rows[0]])):
        held = R.gather(mine.cpu(), perm[:shared], P)
        assert (held.double() - r[0].double()).abs().max() <= 2 * R.u_of(dt) * r[0].abs().max() * 2
    real = [[R.gather(kp.cpu(), perm[:shared], P), R.gather(vp.cpu(), perm[:shared], P)]]
    real += [[R.gather(x.cpu(), table[b], m) for x in (kp, vp)] for b, m in enumerate(lens)]
    check(args, real, fattn._default_scale(D), o, lse)
    ro, rl, av, worst = M.cross(o.cpu(), k.cpu(), v.cpu(), [77, 0, 5], fattn._default_scale(D))
    bo, _ = R.attend_bounds(ro, torch.where(torch.isinf(rl), 0.0, rl), av, worst, D, dt, 2 * R.u_of(dt))
    R.check(o2, ro, bo, "cross")
