"""Refusals of cross attention, decode behind a shared prefix, rotate and the appends
with axes, all before any CUDA call; workspace sizes; the plain forms' gradients
against differences."""
import ctypes

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import more_ref as M

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA_ERR, TIMEOUT, NO_DEVICE = range(7)
A = 1 << 40  # far-apart fake device addresses, never dereferenced
no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")


def i64s(*x):
    return (ctypes.c_int64 * len(x))(*x)


def call_cross(q=A, k=2 * A, v=3 * A, o=4 * A, lse=5 * A, lens=6 * A, ws=7 * A, wsb=None, B=2, H=4, Hkv=2, Nq=40, Nk=300,
               D=64, scale=0.125, dtype=2, strides=None):
    lib = fattn.load()
    sq, sk = [H * Nq * D, Nq * D, D], [Hkv * Nk * D, Nk * D, D]
    st = strides or sq + sk + sk + sq
    wsb = lib.fattn_cross_workspace_bytes(B, H, Hkv, Nq, Nk, D) if wsb is None else wsb
    return lib.fattn_fwd_cross(q, k, v, o, lse, i64s(*st), lens, ws, wsb, B, H, Hkv, Nq, Nk, D, scale, dtype, None)


def call_bwd(q=A, k=2 * A, v=3 * A, o=4 * A, do=5 * A, lse=6 * A, dq=7 * A, dk=8 * A, dv=9 * A, lens=10 * A, ws=11 * A,
             wsb=None, B=2, H=4, Hkv=2, Nq=40, Nk=300, D=64, scale=0.125, dtype=2, strides=None):
    lib = fattn.load()
    sq, sk = [H * Nq * D, Nq * D, D], [Hkv * Nk * D, Nk * D, D]
    st = strides or sq + sk + sk + sq + sq + sq + sk + sk
    wsb = lib.fattn_bwd_cross_workspace_bytes(B, H, Hkv, Nq, Nk, D) if wsb is None else wsb
    return lib.fattn_bwd_cross(q, k, v, o, do, lse, dq, dk, dv, i64s(*st), lens, ws, wsb, B, H, Hkv, Nq, Nk, D, scale,
                               dtype, None)


@pytest.mark.parametrize("call,outs", [(call_cross, ("o",)), (call_bwd, ("dq", "dk", "dv"))])
def test_cross_refusals(call, outs):
    assert call(dtype=0) == UNSUPPORTED and call(dtype=5) == INVALID and call(D=96) == UNSUPPORTED
    for name in ("B", "H", "Nq", "Nk", "D"):
        assert call(**{name: -1}) == INVALID, name
    assert call(Hkv=0) == INVALID and call(Hkv=3) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=-0.5) == INVALID and call(scale=float("inf")) == INVALID
    assert call(B=0) == OK and call(H=0) == OK
    assert call(Nq=(1 << 30) + 1) == UNSUPPORTED and call(B=1 << 20, H=1 << 14) == UNSUPPORTED
    ptrs = ["q", "k", "v", "o", "ws"] + [x for x in outs if x != "o"] + (["do", "lse"] if call is call_bwd else [])
    import inspect
    d = {n: p.default for n, p in inspect.signature(call).parameters.items()}
    for name in ptrs:
        assert call(**{name: None}) == INVALID, name
        if name != "lse":
            assert call(**{name: d[name] + 8}) == MISALIGNED, name
    assert call(lse=d["lse"] + 2) == MISALIGNED and call(lens=d["lens"] + 1) == MISALIGNED
    assert call(wsb=0) == INVALID
    for name in outs:  # over every input, the lengths, the lse and the workspace
        for other in ("q", "k", "v", "lens", "lse", "ws") + (("o", "do") if call is call_bwd else ()):
            assert call(**{name: d[other]}) == INVALID, (name, other)
    assert call(ws=d["q"]) == INVALID and call(ws=d["lse"]) == INVALID
    sq, sk = [4 * 40 * 64, 40 * 64, 64], [2 * 300 * 64, 300 * 64, 64]
    base = sq + sk + sk + sq + ([] if call is call_cross else sq + sq + sk + sk)
    for i in range(len(base)):
        for bad in (-8, 12, 0):
            assert call(strides=base[:i] + [bad] + base[i + 1:]) == INVALID, (i, bad)
        assert call(strides=base[:i] + [1 << 40] + base[i + 1:]) == UNSUPPORTED, i
    first_out = 9 if call is call_cross else 15
    assert call(strides=base[:first_out] + [sq[0], 64, 64] + base[first_out + 3:]) == INVALID  # rows run into one another


@no_gpu
@pytest.mark.parametrize("call", [call_cross, call_bwd])
def test_cross_accepts(call):
    assert call() == NO_DEVICE and call(lens=None) == NO_DEVICE
    assert call(Nk=0, k=None, v=None, **({} if call is call_cross else dict(dk=None, dv=None))) == NO_DEVICE
    st = [300 * 8 * 64, 64, 8 * 64]  # k and v in one tensor of the states; strides of single entries are not looked at
    sq = [0, 40 * 64, 64]
    if call is call_cross:
        assert call(lse=None) == NO_DEVICE
        assert call(B=1, k=2 * A, v=2 * A + 256, strides=sq + [0] + st[1:] + [0] + st[1:] + sq) == NO_DEVICE
        assert call(Nq=1) == NO_DEVICE and call(Nq=0) == OK
        both = [40 * 8 * 64, 64, 8 * 64]  # o another slice of q's tensor
        assert call(o=A + 512, strides=both + st + st + both, k=2 * A, v=2 * A + 256) == NO_DEVICE
        assert call(o=A + 256, strides=both + st + st + both, k=2 * A, v=2 * A + 256) == INVALID
    else:
        dense = [4 * 40 * 64, 40 * 64, 64]
        args = dict(k=2 * A, v=2 * A + 256, dk=8 * A, dv=8 * A + 256, strides=dense + st + st + dense * 3 + st + st)
        assert call(**args) == NO_DEVICE
        assert call(**dict(args, dv=8 * A + 128)) == INVALID   # dv's slice runs into dk's
        assert call(Nq=0, q=None, o=None, do=None, lse=None, dq=None, ws=None) == NO_DEVICE


def call_shared(q=A, o=2 * A, lse=3 * A, strides=None, kp=4 * A, vp=5 * A, page_stride=None, P=9, ps=16, pt=6 * A, W0=4,
                pl=7 * A, table=8 * A, W=3, lens=9 * A, ws=10 * A, wsb=None, B=2, H=4, Hkv=2, Nq=1, D=64, scale=0.125,
                dtype=2):
    lib = fattn.load()
    st = i64s(*(strides or [H * Nq * D, Nq * D, D] * 2))
    wsb = lib.fattn_decode_shared_workspace_bytes(B, H, Hkv, Nq, D) if wsb is None else wsb
    page_stride = Hkv * ps * D if page_stride is None else page_stride
    return lib.fattn_decode_shared(q, o, lse, st, kp, vp, page_stride, P, ps, pt, W0, pl, table, W, lens, ws, wsb, B, H, Hkv,
                                   Nq, D, scale, dtype, None)


def test_shared_refusals():
    call = call_shared
    assert call(dtype=0) == UNSUPPORTED and call(D=32) == UNSUPPORTED and call(ps=24) == UNSUPPORTED and call(Hkv=3) == INVALID
    assert call(scale=-1.0) == INVALID and call(W0=-1) == INVALID and call(W0=1 << 28) == UNSUPPORTED
    assert call(W0=1 << 62) == UNSUPPORTED and call(P=0) == INVALID
    assert call(B=0) == OK and call(H=0) == OK and call(Nq=0) == OK
    for name in ("q", "o", "kp", "vp", "pt", "pl", "table", "lens", "ws"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=A + 8) == MISALIGNED and call(pt=6 * A + 2) == MISALIGNED and call(pl=7 * A + 1) == MISALIGNED
    assert call(wsb=fattn.decode_shared_workspace_bytes(2, 4, 1, 64, 2) - 1) == INVALID
    for other in (4 * A, 5 * A, 6 * A, 7 * A, 8 * A, 9 * A):  # the workspace, o and lse over an input
        assert call(ws=other) == INVALID and call(o=other) == INVALID and call(lse=other) == INVALID
    assert call(strides=[0, 64, 64, 256, 64, 64]) == INVALID     # q broadcast over the batch
    assert call(strides=[256, 64, 64, 0, 64, 64]) == INVALID


@no_gpu
def test_shared_accepts():
    assert call_shared() == NO_DEVICE and call_shared(lse=None) == NO_DEVICE
    assert call_shared(W0=0, pt=None, pl=None) == NO_DEVICE     # no prefix
    assert call_shared(W=0, table=None) == NO_DEVICE            # no tokens of their own
    assert call_shared(B=64, H=32, Hkv=8, Nq=2, D=128) == NO_DEVICE


def call_rotate(q=A, k=2 * A, qo=3 * A, ko=4 * A, strides=None, pos=5 * A, axes=None, n_axes=3, cos=6 * A, sin=7 * A,
                max_pos=100, rot=64, B=2, H=4, Hkv=2, N=10, D=64, dtype=2):
    sq, sk = [H * N * D, N * D, D], [Hkv * N * D, N * D, D]
    st = strides or sq + sk + sq + sk
    axes = bytes(i % 3 for i in range(32)) if axes is None else axes
    return fattn.load().fattn_rotate(q, k, qo, ko, i64s(*st), pos, axes, n_axes, cos, sin, max_pos, rot, 0, 0, B, H, Hkv, N, D,
                                     dtype, None)


def test_rotate_refusals():
    call = call_rotate
    assert call(dtype=0) == UNSUPPORTED and call(D=80, rot=16) == UNSUPPORTED and call(rot=24) == UNSUPPORTED
    assert call(rot=80) == INVALID and call(rot=-16) == INVALID and call(max_pos=-1) == INVALID
    assert call(n_axes=0) == INVALID and call(n_axes=9) == UNSUPPORTED
    assert call(n_axes=2) == INVALID                                   # a pair on the third of two axes
    for name in ("B", "H", "N"):
        assert call(**{name: -1}) == INVALID and call(**{name: 0}) == OK
    for name in ("q", "qo", "pos", "cos", "sin", "k", "ko"):
        assert call(**{name: None}) == INVALID, name
    for name, at in (("q", A), ("k", 2 * A), ("qo", 3 * A), ("ko", 4 * A), ("cos", 6 * A), ("sin", 7 * A)):
        assert call(**{name: at + 8}) == MISALIGNED, name
    assert call(pos=5 * A + 2) == MISALIGNED
    for other in (2 * A, 5 * A, 6 * A, 7 * A, 4 * A, A + 16):
        assert call(qo=other) == INVALID
    base = [2560, 640, 64, 1280, 640, 64] * 2
    for i in range(12):
        for bad in (-8, 4):
            assert call(strides=base[:i] + [bad] + base[i + 1:]) == INVALID
    assert call(strides=base[:6] + [2560, 0, 64] + base[9:]) == INVALID
    assert call(strides=[2560, 64, 256] + base[3:], qo=A) == INVALID    # over its input in another order


@no_gpu
def test_rotate_accepts():
    assert call_rotate() == NO_DEVICE and call_rotate(k=None, ko=None, Hkv=-7) == NO_DEVICE
    assert call_rotate(qo=A, ko=2 * A) == NO_DEVICE                     # in place
    assert call_rotate(rot=0, pos=None, cos=None, sin=None) == NO_DEVICE
    assert call_rotate(n_axes=1, axes=bytes(32)) == NO_DEVICE
    s = [10 * 8 * 64, 64, 8 * 64]                                       # slices of one projection, in place
    assert call_rotate(q=A, k=A + 512, qo=A, ko=A + 512, strides=s * 4) == NO_DEVICE
    assert call_rotate(q=A, k=A + 256, qo=A, ko=A + 512, strides=s * 4) == INVALID
    assert call_rotate(strides=[0, 0, 64] + [1280, 640, 64] + [2560, 640, 64, 1280, 640, 64]) == NO_DEVICE  # a broadcast input


@pytest.mark.parametrize("kv4", [False, True])
def test_append_axes_refusals(kv4):
    lib = fattn.load()

    def call(axes=bytes(i % 3 for i in range(32)), n=3, rot=64, pos=11 * A):
        st = i64s(*([256, 64, 128, 64, 128, 64, 256, 64, 128, 64, 128, 64][:12 if kv4 else 10]))
        if kv4:
            return lib.fattn_cache_append_kv4_axes(A, 2 * A, 3 * A, 4 * A, 5 * A, None, st, 6 * A, 8 * A, 7 * A, 9 * A, 4, 16,
                                                   10 * A, pos, axes, n, 12 * A, 13 * A, 64, rot, 0, 0, 3, 4, 2, 64, 2, None)
        return lib.fattn_cache_append_axes(A, 2 * A, 3 * A, 4 * A, 5 * A, st, 6 * A, 7 * A, 2048, 4, 16, 10 * A, pos, axes, n,
                                           12 * A, 13 * A, 64, rot, 0, 3, 4, 2, 64, 2, None)
    assert call(axes=None) == INVALID and call(n=0) == INVALID and call(n=-1) == INVALID and call(n=9) == UNSUPPORTED
    assert call(n=2) == INVALID and call(rot=24) == UNSUPPORTED and call(rot=80) == INVALID
    assert call(pos=None) == INVALID
    assert call(pos=6 * A - 12 * 3 + 12) == INVALID   # the table of three axes runs into the cache
    if not torch.cuda.is_available():
        assert call() == NO_DEVICE and call(n=8) == NO_DEVICE and call(rot=0, axes=None) == NO_DEVICE


def test_rotary_axes():
    a = fattn.rotary_axes((2, 3, 1))
    assert a == bytes([0, 0, 1, 1, 1, 2]) and fattn.rotary_axes((4,)) == bytes(4)


def test_workspace_sizes():
    """Enough for the parts of every launch, and bounded."""
    assert fattn.cross_workspace_bytes(0, 8, 1, 1, 64, 8) == 0 and fattn.cross_workspace_bytes(1, 8, 1, 1, 96, 8) == 0
    assert fattn.cross_workspace_bytes(2, 32, 8192, 4096, 128, 8) == 16           # enough tasks: no parts
    few = fattn.cross_workspace_bytes(24, 32, 1, 4096, 128, 8)
    assert few == fattn.decode_workspace_bytes(24, 32, 1, 128, 8)
    parts = fattn.cross_workspace_bytes(1, 16, 130, 8192, 64, 4)
    assert 5 * 128 * 4 * (64 + 2) * 4 < parts < 1 << 27
    assert fattn.decode_shared_workspace_bytes(0, 8, 1, 64, 8) == 0
    a = fattn.decode_shared_workspace_bytes(64, 32, 1, 128, 8)                    # 8 heads of 256 rows, 38 parts
    assert 8 * 256 * 38 * (4 * 128 + 8) < a < 1 << 27
    for B in (1, 3, 64, 1000):
        for H, Hkv in ((8, 1), (32, 8), (7, 7)):
            for Nq in (1, 2, 3, 60, 500):
                rows = B * H * Nq
                assert fattn.decode_shared_workspace_bytes(B, H, Nq, 64, Hkv) >= rows * 4 * 66
    assert fattn.bwd_cross_workspace_bytes(2, 8, 257, 777, 64, 2) >= 2 * 8 * 2 * 384 * 4


def test_plain_gradients_against_differences():
    """The 64-bit gradients that the GPU tests compare with are those of the 64-bit forward."""
    g = torch.Generator().manual_seed(0)
    q, k, v, do = (torch.randn(2, h, n, 8, generator=g, dtype=torch.float64) for h, n in ((4, 3), (2, 5), (2, 5), (4, 3)))
    lens, scale = [5, 2], 0.4
    grads = M.cross_grads(q, k, v, do, lens, scale)

    def loss(*x):
        return (M.cross(*x, lens, scale)[0] * do).sum()
    for i, (x, dx) in enumerate(zip((q, k, v), grads)):
        for _ in range(12):
            at = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in x.shape)
            e = torch.zeros_like(x)
            e[at] = 1e-5
            args = [q, k, v]
            up, down = list(args), list(args)
            up[i], down[i] = x + e, x - e
            diff = (loss(*up) - loss(*down)) / 2e-5
            assert abs(diff - dx[at]) <= 1e-8


def test_axes_are_a_list():
    """A number (of axes, of pairs) is no list of axes."""
    for bad in (3, 32, 64):
        with pytest.raises(TypeError):
            fattn.rotate(torch.zeros(1, 1, 1, 64).half(), None, None, None, axes=bad, q_out=torch.zeros(1, 1, 1, 64).half())
    assert fattn._axes([0, 1, 2]) == fattn._axes((0, 1, 2)) == fattn._axes(bytearray([0, 1, 2])) == bytes([0, 1, 2])
