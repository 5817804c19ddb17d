"""Refusals of the serving entry points, all before any CUDA call, and the
layout the header documents for 4-bit rows."""
import ctypes
import os

import pytest
import torch

import tiled_attention_forward_gb300 as fattn
from tests import serving_ref as R

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA_ERR, TIMEOUT, NO_DEVICE = range(7)
A = 1 << 40  # far-apart fake device addresses, never dereferenced
READY = NO_DEVICE if not torch.cuda.is_available() else None


def i64s(*x):
    return (ctypes.c_int64 * len(x))(*x)


def call_append(kv4=False, q=A, k=2 * A, v=3 * A, q_out=4 * A, k_out=5 * A, v_out=None, kp=6 * A, vp=7 * A,
                ks=8 * A, vs=9 * A, strides=None, page_stride=None, P=4, ps=16, slots=10 * A, pos=11 * A, cos=12 * A,
                sin=13 * A, max_pos=64, rot=None, T=3, H=4, Hkv=2, D=64, dtype=2):
    lib = fattn.load()
    rot = D if rot is None else rot
    st = strides or [H * D, D, Hkv * D, D, Hkv * D, D, H * D, D, Hkv * D, D, Hkv * D, D]
    if kv4:
        return lib.fattn_cache_append_kv4(q, k, v, q_out, k_out, v_out, i64s(*st), kp, ks, vp, vs, P, ps, slots, pos,
                                          cos, sin, max_pos, rot, 0, 0, T, H, Hkv, D, dtype, None)
    page_stride = Hkv * ps * D if page_stride is None else page_stride
    return lib.fattn_cache_append(q, k, v, q_out, k_out, i64s(*st[:10]), kp, vp, page_stride, P, ps, slots, pos, cos,
                                  sin, max_pos, rot, 0, T, H, Hkv, D, dtype, None)


@pytest.mark.parametrize("kv4", [False, True])
def test_append_refusals(kv4):
    def call(**kw):
        return call_append(kv4, **kw)
    assert call(dtype=0) == UNSUPPORTED and call(dtype=9) == INVALID
    assert call(D=96) == UNSUPPORTED and call(D=-64) == INVALID
    assert call(ps=24) == UNSUPPORTED and call(ps=0) == INVALID and call(ps=1 << 17) == UNSUPPORTED
    assert call(P=-1) == INVALID and call(P=1 << 31) == UNSUPPORTED
    assert call(Hkv=0) == INVALID and call(T=-1) == INVALID
    assert call(rot=8) == UNSUPPORTED and call(rot=80) == INVALID and call(rot=-16) == INVALID
    assert call(T=0) == OK
    for name in ("k", "v", "kp", "vp", "slots", "pos", "cos", "sin"):
        assert call(**{name: None}) == INVALID, name
    assert call(q=None) == INVALID and call(q_out=None) == INVALID    # one without the other
    for name in ("q", "k", "v", "q_out", "k_out", "kp", "vp", "cos", "sin"):
        good = dict(q=A, k=2 * A, v=3 * A, q_out=4 * A, k_out=5 * A, kp=6 * A, vp=7 * A, cos=12 * A, sin=13 * A)
        assert call(**{name: good[name] + 8}) == MISALIGNED, name
    assert call(slots=10 * A + 4) == MISALIGNED and call(pos=11 * A + 2) == MISALIGNED
    base = [256, 64, 128, 64, 128, 64, 256, 64, 128, 64, 128, 64]
    for i in range(10):
        for bad in (-8, 12):
            assert call(strides=base[:i] + [bad] + base[i + 1:]) == INVALID, i
    assert call(strides=base[:6] + [32, 64] + base[8:]) == INVALID     # q_out's rows run into one another
    assert call(strides=base[:6] + [128, 64] + base[8:]) == INVALID
    assert call(strides=base[:8] + [0, 64] + base[10:]) == INVALID
    # overlaps
    assert call(k_out=4 * A + 64) == INVALID        # k_out in q_out
    assert call(q_out=2 * A) == INVALID             # q_out over k
    assert call(q_out=A + 16) == INVALID            # q_out over q, not in place
    assert call(kp=2 * A) == INVALID and call(vp=6 * A) == INVALID
    assert call(k_out=7 * A) == INVALID and call(kp=10 * A) == INVALID and call(q_out=12 * A) == INVALID
    if kv4:
        assert call(ks=None) == INVALID and call(vs=None) == INVALID and call(ks=8 * A + 4) == MISALIGNED
        assert call(vs=8 * A) == INVALID and call(ks=6 * A + 64) == INVALID
        assert call(v_out=5 * A) == INVALID and call(v_out=15 * A, strides=base[:10] + [64, 64]) == INVALID
    else:
        assert call(page_stride=16) == INVALID and call(page_stride=4096 + 4) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("kv4", [False, True])
def test_append_accepts(kv4):
    def call(**kw):
        return call_append(kv4, **kw)
    assert call() == NO_DEVICE
    assert call(q=None, q_out=None) == NO_DEVICE and call(k_out=None) == NO_DEVICE
    assert call(q=None, q_out=None, H=-3) == NO_DEVICE               # H is ignored without q
    assert call(rot=0, pos=None, cos=None, sin=None) == NO_DEVICE
    # slices of one projection, q and k turned in place
    st = [512, 64] * 6
    assert call(q=A, k=A + 512, v=A + 768, q_out=A, k_out=A + 512, strides=st) == NO_DEVICE
    assert call(q=A, k=A + 512, v=A + 768, q_out=A + 16, strides=st) == INVALID
    assert call(q=A, k=A + 512, v=A + 640, q_out=4 * A, k_out=A + 512, strides=st) == INVALID  # k_out runs into v
    if not kv4:  # K and V pages in one tensor
        inner = 2 * 16 * 64
        assert call(vp=6 * A + 2 * inner, page_stride=2 * inner) == NO_DEVICE
        assert call(vp=6 * A + 2 * inner - 16, page_stride=2 * inner) == INVALID
        assert call(vp=6 * A + 2 * inner, page_stride=2 * inner - 8) == INVALID


def call_decode(kv4=False, q=A, o=2 * A, lse=3 * A, strides=None, kp=4 * A, vp=5 * A, ks=6 * A, vs=7 * A,
                page_stride=None, P=4, ps=16, table=8 * A, W=3, lens=9 * A, ws=10 * A, wsb=None, B=2, H=4, Hkv=2, Nq=1,
                D=64, scale=0.125, dtype=2):
    lib = fattn.load()
    st = i64s(*(strides or [H * Nq * D, Nq * D, D] * 2))
    wsb = lib.fattn_decode_workspace_bytes(B, H, Hkv, Nq, D) if wsb is None else wsb
    if kv4:
        return lib.fattn_decode_kv4(q, o, lse, st, kp, ks, vp, vs, P, ps, table, W, lens, ws, wsb, B, H, Hkv, Nq, D,
                                    scale, dtype, None)
    page_stride = Hkv * ps * D if page_stride is None else page_stride
    return lib.fattn_decode(q, o, lse, st, kp, vp, page_stride, P, ps, table, W, lens, ws, wsb, B, H, Hkv, Nq, D, scale,
                            dtype, None)


@pytest.mark.parametrize("kv4", [False, True])
def test_decode_refusals(kv4):
    def call(**kw):
        return call_decode(kv4, **kw)
    assert call(dtype=0) == UNSUPPORTED and call(dtype=-1) == INVALID and call(D=80) == UNSUPPORTED
    assert call(ps=8) == UNSUPPORTED and call(Hkv=0) == INVALID and call(Hkv=3) == INVALID and call(B=-1) == INVALID
    assert call(scale=float("nan")) == INVALID and call(scale=-1.0) == INVALID
    assert call(W=(1 << 27)) == UNSUPPORTED and call(W=-1) == INVALID
    assert call(B=0) == OK and call(Nq=0) == OK and call(H=0) == OK
    for name in ("q", "o", "kp", "vp", "table", "lens", "ws"):
        assert call(**{name: None}) == INVALID, name
    need = fattn.load().fattn_decode_workspace_bytes(2, 4, 2, 1, 64)
    assert need > 0 and call(wsb=need - 1) == INVALID
    for name, at in (("q", A), ("o", 2 * A), ("kp", 4 * A), ("vp", 5 * A), ("ws", 10 * A)):
        assert call(**{name: at + 8}) == MISALIGNED, name
    for name, at in (("lse", 3 * A), ("table", 8 * A), ("lens", 9 * A)):
        assert call(**{name: at + 2}) == MISALIGNED, name
    base = [256, 64, 64] * 2
    for i in range(6):
        for bad in (-64, 4):
            assert call(strides=base[:i] + [bad] + base[i + 1:]) == INVALID, i
    assert call(strides=base[:3] + [128, 64, 64]) == INVALID and call(strides=base[:3] + [256, 32, 64]) == INVALID
    assert call(o=A) == INVALID and call(o=4 * A) == INVALID and call(lse=2 * A) == INVALID
    assert call(ws=9 * A) == INVALID and call(ws=2 * A) == INVALID and call(lse=8 * A) == INVALID
    if kv4:
        assert call(ks=None) == INVALID and call(vs=None) == INVALID and call(vs=7 * A + 4) == MISALIGNED
        assert call(o=7 * A) == INVALID
    else:
        assert call(page_stride=100) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("kv4", [False, True])
def test_decode_accepts(kv4):
    def call(**kw):
        return call_decode(kv4, **kw)
    assert call() == NO_DEVICE and call(lse=None) == NO_DEVICE
    assert call(W=0, table=None) == NO_DEVICE           # no page at all: every row is empty
    assert call(strides=[256, 64, 0, 64, 128, 0]) == NO_DEVICE  # o head-major
    assert call(H=64, Hkv=1, Nq=8) == NO_DEVICE


def test_decode_workspace_bytes():
    ws = fattn.load().fattn_decode_workspace_bytes
    for bad in ((0, 1, 1, 1, 64), (1, 0, 1, 1, 64), (1, 3, 2, 1, 64), (1, 2, 2, 0, 64), (1, 2, 2, 1, 96),
                (1 << 31, 1, 1, 1, 64), (-1, 1, 1, 1, 64)):
        assert ws(*bad) == 0, bad
    assert ws(1, 8, 1, 1, 128) > 0 and fattn.decode_workspace_bytes(1, 8, 1, 128, Hkv=1) == ws(1, 8, 1, 1, 128)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nibble_order_is_a_permutation(D, which):
    n = R.nibble_index(D, which)
    assert sorted(n.tolist()) == list(range(D))
    codes = torch.randint(0, 16, (3, D))
    assert torch.equal(R.unpack(R.pack(codes, which), which), codes)


def test_binding_refuses_what_the_library_cannot_see():
    T, Hkv, D = 2, 1, 64
    x = torch.zeros(T, Hkv, D, dtype=torch.bfloat16)
    pages = torch.zeros(1, Hkv, 16, D, dtype=torch.bfloat16)
    slots = torch.arange(T)
    with pytest.raises(ValueError):
        fattn.cache_append(x, x, pages, pages.clone(), slots)      # not on a GPU
    with pytest.raises(ValueError):
        fattn.decode(x.view(T, Hkv, 1, D), pages, pages, slots[None].int(), slots.int())
    with pytest.raises(ValueError):
        fattn.decode_kv4(x, pages, pages, pages, pages, slots, slots)


def test_header_documents_the_entry_points():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fattn.h")).read()
    for name in ("fattn_cache_append(", "fattn_cache_append_kv4(", "fattn_decode(", "fattn_decode_kv4(",
                 "fattn_decode_workspace_bytes("):
        assert "FATTN_API" in text and name in text
    assert "32 i + 8 t + e at nibble 8 (t D/32 + i) + e/2 + 4 (e mod 2)" in text
    assert "16 j + 8 u + g at nibble (D/8) g + (D/16) u + j" in text


def call_packed(q=A, k=2 * A, v=3 * A, o=4 * A, lse=5 * A, strides=None, cu=6 * A, ws=7 * A, wsb=None, B=3, T=100, H=4,
                Hkv=2, D=64, scale=0.125, causal=1, dtype=2):
    lib = fattn.load()
    st = i64s(*(strides or [H * D, D, Hkv * D, D, Hkv * D, D, H * D, D]))
    wsb = lib.fattn_packed_workspace_bytes(B, T) if wsb is None else wsb
    return lib.fattn_fwd_packed(q, k, v, o, lse, st, cu, ws, wsb, B, T, H, Hkv, D, scale, causal, dtype, None)


def test_packed_refusals():
    call = call_packed
    assert call(dtype=0) == UNSUPPORTED and call(dtype=3) == INVALID and call(D=32) == UNSUPPORTED
    assert call(B=-1) == INVALID and call(T=-1) == INVALID and call(Hkv=3) == INVALID and call(Hkv=0) == INVALID
    assert call(scale=float("inf")) == INVALID and call(scale=-0.5) == INVALID
    assert call(B=0) == OK and call(T=0) == OK and call(H=0) == OK
    for name in ("q", "k", "v", "o", "cu", "ws"):
        assert call(**{name: None}) == INVALID, name
    assert call(wsb=fattn.packed_workspace_bytes(3, 100) - 1) == INVALID
    for name, at in (("q", A), ("k", 2 * A), ("v", 3 * A), ("o", 4 * A), ("ws", 7 * A)):
        assert call(**{name: at + 8}) == MISALIGNED, name
    assert call(lse=5 * A + 2) == MISALIGNED and call(cu=6 * A + 1) == MISALIGNED
    base = [256, 64, 128, 64, 128, 64, 256, 64]
    for i in range(8):
        for bad in (-64, 4, 0):
            assert call(strides=base[:i] + [bad] + base[i + 1:]) == INVALID, i
    assert call(strides=base[:6] + [128, 64]) == INVALID   # o's rows run into one another
    assert call(strides=[1 << 39] + base[1:]) == UNSUPPORTED
    assert call(o=A) == INVALID and call(o=3 * A + 128) == INVALID and call(lse=4 * A) == INVALID
    assert call(ws=6 * A) == INVALID and call(ws=2 * A) == INVALID and call(lse=7 * A) == INVALID
    far = dict(q=1 << 45, k=1 << 46, v=1 << 47, o=1 << 48, lse=1 << 49, cu=1 << 50, ws=1 << 51)
    assert call(T=1 << 30, H=1 << 9, **far) == UNSUPPORTED  # more than 2^30 tasks
    assert call(T=(1 << 30) + 1, **far) == UNSUPPORTED


def test_packed_workspace_bytes():
    ws = fattn.load().fattn_packed_workspace_bytes
    for B, T in ((1, 1), (3, 255), (64, 16384), (1, 256), (64, 255), (65, 255), (1, 64 * 256)):
        blocks = T // 256 + B
        assert ws(B, T) == (16 * (1 + blocks) if blocks > 64 else 160 * 16 * 65)
        # one list entry per Q block, however the tokens are dealt out
        assert T // 256 + B >= sum(-(-n // 256) for n in [T - (B - 1)] + [1] * (B - 1) if n > 0)
    for bad in ((0, 1), (1, 0), (-1, 5), (1 << 31, 1), (1, 1 << 31)):
        assert ws(*bad) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
def test_packed_accepts():
    call = call_packed
    assert call() == NO_DEVICE and call(lse=None) == NO_DEVICE
    # slices of one projection; head-major; a single token or head with any stride
    assert call(k=A + 512, v=A + 768, strides=[512, 64] * 3 + [256, 64]) == NO_DEVICE
    assert call(strides=[64, 6400] * 4) == NO_DEVICE
    assert call(T=1, H=1, Hkv=1, strides=[0] * 8) == NO_DEVICE
    # o in a slice of the tensor that q, k and v are slices of, beside them
    assert call(k=A + 512, v=A + 768, o=A + 1024, strides=[768, 64] * 4) == NO_DEVICE
    assert call(k=A + 512, v=A + 768, o=A + 1008, strides=[768, 64] * 4) == INVALID
