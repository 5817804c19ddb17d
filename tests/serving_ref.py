"""Plain 64-bit forms of the serving operators (CPU, torch float64) and the
error bounds their tests use, derived from the kernels' arithmetic:

  * a rounding to a 16-bit type is off by at most u = finfo(t).eps / 2 of the
    value, an fp32 operation by 2^-24;
  * rotation: two fp32 products and a sum of them, one rounding to the output
    type;
  * attention: scores are fp32 sums of D exact products (any order, each
    addition off by at most 2^-23 of the partial sum, so D * 2^-23 of the sum of
    magnitudes in all), P is rounded once to 16 bits before P.V, the
    normaliser is the fp32 sum of the unrounded P, the output is rounded once.
"""
import math

import numpy as np
import torch

GROUP = 32


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the spacing of the subnormal numbers of a type: the rounding near zero."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def tables(max_pos, rot, base=10000.0):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv[None]
    return ang.cos().float(), ang.sin().float()


def rotate(x, pos, cos, sin, interleaved):
    """(rotated x, sum of the two products' magnitudes), float64; x [T, h, D]."""
    x = x.double()
    rot = 2 * cos.shape[1]
    if rot == 0:
        return x.clone(), x.abs()
    c, s = cos.double()[pos.long()][:, None], sin.double()[pos.long()][:, None]
    y, mag = x.clone(), x.abs()
    if interleaved:
        ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        ia, ib = torch.arange(0, rot // 2), torch.arange(rot // 2, rot)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    mag[..., ia] = (a * c).abs() + (b * s).abs()
    mag[..., ib] = (b * c).abs() + (a * s).abs()
    return y, mag


def rotated_bound(y, mag, dtype):
    """Error of a rotated element: three fp32 roundings, then one to `dtype`."""
    fp32 = 3 * 2.0 ** -24 * mag
    return fp32 + u_of(dtype) * (y.abs() + fp32) + tiny(dtype)


def nibble_index(D, which):
    d = np.arange(D)
    if which == "k":
        return 8 * ((d % 32) // 8 * (D // 32) + d // 32) + (d % 8) // 2 + 4 * (d % 2)
    return (D // 8) * (d % 8) + (D // 16) * (d % 16 // 8) + d // 16


def unpack(codes, which):
    """codes uint8 [..., D/2] -> integer codes [..., D] in the order of the elements."""
    D = codes.shape[-1] * 2
    n = torch.as_tensor(nibble_index(D, which))
    b = codes.long()[..., n // 2]
    return (b >> (4 * (n % 2))) & 15


def pack(codes, which):
    """The inverse of unpack."""
    D = codes.shape[-1]
    n = torch.as_tensor(nibble_index(D, which))
    nib = torch.zeros_like(codes.long())
    nib[..., n] = codes.long()
    return (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8)


def held(codes, scales, which):
    """The values that a 4-bit row stands for, float64."""
    sc = scales.double().repeat_interleave(GROUP, dim=-2)
    return unpack(codes, which).double() * sc[..., 0] + sc[..., 1]


def gather(pages, table_row, n):
    """Rows 0..n-1 of a sequence from pages [P, Hkv, ps, X...] -> [Hkv, n, X...]."""
    ps = pages.shape[2]
    j = torch.arange(n)
    return pages[table_row.long()[j // ps], :, j % ps].transpose(0, 1)


def attend(q, k, v, scale, ends):
    """q [H, M, D], k, v [Hkv, n, D] float64; row m sees keys < ends[m].
    Returns O, LSE, sum p|v| / l and the largest sum of |q k| scale over visible keys."""
    H, M, D = q.shape
    share = H // k.shape[0]
    n = k.shape[1]
    kk, vv = k.repeat_interleave(share, 0), v.repeat_interleave(share, 0)
    s = torch.einsum("hmd,hnd->hmn", q, kk) * scale
    mag = torch.einsum("hmd,hnd->hmn", q.abs(), kk.abs()) * abs(scale)
    seen = torch.arange(n)[None, :] < torch.as_tensor(ends)[:, None]
    s = torch.where(seen, s, -math.inf)
    mag = torch.where(seen, mag, 0.0)
    lse = torch.logsumexp(s, -1) if n else torch.full((H, M), -math.inf, dtype=torch.float64)
    p = torch.where(seen, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[..., None]), 0.0)
    seen_v = torch.where(seen.any(0)[None, :, None], vv, 0.0)  # what no row sees may hold anything
    o = torch.einsum("hmn,hnd->hmd", p, seen_v)
    av = torch.einsum("hmn,hnd->hmd", p, seen_v.abs())
    worst = mag.amax(-1) if n else torch.zeros(H, M, dtype=torch.float64)
    return o, lse, av, worst


def attend_bounds(o, lse, av, worst, D, dtype, u_p, v_err=0.0):
    """(bound of O, bound of LSE).  The score of a key is off by at most
    ds = D 2^-23 worst (the sum) + 2^-23 worst (scale) in natural-log units;
    each exponential by ds and a few fp32 roundings (2^-20 in all, with the
    running sums); P by its rounding u_p; V by v_err (an array like o: the
    weighted error of the values as the kernel takes them)."""
    ds = (D + 1) * 2.0 ** -23 * worst
    w = 2 * ds + 2.0 ** -20
    core = (u_p + w)[..., None] * av + v_err
    bound = core + u_of(dtype) * (o.abs() + core) + tiny(dtype)
    lb = ds + 2.0 ** -20 * (1 + lse.abs())
    return bound, lb


def check(got, ref, bound, what):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all(), what + ": not finite"
    over = ((got - ref).abs() / bound)
    assert (over <= 1).all(), "%s: %.3g of the bound (max error %.3g)" % (what, over.max(), (got - ref).abs().max())
