"""Plain 64-bit forms of cross attention's gradients, of attention behind a shared
prefix and of rotation by several axes (CPU, torch float64), and the error bounds
their tests use (derived as in serving_ref.py and parity.py)."""
import math

import torch

from tests import serving_ref as R


def cross(q, k, v, lens, scale):
    """O, LSE, sum p|v|, worst score magnitudes; q [B,H,Nq,D], k, v [B,Hkv,Nk,D] (any type)."""
    outs = []
    for b in range(q.shape[0]):
        n = int(lens[b])
        kk, vv = k[b, :, :n].double(), v[b, :, :n].double()
        outs.append(R.attend(q[b].double(), kk, vv, scale, [n] * q.shape[2]))
    return [torch.stack(x) for x in zip(*outs)]


def cross_grads(q, k, v, do, lens, scale):
    """(dq, dk, dv) of sum(do * O), float64, by the chain rule."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    B, H, Nq, D = q.shape
    share = H // k.shape[1]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(H):
            g = h // share
            p = torch.softmax(scale * q[b, h] @ k[b, g, :n].T, 1)
            dp = do[b, h] @ v[b, g, :n].T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            dq[b, h] = scale * ds @ k[b, g, :n]
            dk[b, g, :n] += scale * ds.T @ q[b, h]
            dv[b, g, :n] += p.T @ do[b, h]
    return dq, dk, dv


def half_ulp(x, dtype):
    return R.u_of(dtype) * x.abs() + R.tiny(dtype)


def cross_grad_bounds(q, k, v, do, lens, scale, dtype, grads):
    """Bounds of dq, dk, dv per element, from the kernels' arithmetic: P off by EPS
    (the forward's LSE, exp2.approx, and fp32 sums of products), P and dS rounded
    once to the type (u, and 2^-24 absolute: fp16's subnormal spacing), Delta from
    the 16-bit O (u sum |dO O|), the result rounded once."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    B, H, Nq, D = q.shape
    share, u = H // k.shape[1], R.u_of(dtype)
    eps = 1e-4 + (max(Nq * share, k.shape[2]) / 16.0 + 8.0) * 2.0 ** -24
    bq, bk, bv = (half_ulp(g, dtype) for g in grads)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(H):
            g = h // share
            kk, vv = k[b, g, :n], v[b, g, :n]
            p = torch.softmax(scale * q[b, h] @ kk.T, 1)
            dp = do[b, h] @ vv.T
            delta = (p * dp).sum(1, keepdim=True)
            doo = (do[b, h].abs() * (p @ vv).abs()).sum(1, keepdim=True)
            ds = p * (dp - delta)
            w = (1.05 * u + eps) * ds.abs() + p * (u * doo + eps * (dp.abs() + delta.abs())) + 2.0 ** -24
            bq[b, h] += scale * w @ kk.abs()
            bk[b, g, :n] += scale * w.T @ q[b, h].abs()
            bv[b, g, :n] += ((1.05 * u + eps) * p + 2.0 ** -24).T @ do[b, h].abs()
    return bq, bk, bv


def shared(q, k_prefix, v_prefix, k_own, v_own, scale):
    """One sequence: q [H, Nq, D]; prefix [Hkv, P, D] and own [Hkv, n, D] rows, float64."""
    Nq, P, n = q.shape[1], k_prefix.shape[1], k_own.shape[1]
    ends = [P + max(0, n - Nq + i + 1) for i in range(Nq)]
    return R.attend(q, torch.cat([k_prefix, k_own], 1), torch.cat([v_prefix, v_own], 1), scale, ends)


def rotated(x, pos, axis_of_pair, cos, sin, interleaved, inverse=False):
    """(rotated x, sum of the two products' magnitudes); x [B, H, N, D], pos [A, B, N]."""
    axis = torch.as_tensor(list(axis_of_pair), dtype=torch.long)
    half = len(axis)
    x = x.double()
    at = pos.long()[axis].movedim(0, -1)[:, None]             # [B, 1, N, rot/2]
    i = torch.arange(half)
    c, s = cos.double()[at, i], sin.double()[at, i]
    if inverse:
        s = -s
    ia, ib = (torch.arange(0, 2 * half, 2), torch.arange(1, 2 * half, 2)) if interleaved else \
        (torch.arange(half), torch.arange(half, 2 * half))
    y, mag = x.clone(), x.abs()
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia], mag[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return y, mag


def check_rows_without_keys(o, lse, lens):
    for b, n in enumerate(lens):
        if n == 0:
            assert (o[b] == 0).all() and (lse[b] == -math.inf).all()
