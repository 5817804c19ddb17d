"""Measured workloads of the operators for keys that are not the queries' own and
for positions with several axes: cross attention to an encoder's states (forward
and gradients), decode attention of a batch that shares a long prefix, rotation of
queries and keys by positions with several axes (and its gradient), and the same
rotation on the way into a paged cache.

Each case is one call of one operator on seeded data.  ``run`` computes it either
in a plain form (elementary torch operations in 32 bits) or, with ``own`` set,
through this package's entry points.  ``exact`` gives the same outputs from the
definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
MAX_POS = 1 << 15  # rows of the rotation tables


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One step of a decoder: every request's new token over its encoder's states.
        dict(name="cross_step", op="cross", dtype="bf16", B=24, H=32, Hkv=8, D=128, Nq=1, Nk=4096, ragged=True),
        # A few short target prompts over long encoder states (few rows, many keys).
        dict(name="cross_prompt", op="cross", dtype="fp16", B=3, H=16, Hkv=4, D=64, Nq=130, Nk=8192, ragged=True),
        # A training batch: long targets over padded encoder states, grouped heads.
        dict(name="cross_train", op="cross", dtype="bf16", B=2, H=32, Hkv=8, D=128, Nq=8192, Nk=4096, ragged=False),
        # The gradients of a small ragged batch (fine-tuning), and of a training batch.
        dict(name="cross_bwd_small", op="cross_bwd", dtype="fp16", B=2, H=8, Hkv=2, D=64, Nq=257, Nk=777, ragged=True),
        dict(name="cross_bwd_train", op="cross_bwd", dtype="bf16", B=4, H=16, Hkv=16, D=128, Nq=4096, Nk=2000,
             ragged=True),
        # A handful of requests behind one system prompt.
        dict(name="shared_small", op="shared", dtype="fp16", B=4, H=16, Hkv=4, D=64, Nq=1, prefix=2000, longest=100,
             page=16),
        # A busy server's step: all requests share a long instruction prompt.
        dict(name="shared_batch", op="shared", dtype="bf16", B=64, H=32, Hkv=8, D=128, Nq=1, prefix=16000, longest=1024,
             page=64),
        # Several answers to one very long document, two tokens a request (a drafted token is checked).
        dict(name="shared_long", op="shared", dtype="bf16", B=16, H=32, Hkv=8, D=128, Nq=2, prefix=120001, longest=300,
             page=128),
        # q and k of a training batch with images, from one projection into the layout that attention takes.
        dict(name="rotate_train", op="rotate", dtype="bf16", B=2, H=32, Hkv=8, D=128, N=8192, rot=128, axes=3,
             cyclic=False, interleaved=False, inverse=False),
        # Gradients of q and k, height and width positions of an image encoder, back into the projection's layout.
        dict(name="rotate_grad", op="rotate", dtype="fp16", B=4, H=16, Hkv=16, D=64, N=1000, rot=64, axes=2,
             cyclic=True, interleaved=True, inverse=True),
        # One decode step's new tokens, and a prompt with images, on their way into the cache.
        dict(name="append_axes_step", op="append", dtype="bf16", T=64, H=32, Hkv=8, D=128, rot=128, axes=3, cyclic=True,
             interleaved=False, page=64),
        dict(name="append_axes_prompt", op="append", dtype="bf16", T=16000, H=32, Hkv=8, D=128, rot=128, axes=3,
             cyclic=False, interleaved=False, page=64),
    ]


HEADS = [(8, 1), (8, 2), (16, 4), (16, 16), (32, 8), (32, 4)]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["cross", "cross", "cross_bwd", "shared", "shared", "rotate", "append"])
    H, Hkv = rng.choice(HEADS)
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), H=H, Hkv=Hkv, D=rng.choice([64, 128]))
    if op in ("cross", "cross_bwd"):
        # no more pairs of a query and a key than the largest listed case has
        pairs = 64 * 8192 * 4096 // 2 if op == "cross" else 64 * 4096 * 2000 // 2
        c["B"] = _log_int(rng, 1, 24)
        c["Nk"] = _log_int(rng, 1, 16000)
        c["Nq"] = _log_int(rng, 1, min(8192, max(1, pairs // (c["B"] * H * c["Nk"]))))
        c["ragged"] = rng.random() < 0.6
    elif op == "shared":
        c["B"] = _log_int(rng, 1, 64)
        c["Nq"] = rng.choice([1, 1, 1, 2, 3])
        c["prefix"] = _log_int(rng, 1, max(1, min(120000, 960000 // Hkv, (1 << 26) // (c["B"] * H * c["Nq"]))))
        c["longest"] = _log_int(rng, c["Nq"], 1500)
        c["page"] = rng.choice([16, 32, 48, 64, 128])
    else:
        c["rot"] = rng.choice([c["D"], c["D"], c["D"] // 2])
        c["axes"] = rng.choice([2, 3])
        c["cyclic"] = rng.random() < 0.5
        c["interleaved"] = rng.random() < 0.5
        if op == "rotate":
            c["B"] = _log_int(rng, 1, 8)
            c["N"] = _log_int(rng, 1, 16000 // c["B"])
            c["inverse"] = rng.random() < 0.5
        else:
            c["T"] = _log_int(rng, 1, 12000)
            c["page"] = rng.choice([16, 48, 64, 128])
    return c


def _lens(case):
    """Encoder states of each batch entry (a function of the case alone)."""
    if not case["ragged"]:
        return [case["Nk"]] * case["B"]
    r = random.Random(case["B"] * 1000003 + case["Nk"])
    return [case["Nk"]] + [r.randint(max(1, case["Nk"] // 4), case["Nk"]) for _ in range(case["B"] - 1)]


def _own_lens(case):
    """Cached tokens of each request behind the shared prefix."""
    r = random.Random(case["B"] * 1000003 + case["longest"])
    return [case["longest"]] + [r.randint(case["Nq"], case["longest"]) for _ in range(case["B"] - 1)]


def _axis_of_pair(case):
    """Which axis each of the rot/2 pairs of a row turns by: in sections, or in turn."""
    n, A = case["rot"] // 2, case["axes"]
    if case["cyclic"]:
        return [i % A for i in range(n)]
    each = 3 * n // (4 * (A - 1))  # the later axes; the first one has the rest
    return [max(0, 1 + (i - (n - each * (A - 1))) // each) if i >= n - each * (A - 1) else 0 for i in range(n)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _rotation_tables(rot, device):
    """cos and sin of pos * 10000^(-2 i / rot), formed in 64 bits, kept in 32."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    ang = torch.arange(MAX_POS, device=device, dtype=torch.float64)[:, None] * inv[None, :]
    return ang.cos().float(), ang.sin().float()


def _positions(axes, count, generator, device):
    """[axes, count]: text (the same on every axis), then an image of 32 columns, then text."""
    n = torch.arange(count, device=device)
    first = int(torch.randint(0, MAX_POS // 2, (1,), generator=generator, device=device))
    a, b = count // 5, count - count // 5
    image = (n >= a) & (n < b)
    text = first + torch.where(n < a, n, n - b + a + 64)
    grid = [(n - a) // 32, (n - a) % 32]
    own_axis = ([torch.zeros_like(n)] + grid)[3 - axes:]
    return torch.stack([torch.where(image, first + a + x, text) for x in own_axis]).clamp_(0, MAX_POS - 1).int()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    H, Hkv, D = case["H"], case["Hkv"], case["D"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    s = dict(case=dict(case), scale=1.0 / math.sqrt(D))
    if case["op"] in ("cross", "cross_bwd"):
        B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
        s["q"] = normal(B, Nq, H, D, std=2.0).transpose(1, 2)
        kv = normal(B, Nk, 2 * Hkv, D)  # one projection of the encoder's states; k and v are slices of it
        s["k"], s["v"] = kv[:, :, :Hkv].transpose(1, 2), kv[:, :, Hkv:].transpose(1, 2)
        s["kv_lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=dev)
        if case["op"] == "cross":
            s["out"] = torch.empty(B, Nq, H, D, dtype=dt, device=dev).transpose(1, 2)
            s["lse"] = torch.empty(B, H, Nq, dtype=torch.float32, device=dev)
            if own:
                import tiled_attention_forward_gb300 as fattn
                s["workspace"] = torch.empty(fattn.cross_workspace_bytes(B, H, Nq, Nk, D, Hkv), dtype=torch.uint8,
                                             device=dev)
            return s
        s["dout"] = normal(B, Nq, H, D).transpose(1, 2)
        s["o"], s["lse"] = _plain_cross(s)  # what the forward left
        s["dq"] = torch.empty(B, Nq, H, D, dtype=dt, device=dev).transpose(1, 2)
        dkv = torch.empty(B, Nk, 2 * Hkv, D, dtype=dt, device=dev)
        s["dk"], s["dv"] = dkv[:, :, :Hkv].transpose(1, 2), dkv[:, :, Hkv:].transpose(1, 2)
        if own:
            import tiled_attention_forward_gb300 as fattn
            s["workspace"] = torch.empty(fattn.bwd_cross_workspace_bytes(B, H, Nq, Nk, D, Hkv), dtype=torch.uint8, device=dev)
        return s
    if case["op"] == "shared":
        B, Nq, page, lens = case["B"], case["Nq"], case["page"], _own_lens(case)
        shared = -(-case["prefix"] // page)
        need = [-(-n // page) for n in lens]
        pages = shared + sum(need) + 2
        s["q"] = normal(B, H, Nq, D, std=3.0)
        perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        s["prefix_table"] = perm[:shared].clone()
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device=dev)
        table = torch.zeros(B, max(need), dtype=torch.int32, device=dev)
        at = shared
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        s["block_table"] = table
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        s["k_pages"] = normal(pages, Hkv, page, D)
        s["v_pages"] = normal(pages, Hkv, page, D)
        s["out"] = torch.empty(B, H, Nq, D, dtype=dt, device=dev)
        s["lse"] = torch.empty(B, H, Nq, dtype=torch.float32, device=dev)
        if own:
            import tiled_attention_forward_gb300 as fattn
            s["workspace"] = torch.empty(fattn.decode_shared_workspace_bytes(B, H, Nq, D, Hkv), dtype=torch.uint8,
                                         device=dev)
        return s
    s["cos"], s["sin"] = _rotation_tables(case["rot"], dev)
    s["axis_of_pair"] = torch.tensor(_axis_of_pair(case), device=dev)
    s["axes"] = bytes(_axis_of_pair(case))
    if case["op"] == "rotate":
        B, N, A = case["B"], case["N"], case["axes"]
        s["pos"] = torch.stack([_positions(A, N, g, dev) for _ in range(B)], 1).contiguous()
        qkv = normal(B, N, H + 2 * Hkv, D)  # [B, N, heads, D]: a projection's output, or its gradient
        dense_q, dense_k = normal(B, H, N, D), normal(B, Hkv, N, D)
        ends = [(qkv[:, :, :H].transpose(1, 2), dense_q), (qkv[:, :, H:H + Hkv].transpose(1, 2), dense_k)]
        (s["q"], s["q_out"]), (s["k"], s["k_out"]) = [e[::-1] if case["inverse"] else e for e in ends]
        return s
    T, page = case["T"], case["page"]
    pages = -(-T // page) + 3
    qkv = normal(T, H + 2 * Hkv, D)
    s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:])
    s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].contiguous()
    s["pos"] = _positions(case["axes"], T, g, dev).contiguous()
    s["q_out"] = torch.empty(T, H, D, dtype=dt, device=dev)
    s["k_pages"] = torch.zeros(pages, Hkv, page, D, dtype=dt, device=dev)
    s["v_pages"] = torch.zeros(pages, Hkv, page, D, dtype=dt, device=dev)
    return s


# ---------------------------------------------------------------------------
# The operators, through the framework or in their plain form
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"cross": _plain_cross, "cross_bwd": _plain_cross_bwd, "shared": _plain_shared, "rotate": _plain_rotate,
            "append": _plain_append}[op](s)


def _own(op, s):
    import tiled_attention_forward_gb300 as fattn
    c = s["case"]
    if op == "cross":
        return fattn.fwd_cross(s["q"], s["k"], s["v"], s["kv_lens"], scale=s["scale"], out=s["out"], lse=s["lse"],
                               workspace=s["workspace"])
    if op == "cross_bwd":
        return fattn.bwd_cross(s["q"], s["k"], s["v"], s["o"], s["lse"], s["dout"], s["kv_lens"], scale=s["scale"],
                               dq=s["dq"], dk=s["dk"], dv=s["dv"], workspace=s["workspace"])
    if op == "shared":
        return fattn.decode_shared(s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_len"],
                                   s["block_table"], s["seq_lens"], scale=s["scale"], out=s["out"], lse=s["lse"],
                                   workspace=s["workspace"])
    if op == "rotate":
        return fattn.rotate(s["q"], s["pos"], s["cos"], s["sin"], axes=s["axes"], interleaved=c["interleaved"],
                            inverse=c["inverse"], k=s["k"], q_out=s["q_out"], k_out=s["k_out"])
    q, _ = fattn.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], pos=s["pos"], cos=s["cos"],
                              sin=s["sin"], axes=s["axes"], interleaved=c["interleaved"], q=s["q"], q_out=s["q_out"])
    return q, s["k_pages"], s["v_pages"]


def _seen(s):
    """[B, 1, 1, Nk]: the keys that are encoder states and not padding."""
    Nk = s["k"].shape[2]
    return (torch.arange(Nk, device=s["k"].device)[None, :] < s["kv_lens"][:, None])[:, None, None, :]


def _grouped(x, Hkv):
    """[B, H, N, D] -> [B, Hkv, H/Hkv * N, D] in 32 bits."""
    B, H, N, D = x.shape
    return x.float().reshape(B, Hkv, H // Hkv * N, D)


def _plain_cross(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, H, Nq, D = q.shape
    p = torch.matmul(_grouped(q, k.shape[1]).mul_(s["scale"]), k.float().transpose(-1, -2))
    p.masked_fill_(~_seen(s), float("-inf"))
    m = p.amax(-1, keepdim=True)
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (torch.matmul(p, v.float()) / l).view(B, H, Nq, D)
    lse = (m + l.log()).view(B, H, Nq)
    if "out" not in s:
        return o.to(q.dtype), lse
    s["out"].copy_(o.to(q.dtype))
    s["lse"].copy_(lse)
    return s["out"], s["lse"]


def _plain_cross_bwd(s):
    q, k, v, dt = s["q"], s["k"], s["v"], s["q"].dtype
    B, H, Nq, D = q.shape
    Hkv = k.shape[1]
    qg, dog, kf, vf = _grouped(q, Hkv), _grouped(s["dout"], Hkv), k.float(), v.float()
    delta = (dog * _grouped(s["o"], Hkv)).sum(-1, keepdim=True)
    p = torch.matmul(qg, kf.transpose(-1, -2)).mul_(s["scale"]).sub_(s["lse"].view(B, Hkv, -1, 1))
    p.masked_fill_(~_seen(s), float("-inf")).exp_()
    dv = torch.matmul(p.transpose(-1, -2), dog)
    p.mul_(torch.matmul(dog, vf.transpose(-1, -2)).sub_(delta)).mul_(s["scale"])
    s["dq"].copy_(torch.matmul(p, kf).view(B, H, Nq, D).to(dt))
    s["dk"].copy_(torch.matmul(p.transpose(-1, -2), qg).to(dt))
    s["dv"].copy_(dv.to(dt))
    return s["dq"], s["dk"], s["dv"]


def _plain_shared(s):
    c = s["case"]
    B, H, Nq, D = s["q"].shape
    Hkv, P, W = c["Hkv"], c["prefix"], s["block_table"].shape[1] * c["page"]
    share = H // Hkv
    table, shared = s["block_table"].long(), s["prefix_table"].long()

    def prefix(pages):  # [Hkv, P, D]
        return pages[shared].transpose(0, 1).reshape(Hkv, -1, D)[:, :P].float()

    def cached(pages):  # [B, Hkv, W, D]
        return pages[table].transpose(1, 2).reshape(B, Hkv, W, D).float()

    q = s["q"].float().mul(s["scale"]).view(B, Hkv, share * Nq, D)
    a = torch.matmul(q.transpose(0, 1).reshape(Hkv, B * share * Nq, D), prefix(s["k_pages"]).transpose(-1, -2))
    j, i = torch.arange(W, device=q.device), torch.arange(Nq, device=q.device)
    hidden = j[None, None, :] > (s["seq_lens"][:, None].long() - Nq + i[None, :])[..., None]      # [B, Nq, W]
    b = torch.matmul(q, cached(s["k_pages"]).transpose(-1, -2)).view(B, Hkv, share, Nq, W)
    b.masked_fill_(hidden[:, None, None], float("-inf"))
    b = b.view(B, Hkv, share * Nq, W)
    m = torch.maximum(a.amax(-1).view(Hkv, B, share * Nq).transpose(0, 1), b.amax(-1))
    a.sub_(m.transpose(0, 1).reshape(Hkv, -1, 1)).exp_()
    b.sub_(m[..., None]).exp_()
    l = a.sum(-1).view(Hkv, B, share * Nq).transpose(0, 1) + b.sum(-1)
    v = cached(s["v_pages"]).masked_fill_(hidden.all(1)[:, None, :, None], 0.0)
    o = torch.matmul(a, prefix(s["v_pages"])).view(Hkv, B, share * Nq, D).transpose(0, 1) + torch.matmul(b, v)
    s["out"].copy_((o / l[..., None]).reshape(B, H, Nq, D).to(s["out"].dtype))
    s["lse"].copy_((m + l.log()).reshape(B, H, Nq))
    return s["out"], s["lse"]


def _turn(x, cos, sin, rot, interleaved):
    """The rotated rows in 32 bits; cos and sin have the shape of x but for its last dimension, rot/2."""
    y = x.float()
    at = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = y[..., at[0]], y[..., at[1]]
    y = y.clone() if y is x else y
    y[..., at[0]], y[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    return y.to(x.dtype)


def _angles(s):
    """cos and sin [..., rot/2] of positions [axes, ...]: pair i by the position on its axis."""
    at = s["pos"].long()[s["axis_of_pair"]].movedim(0, -1)   # [..., rot/2]
    i = torch.arange(at.shape[-1], device=at.device)
    return s["cos"][at, i], s["sin"][at, i]


def _plain_rotate(s):
    c = s["case"]
    cos, sin = (x[:, None] for x in _angles(s))  # [B, 1, N, rot/2]
    if c["inverse"]:
        sin = -sin
    s["q_out"].copy_(_turn(s["q"], cos, sin, c["rot"], c["interleaved"]))
    s["k_out"].copy_(_turn(s["k"], cos, sin, c["rot"], c["interleaved"]))
    return s["q_out"], s["k_out"]


def _plain_append(s):
    c = s["case"]
    cos, sin = (x[:, None] for x in _angles(s))  # [T, 1, rot/2]
    page, at = s["slots"] // c["page"], s["slots"] % c["page"]
    s["q_out"].copy_(_turn(s["q"], cos, sin, c["rot"], c["interleaved"]))
    s["k_pages"][page, :, at] = _turn(s["k"], cos, sin, c["rot"], c["interleaved"])
    s["v_pages"][page, :, at] = s["v"]
    return s["q_out"], s["k_pages"], s["v_pages"]


# ---------------------------------------------------------------------------
# The work of one call
# ---------------------------------------------------------------------------
def work(case):
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] in ("cross", "cross_bwd"):
        keys, rows = sum(_lens(case)), case["B"] * case["Nq"] * H
        q, kv = 2 * rows * D, 2 * keys * Hkv * D
        if case["op"] == "cross":
            return {"bytes": 2 * q + 2 * kv + 4 * rows, "flops": 4 * keys * case["Nq"] * H * D}
        out = 2 * 2 * case["B"] * case["Nk"] * Hkv * D  # dk and dv have rows for the padding too
        return {"bytes": 4 * q + 2 * kv + out + 4 * rows, "flops": 10 * keys * case["Nq"] * H * D}
    if case["op"] == "shared":
        keys, rows = sum(_own_lens(case)), case["B"] * H * case["Nq"]
        return {"bytes": 4 * (case["prefix"] + keys) * Hkv * D + rows * (4 * D + 4),
                "flops": 4 * rows * case["prefix"] * D + 4 * keys * H * case["Nq"] * D}
    if case["op"] == "rotate":
        tokens = case["B"] * case["N"]
        return {"bytes": tokens * (4 * D * (H + Hkv) + 4 * case["rot"] + 4 * case["axes"]),
                "flops": 3 * tokens * case["rot"] * (H + Hkv)}
    T = case["T"]
    return {"bytes": T * (4 * D * (H + 2 * Hkv) + 4 * case["rot"] + 4 * case["axes"] + 8),
            "flops": 3 * T * case["rot"] * (H + Hkv)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"cross": _exact_cross, "cross_bwd": _exact_cross_bwd, "shared": _exact_shared, "rotate": _exact_rotate,
            "append": _exact_append}[case["op"]](case, s)


def _exact_cross(case, s):
    B, H, Nq, D = s["q"].shape
    share = H // case["Hkv"]
    out = torch.zeros(B, H, Nq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, Nq, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(case)):
        for h in range(H):
            z = s["scale"] * torch.einsum("id,jd->ij", s["q"][b, h].double(), s["k"][b, h // share, :n].double())
            lse[b, h] = torch.logsumexp(z, 1)
            out[b, h] = torch.softmax(z, 1) @ s["v"][b, h // share, :n].double()
    return out, lse


def _exact_cross_bwd(case, s):
    """The chain rule with the forward's own o and lse, which the operator takes."""
    B, H, Nq, D = s["q"].shape
    share = H // case["Hkv"]
    dq = torch.zeros(B, H, Nq, D, dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(B, case["Hkv"], case["Nk"], D, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, n in enumerate(_lens(case)):
        for h in range(H):
            g = h // share
            q, do, o = (s[x][b, h].double() for x in ("q", "dout", "o"))
            k, v = s["k"][b, g, :n].double(), s["v"][b, g, :n].double()
            w = torch.exp(s["scale"] * (q @ k.T) - s["lse"][b, h].double()[:, None])
            dz = w * (do @ v.T - torch.einsum("id,id->i", do, o)[:, None])
            dq[b, h] = s["scale"] * (dz @ k)
            dk[b, g, :n] += s["scale"] * (dz.T @ q)
            dv[b, g, :n] += w.T @ do
    return dq, dk, dv


def _exact_shared(case, s):
    B, H, Nq, D = s["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    share = H // Hkv
    out = torch.zeros(B, H, Nq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, H, Nq, dtype=torch.float64, device="cuda")

    def rows(pages, table, n, kvh):
        j = torch.arange(n, device="cuda")
        return pages[table.long()[j // page], kvh, j % page].double()

    for kvh in range(Hkv):
        pk, pv = (rows(s[x], s["prefix_table"], case["prefix"], kvh) for x in ("k_pages", "v_pages"))
        heads = slice(kvh * share, (kvh + 1) * share)
        zp = s["scale"] * torch.einsum("bhid,nd->bhin", s["q"][:, heads].double(), pk)
        for b, n in enumerate(_own_lens(case)):
            ok, ov = (rows(s[x], s["block_table"][b], n, kvh) for x in ("k_pages", "v_pages"))
            zo = s["scale"] * torch.einsum("hid,nd->hin", s["q"][b, heads].double(), ok)
            zo = zo.masked_fill(torch.ones(Nq, n, dtype=torch.bool, device="cuda").triu(n - Nq + 1), -torch.inf)
            z = torch.cat([zp[b], zo], -1)
            e = torch.logsumexp(z, -1)
            lse[b, heads] = e
            out[b, heads] = torch.exp(z - e[..., None]) @ torch.cat([pv, ov])
    return out, lse


def _exact_turned(case, s, x):
    """Rows as complex numbers times the unit numbers of their pairs; x [tokens, heads, D] or [B, heads, N, D]."""
    r, axis = case["rot"], _axis_of_pair(case)
    unit = torch.stack([torch.complex(s["cos"][:, i].double(), s["sin"][:, i].double())[s["pos"][axis[i]].long()]
                        for i in range(r // 2)], -1)
    if case.get("inverse"):
        unit = unit.conj()
    unit = unit[:, None]  # heads
    x = x.double()
    if case["interleaved"]:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * unit
        turned = torch.stack([z.real, z.imag], -1).flatten(-2)
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * unit
        turned = torch.cat([z.real, z.imag], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _exact_rotate(case, s):
    return _exact_turned(case, s, s["q"]), _exact_turned(case, s, s["k"])


def _exact_append(case, s):
    pages = []
    for old, x in ((s["k_pages"], _exact_turned(case, s, s["k"])), (s["v_pages"], s["v"].double())):
        flat = old.double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
        flat[s["slots"]] = x
        pages.append(flat.view(old.shape[0], case["page"], case["Hkv"], case["D"]).transpose(1, 2).contiguous())
    return _exact_turned(case, s, s["q"]), pages[0], pages[1]
