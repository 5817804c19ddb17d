"""Measured workloads of the serving operators: attention over packed prompts,
appending keys and values to a paged cache (16-bit or 4-bit) with the position
rotation applied on the way, and attention of new tokens over such a cache.

Each case is one call of one operator on seeded data.  ``run`` computes it
either in a plain form (elementary torch operations in 32 bits or more) or, with
``own`` set, through this package's entry points.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32        # elements of a row of the 4-bit cache that share one scale and zero
FP16_MAX = 65504.0
MAX_POS = 1 << 17  # rows of the rotation tables


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # A handful of short requests prefilled together (latency counts).
        dict(name="packed_short", op="packed", dtype="fp16", H=16, Hkv=4, D=64, lens="1,17,64,128,90"),
        # A prefill batch of a server: ragged prompts, grouped heads, Q/K/V as slices of one projection.
        dict(name="packed_mixed", op="packed", dtype="bf16", H=32, Hkv=8, D=128,
             lens="4096,1,2900,513,128,1777,255,3500,64,1024,700,300,33,950,129,14"),
        # One long prompt (the N = 16000 of the causal benchmark workload) beside short ones.
        dict(name="packed_long", op="packed", dtype="bf16", H=32, Hkv=8, D=128, lens="200,16000,1,77"),
        # One decode step of 64 requests: their new tokens enter the cache.
        dict(name="append_step", op="append", dtype="bf16", H=32, Hkv=8, D=128, T=64, page=64, rot=128,
             interleaved=False),
        # A whole prompt batch enters the cache; rotation of half of each head, interleaved pairs.
        dict(name="append_prompt", op="append", dtype="fp16", H=16, Hkv=2, D=64, T=8191, page=16, rot=32,
             interleaved=True),
        # The same steps with the cache held in 4 bits.
        dict(name="append_kv4_step", op="append_kv4", dtype="fp16", H=16, Hkv=16, D=64, T=17, page=32, rot=64,
             interleaved=True),
        dict(name="append_kv4_prompt", op="append_kv4", dtype="bf16", H=32, Hkv=8, D=128, T=16000, page=64,
             rot=128, interleaved=False),
        # One request, short context: the smallest decode call.
        dict(name="decode_small", op="decode", dtype="fp16", H=16, Hkv=4, D=64, B=1, longest=777, ragged=False,
             Nq=1, page=16),
        # A decode step of a busy server over a 16-bit cache, contexts of very different lengths.
        dict(name="decode_batch", op="decode", dtype="bf16", H=32, Hkv=8, D=128, B=64, longest=8192, ragged=True,
             Nq=1, page=64),
        # Multi-query heads, two tokens a request (a drafted token is checked).
        dict(name="decode_kv4_small", op="decode_kv4", dtype="fp16", H=8, Hkv=1, D=64, B=3, longest=1000,
             ragged=True, Nq=2, page=32),
        # The busy server's step with the cache held in 4 bits.
        dict(name="decode_kv4_batch", op="decode_kv4", dtype="bf16", H=32, Hkv=8, D=128, B=64, longest=8192,
             ragged=True, Nq=1, page=64),
        # Few requests with very long contexts.
        dict(name="decode_kv4_long", op="decode_kv4", dtype="bf16", H=32, Hkv=8, D=128, B=3, longest=120001,
             ragged=False, Nq=1, page=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed", "append", "append_kv4", "decode", "decode_kv4"])
    H, Hkv = rng.choice([(8, 1), (16, 2), (16, 4), (16, 16), (24, 8), (32, 8), (32, 4), (32, 32)])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), H=H, Hkv=Hkv, D=rng.choice([64, 128]))
    if op == "packed":
        lens, room = [], 16000
        for _ in range(_log_int(rng, 1, 24)):
            n = _log_int(rng, 1, 8000)
            if n <= room:
                lens.append(n)
                room -= n
        c["lens"] = ",".join(str(n) for n in lens)
        return c
    c["page"] = rng.choice([16, 32, 48, 64, 128])
    if op in ("append", "append_kv4"):
        c["T"] = _log_int(rng, 1, 12000)
        c["rot"] = rng.choice([c["D"], c["D"] // 2, 16])
        c["interleaved"] = rng.random() < 0.5
        return c
    c["B"] = _log_int(rng, 1, 48)
    c["Nq"] = rng.choice([1, 1, 1, 2, 4])
    # no more cached tokens in all than the listed batch has
    c["longest"] = _log_int(rng, 1, max(1, min(100000, 240000 // c["B"] * 8 // Hkv)))
    c["ragged"] = rng.random() < 0.7
    return c


def _packed_lens(case):
    return [int(n) for n in case["lens"].split(",")]


def _contexts(case):
    """Cached tokens of each request (a function of the case alone)."""
    if not case["ragged"]:
        return [case["longest"]] * case["B"]
    r = random.Random(case["B"] * 1000003 + case["longest"])
    return [case["longest"]] + [max(case["Nq"], r.randint(1, case["longest"])) for _ in range(case["B"] - 1)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _rotation_tables(rot, device):
    """cos and sin of pos * 10000^(-2 i / rot), formed in 64 bits, kept in 32."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    ang = torch.arange(MAX_POS, device=device, dtype=torch.float64)[:, None] * inv[None, :]
    return ang.cos().float(), ang.sin().float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    H, Hkv, D = case["H"], case["Hkv"], case["D"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dt)

    s = dict(case=dict(case), scale=1.0 / math.sqrt(D))
    if case["op"] == "packed":
        lens = _packed_lens(case)
        T = sum(lens)
        qkv = normal(T, H + 2 * Hkv, D)  # one projection's output; q, k, v are slices of it
        qkv[:, :H] *= 2
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:], lens=lens,
                 out=torch.zeros(T, H, D, dtype=dt, device=dev),
                 lse=torch.zeros(H, T, dtype=torch.float32, device=dev))
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if own:
            import tiled_attention_forward_gb300 as fattn
            s["workspace"] = torch.empty(fattn.packed_workspace_bytes(len(lens), T), dtype=torch.uint8, device=dev)
        return s
    page = case["page"]
    if case["op"] in ("append", "append_kv4"):
        T = case["T"]
        pages = -(-T // page) + 3
        qkv = normal(T, H + 2 * Hkv, D)
        s.update(q=qkv[:, :H], k=qkv[:, H:H + Hkv], v=qkv[:, H + Hkv:])
        # channels of very different size, as keys have them
        s["k"] *= torch.exp(0.5 * torch.randn(Hkv, D, generator=g, device=dev)).to(dt)
        s["slots"] = torch.randperm(pages * page, generator=g, device=dev)[:T].contiguous()
        s["pos"] = torch.randint(0, MAX_POS, (T,), generator=g, device=dev, dtype=torch.int32)
        s["cos"], s["sin"] = _rotation_tables(case["rot"], dev)
        s["q_out"] = torch.empty(T, H, D, dtype=dt, device=dev)
        s["k_out"] = torch.empty(T, Hkv, D, dtype=dt, device=dev)
        if case["op"] == "append":
            s["k_pages"] = torch.zeros(pages, Hkv, page, D, dtype=dt, device=dev)
            s["v_pages"] = torch.zeros(pages, Hkv, page, D, dtype=dt, device=dev)
        else:
            s["v_out"] = torch.empty(T, Hkv, D, dtype=dt, device=dev)
            for n in "kv":
                s[n + "_codes"] = torch.zeros(pages, Hkv, page, D // 2, dtype=torch.uint8, device=dev)
                s[n + "_scales"] = torch.zeros(pages, Hkv, page, D // GROUP, 2, dtype=torch.float16, device=dev)
        return s
    lens = _contexts(case)
    B, Nq = case["B"], case["Nq"]
    width = -(-max(lens) // page)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    s["q"] = normal(B, H, Nq, D, std=3.0)
    perm = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    s["block_table"] = table
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["op"] == "decode":
        s["k_pages"] = normal(pages, Hkv, page, D)
        s["v_pages"] = normal(pages, Hkv, page, D)
    else:
        for n in "kv":
            shape = (pages, Hkv, page, D // 2)
            lo, hi = ((torch.randn(*shape, generator=g, device=dev) * 3.2 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
                      for _ in range(2))
            s[n + "_codes"] = lo | (hi << 4)
            sc = 0.2 + 0.2 * torch.rand(pages, Hkv, page, D // GROUP, generator=g, device=dev)
            zero = -7.5 * sc + 0.1 * torch.randn(sc.shape, generator=g, device=dev)
            s[n + "_scales"] = torch.stack([sc, zero], -1).half()
    s["out"] = torch.empty(B, H, Nq, D, dtype=dt, device=dev)
    s["lse"] = torch.empty(B, H, Nq, dtype=torch.float32, device=dev)
    if own:
        import tiled_attention_forward_gb300 as fattn
        s["workspace"] = torch.empty(fattn.decode_workspace_bytes(B, H, Nq, D, Hkv), dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# The operators, through the framework or in their plain form
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return _own(c["op"], s)
    return {"packed": _plain_packed, "append": _plain_append, "append_kv4": _plain_append,
            "decode": _plain_decode, "decode_kv4": _plain_decode}[c["op"]](s)


def _own(op, s):
    import tiled_attention_forward_gb300 as fattn
    c = s["case"]
    if op == "packed":
        return fattn.fwd_packed(s["q"], s["k"], s["v"], s["cu_seqlens"], causal=True, scale=s["scale"], out=s["out"],
                                lse=s["lse"], workspace=s["workspace"])
    if op == "append":
        q, k = fattn.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"], pos=s["pos"], cos=s["cos"],
                                  sin=s["sin"], interleaved=c["interleaved"], q=s["q"], q_out=s["q_out"],
                                  k_out=s["k_out"])
        return q, k, s["k_pages"], s["v_pages"]
    if op == "append_kv4":
        # held=True: k_out and v_out are the values that the cache now stands for
        return fattn.cache_append_kv4(s["k"], s["v"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"],
                                      s["slots"], pos=s["pos"], cos=s["cos"], sin=s["sin"],
                                      interleaved=c["interleaved"], q=s["q"], q_out=s["q_out"], k_out=s["k_out"],
                                      v_out=s["v_out"], held=True)
    if op == "decode":
        return fattn.decode(s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], scale=s["scale"],
                            out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return fattn.decode_kv4(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["block_table"],
                            s["seq_lens"], scale=s["scale"], out=s["out"], lse=s["lse"], workspace=s["workspace"])


def _plain_packed(s):
    q, k, v, out, lse = s["q"], s["k"], s["v"], s["out"], s["lse"]
    H, Hkv = q.shape[1], k.shape[1]
    at = 0
    for n in s["lens"]:  # one request after the other: their scores are matrices of different sizes
        qs = q[at:at + n].float().mul_(s["scale"]).transpose(0, 1).reshape(Hkv, H // Hkv * n, -1)
        ks = k[at:at + n].float().permute(1, 2, 0)
        vs = v[at:at + n].float().transpose(0, 1)
        p = torch.bmm(qs, ks).view(H, n, n)
        i = torch.arange(n, device=q.device)
        p.masked_fill_(i[None, :] > i[:, None], float("-inf"))
        m = p.amax(-1, keepdim=True)
        p.sub_(m).exp_()
        l = p.sum(-1, keepdim=True)
        o = torch.bmm(p.view(Hkv, H // Hkv * n, n), vs).view(H, n, -1) / l
        out[at:at + n] = o.transpose(0, 1).to(out.dtype)
        lse[:, at:at + n] = (m + l.log()).squeeze(-1)
        at += n
    return out, lse


def _rotate(x, cos, sin, rot, interleaved):
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = b * cos + a * sin
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = b * cos + a * sin
    return y


def _quantise(x):
    """Codes 0..15, scale and zero of groups of 32: x ~ code * scale + zero (64 bits: codes sit next to borders)."""
    x = x.unflatten(-1, (-1, GROUP)).clamp(-FP16_MAX, FP16_MAX)
    lo, hi = x.amin(-1), x.amax(-1)
    scale, zero = ((hi - lo) / 15).half(), lo.half()
    sd = scale.double()[..., None]
    code = torch.where(sd > 0, ((x - zero.double()[..., None]) / torch.where(sd > 0, sd, 1.0)).round(), 0.0).clamp(0, 15)
    return code, scale, zero


def _pack_k(code):
    """[.., D/32, 32] codes -> [.., D/2] bytes of a K row: word t * (D/32) + i holds dims 32 i + 8 t + e at nibble e/2 + 4 (e & 1)."""
    D = code.shape[-2] * GROUP
    w = code.to(torch.int64).unflatten(-1, (4, 4, 2)).movedim(-4, -3)      # [.., t, i, lo, hi], e = 2 lo + hi
    n = w.transpose(-1, -2).flatten(-2)                                    # nibble 4 hi + lo
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8).flatten(-3).reshape(*code.shape[:-2], D // 2)


def _pack_v(code):
    """[.., D/32, 32] codes -> bytes of a V row: dim 16 j + 8 h + g at nibble h * (D/16) + j of the g-th (D/16 * 2 nibbles)."""
    D = code.shape[-2] * GROUP
    w = code.to(torch.int64).flatten(-2).unflatten(-1, (D // 16, 2, 8))    # [.., j, h, g]
    n = w.movedim(-1, -3).movedim(-1, -2).flatten(-2)                      # [.., g, h * (D/16) + j]
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8).flatten(-2)


def _nibbles(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def _unpack_k(codes):
    D = codes.shape[-1] * 2
    n = _nibbles(codes).unflatten(-1, (4, D // 32, 2, 4))                  # [.., t, i, hi, lo]
    return n.movedim(-4, -3).transpose(-1, -2).flatten(-4)


def _unpack_v(codes):
    D = codes.shape[-1] * 2
    n = _nibbles(codes).unflatten(-1, (8, 2, D // 16))                     # [.., g, h, j]
    return n.movedim(-3, -1).transpose(-3, -2).flatten(-3)


def _plain_append(s):
    c = s["case"]
    page, kv4 = c["page"], c["op"] == "append_kv4"
    at = s["pos"].long()
    slot_page, slot_at = s["slots"] // page, s["slots"] % page
    cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
    dt = s["q"].dtype
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, c["rot"], c["interleaved"]).to(dt))
    if not kv4:
        s["k_out"].copy_(_rotate(s["k"].float(), cos, sin, c["rot"], c["interleaved"]).to(dt))
        s["k_pages"][slot_page, :, slot_at] = s["k_out"]
        s["v_pages"][slot_page, :, slot_at] = s["v"]
        return s["q_out"], s["k_out"], s["k_pages"], s["v_pages"]
    for n, x, pack in (("k", _rotate(s["k"].double(), cos.double(), sin.double(), c["rot"], c["interleaved"]), _pack_k),
                       ("v", s["v"].double(), _pack_v)):
        code, scale, zero = _quantise(x)
        s[n + "_codes"][slot_page, :, slot_at] = pack(code)
        s[n + "_scales"][slot_page, :, slot_at] = torch.stack([scale, zero], -1)
        s[n + "_out"].copy_((code.float() * scale.float()[..., None] + zero.float()[..., None]).flatten(-2).to(dt))
    return s["q_out"], s["k_out"], s["v_out"]


def _plain_decode(s):
    c = s["case"]
    B, H, Nq, D = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    width = s["block_table"].shape[1]

    def cached(name):  # [B, Hkv, width * page, D], 32 bits
        if c["op"] == "decode":
            x = s[name + "_pages"][s["block_table"].long()].float()
        else:
            sc = s[name + "_scales"][s["block_table"].long()].float()
            x = (_unpack_k if name == "k" else _unpack_v)(s[name + "_codes"][s["block_table"].long()]).float()
            x = x.unflatten(-1, (-1, GROUP)).mul_(sc[..., :1]).add_(sc[..., 1:]).flatten(-2)
        return x.transpose(1, 2).reshape(B, Hkv, width * page, D)

    j = torch.arange(width * page, device=s["q"].device)
    i = torch.arange(Nq, device=s["q"].device)
    seen = j[None, None, :] <= (s["seq_lens"][:, None].long() - Nq + i[None, :])[..., None]      # [B, Nq, keys]
    p = torch.matmul(s["q"].float().view(B, Hkv, H // Hkv * Nq, D), cached("k").transpose(-1, -2)).mul_(s["scale"])
    p = p.view(B, Hkv, H // Hkv, Nq, -1).masked_fill_(~seen[:, None, None], float("-inf"))
    m = p.amax(-1, keepdim=True).clamp_min_(-3e38)
    p.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = cached("v").masked_fill_(~seen.any(1)[:, None, :, None], 0.0)
    o = torch.matmul(p.view(B, Hkv, H // Hkv * Nq, -1), v).view(B, Hkv, H // Hkv, Nq, D)
    o = torch.where(l > 0, o / l, 0.0)
    s["out"].copy_(o.view(B, H, Nq, D).to(s["out"].dtype))
    s["lse"].copy_((m + l.log()).view(B, H, Nq))
    return s["out"], s["lse"]


# ---------------------------------------------------------------------------
# The work of one call
# ---------------------------------------------------------------------------
def work(case):
    H, Hkv, D = case["H"], case["Hkv"], case["D"]
    if case["op"] == "packed":
        lens = _packed_lens(case)
        T, pairs = sum(lens), sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": 2 * T * D * (2 * H + 2 * Hkv) + 4 * T * H, "flops": 4 * pairs * D * H}
    row4 = D // 2 + D // GROUP * 4  # bytes of a row of the 4-bit cache
    if case["op"] in ("append", "append_kv4"):
        T = case["T"]
        table = 4 * case["rot"] * T
        rows_in = 2 * T * D * (H + 2 * Hkv)
        rows_out = 2 * T * D * (H + (Hkv if case["op"] == "append" else 2 * Hkv))
        cache = 2 * T * Hkv * (2 * D if case["op"] == "append" else row4)
        return {"bytes": rows_in + rows_out + cache + table + 12 * T, "flops": 3 * T * case["rot"] * (H + Hkv)}
    lens, Nq = _contexts(case), case["Nq"]
    row = 2 * D if case["op"] == "decode" else row4
    qo = case["B"] * H * Nq * (4 * D + 4)
    return {"bytes": 2 * sum(lens) * Hkv * row + qo, "flops": 4 * sum(lens) * H * Nq * D}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "packed":
        return _exact_packed(s)
    if case["op"] in ("append", "append_kv4"):
        return _exact_append(case, s)
    return _exact_decode(case, s)


def _exact_packed(s):
    q, k, v = s["q"], s["k"], s["v"]
    T, H, D = q.shape
    share = H // k.shape[1]
    out = torch.zeros(T, H, D, dtype=torch.float64, device=q.device)
    lse = torch.zeros(H, T, dtype=torch.float64, device=q.device)
    cu = s["cu_seqlens"].tolist()
    for a, b in zip(cu[:-1], cu[1:]):
        hidden = torch.ones(b - a, b - a, dtype=torch.bool, device=q.device).triu(1)
        for h in range(H):
            z = s["scale"] * (q[a:b, h].double() @ k[a:b, h // share].double().T)
            z = torch.where(hidden, -torch.inf, z)
            e = torch.logsumexp(z, 1)
            lse[h, a:b] = e
            out[a:b, h] = torch.exp(z - e[:, None]) @ v[a:b, h // share].double()
    return out, lse


def _exact_rotated(case, s, x):
    r = case["rot"]
    unit = torch.complex(s["cos"].double(), s["sin"].double())[s["pos"].long()][:, None]
    x = x.double()
    head, tail = x[..., :r], x[..., r:]
    if case["interleaved"]:
        z = torch.view_as_complex(head.unflatten(-1, (r // 2, 2)).contiguous()) * unit
        return torch.cat([torch.view_as_real(z).flatten(-2), tail], -1)
    z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * unit
    return torch.cat([z.real, z.imag, tail], -1)


def _exact_append(case, s):
    q, k = _exact_rotated(case, s, s["q"]), _exact_rotated(case, s, s["k"])
    if case["op"] == "append":
        flat = []
        for pages, x in ((s["k_pages"], k), (s["v_pages"], s["v"].double())):
            rows = pages.double().transpose(1, 2).reshape(-1, case["Hkv"], case["D"])
            rows[s["slots"]] = x
            flat.append(rows.view(pages.shape[0], case["page"], case["Hkv"], case["D"]).transpose(1, 2).contiguous())
        return q, k, flat[0], flat[1]
    held = []
    for x in (k, s["v"].double()):
        parts = []
        for i in range(case["D"] // GROUP):
            y = x[..., GROUP * i:GROUP * (i + 1)].clip(-FP16_MAX, FP16_MAX)
            low = y.min(-1, keepdim=True).values
            step = ((y.max(-1, keepdim=True).values - low) / 15).to(torch.float16).double()
            low = low.to(torch.float16).double()
            steps = torch.nan_to_num((y - low) / step, nan=0.0, posinf=0.0, neginf=0.0)
            parts.append(low + step * torch.round(steps).clip(0, 15))
        held.append(torch.cat(parts, -1))
    return q, held[0], held[1]


def _exact_values(case, s, name, rows):
    """The cached rows of one request in 64 bits; rows: (page, offset) of each token."""
    if case["op"] == "decode":
        return s[name + "_pages"][rows[0], :, rows[1]].double()
    D = case["D"]
    d = torch.arange(D, device=rows[0].device)
    if name == "k":
        nibble = 8 * ((d % 32) // 8 * (D // 32) + d // 32) + (d % 8) // 2 + 4 * (d % 2)
    else:
        nibble = (d % 8) * (D // 8) + (d % 16) // 8 * (D // 16) + d // 16
    codes, scales = s[name + "_codes"][rows[0], :, rows[1]], s[name + "_scales"][rows[0], :, rows[1]]
    code = (codes[..., nibble // 2].int() >> (4 * (nibble % 2))) % 16
    sc = scales.double()[..., d // GROUP, :]
    return code * sc[..., 0] + sc[..., 1]


def _exact_decode(case, s):
    B, H, Nq, D = s["q"].shape
    Hkv, page = case["Hkv"], case["page"]
    out = torch.zeros(B, H, Nq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((B, H, Nq), -torch.inf, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(_contexts(case)):
        j = torch.arange(n, device=s["q"].device)
        rows = (s["block_table"][b].long()[j // page], j % page)
        k = _exact_values(case, s, "k", rows)
        v = _exact_values(case, s, "v", rows)
        for i in range(Nq):
            end = n - Nq + i + 1
            if end <= 0:
                continue
            z = s["scale"] * torch.einsum("hgd,nhd->hgn", s["q"][b, :, i].double().view(Hkv, H // Hkv, D), k[:end])
            e = torch.logsumexp(z, -1)
            lse[b, :, i] = e.view(H)
            out[b, :, i] = torch.einsum("hgn,nhd->hgd", torch.exp(z - e[..., None]), v[:end]).reshape(H, D)
    return out, lse
