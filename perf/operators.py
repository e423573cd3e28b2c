"""Performance cases of the serving operators around the paged K/V cache.

Five calls make up the way of a prompt and of its answer through a layer: rotary positions
(``rope``), the write of new keys and values into a paged cache, plain or quantised to 8 bits
(``cache_write``), its counterpart that reads rows back (``cache_read``), attention of new tokens over
the paged cache (``chunk_attn_paged``, from one token a sequence to thousands), and causal
attention over whole packed prompts (``packed_attn``).

With ``own`` false, ``run`` computes each of them in plain torch operations in 32 bits; with
``own`` true it makes the package's calls.  ``exact`` restates the definitions in 64 bits, one
sequence at a time.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one new token for each of 64 sequences of the decode workload: q and k are slices of one
        # projection's output, and the call is over in a few microseconds
        dict(name="rope_decode_64", op="rope", tokens=64, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             dtype="bf16", max_pos=32768, fused=True, inverse=False),
        # the 512-token fp32 workload with half of each head rotated, neighbouring pairs, transposed
        # (the rotation's gradient)
        dict(name="rope_part_f32", op="rope", tokens=511, hq=4, hkv=1, d=64, rot=32, interleaved=True,
             dtype="f32", max_pos=8192, fused=False, inverse=True),
        # a 65536-token prompt of the 64-head configuration at the end of a million positions
        dict(name="rope_long_64k", op="rope", tokens=65536, hq=64, hkv=4, d=128, rot=128, interleaved=False,
             dtype="bf16", max_pos=1 << 20, fused=False, inverse=False),
        # the decode step's write: one row a sequence, quantised, at each sequence's own position
        dict(name="write_decode_e4m3", op="write", batch=64, new=1, cached=4095, page=64, hkv=8, d=128,
             dtype="bf16", kv8=True, rope=False, lens=1),
        # a prompt chunk's write: keys rotated on their way into bf16 pages
        dict(name="write_chunk_rope", op="write", batch=16, new=2048, cached=4000, page=16, hkv=8, d=128,
             dtype="bf16", kv8=False, rope=True, lens=2),
        # a quantised cache of mixed lengths read back whole, packed (moved to another pool or to a
        # call that wants plain rows)
        dict(name="read_back_e4m3", op="read", batch=24, rows=16384, page=64, hkv=8, d=128, kv8=True, lens=3),
        # the first token after a short prompt, alone on the GPU: latency
        dict(name="chunk_one_token", op="chunk", batch=1, new=1, cached=699, page=16, hq=32, hkv=8, kv8=False,
             lens=4),
        # the decode workload over quantised caches of mixed lengths
        dict(name="chunk_decode_e4m3", op="chunk", batch=64, new=1, cached=32767, page=64, hq=32, hkv=8,
             kv8=True, lens=5),
        # prompt chunks of several sequences over what they have cached
        dict(name="chunk_prefill", op="chunk", batch=4, new=1000, cached=12000, page=128, hq=32, hkv=8,
             kv8=False, lens=6),
        # three short prompts, an odd number of heads a group
        dict(name="packed_short", op="packed", batch=3, max_len=37, hq=6, hkv=2, lens=7),
        # a batch of prompts of mixed lengths
        dict(name="packed_mixed", op="packed", batch=16, max_len=2000, hq=32, hkv=8, lens=8),
        # one long prompt, 8192 tokens of the 64-head configuration
        dict(name="packed_8k", op="packed", batch=1, max_len=8192, hq=64, hkv=4, lens=9),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "chunk", "packed"])
    lens = rng.randrange(1 << 30)
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * hkv <= 64])
    page = rng.choice([1, 8, 16, 32, 64, 128, 256])
    if op == "rope":
        d = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([d, d, d // 2, d // 4])
        heads = hkv * (group + 1)
        return dict(op=op, tokens=_log_int(rng, 1, (1 << 29) // (heads * d)), hq=hkv * group, hkv=hkv, d=d, rot=rot,
                    interleaved=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    max_pos=_log_int(rng, 1024, 1 << 20), fused=rng.random() < 0.5, inverse=rng.random() < 0.5)
    if op == "write":
        batch = _log_int(rng, 1, 128)
        new = _log_int(rng, 1, 32768 // batch)
        return dict(op=op, batch=batch, new=new, cached=_log_int(rng, 1, 16384), page=page, hkv=hkv,
                    d=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]), kv8=rng.random() < 0.5,
                    rope=rng.random() < 0.5, lens=lens)
    if op == "read":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, rows=_log_int(rng, 1, (1 << 19) // batch), page=page, hkv=hkv,
                    d=rng.choice([64, 128]), kv8=rng.random() < 0.7, lens=lens)
    if op == "chunk":
        # one token a sequence (a decode step) as often as chunks of them
        batch = _log_int(rng, 1, 64)
        new = 1 if rng.random() < 0.5 else _log_int(rng, 2, 2048)
        hq = hkv * group
        most = min(32768, (1 << 31) // (batch * hq * new), (1 << 24) // (batch * hkv))
        if most <= new:
            batch, most = 1, min(32768, (1 << 31) // (hq * new))
        cached = _log_int(rng, 1, max(1, most - new))
        return dict(op=op, batch=batch, new=new, cached=cached, page=page, hq=hq, hkv=hkv, kv8=rng.random() < 0.5,
                    lens=lens)
    batch = _log_int(rng, 1, 32)
    hq = hkv * group
    return dict(op="packed", batch=batch, max_len=_log_int(rng, 1, min(8192, int(math.sqrt((1 << 31) / (batch * hq))))),
                hq=hq, hkv=hkv, lens=lens)


def _lengths(case):
    """Lengths of the case's sequences: (new tokens, tokens in the cache with them)."""
    rng = random.Random(case["lens"])
    op, n = case["op"], case["batch"]
    if op == "packed":
        new = [case["max_len"]] + [0 if rng.random() < 0.05 else _log_int(rng, 1, case["max_len"]) for _ in range(n - 1)]
        return new, list(new)
    if op == "read":
        rows = [case["rows"]] + [rng.randint(1, case["rows"]) for _ in range(n - 1)]
        return rows, list(rows)
    new = [case["new"]] + [rng.randint(1, case["new"]) for _ in range(n - 1)]
    old = [case["cached"]] + [rng.randint(0, case["cached"]) for _ in range(n - 1)]
    return new, [a + b for a, b in zip(new, old)]


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


# ------------------------------------------------------------------ inputs

def _frequencies(case):
    """Angle per position of each rotated pair: base 10000, and beyond 32768 positions the slow
    pairs slowed further (a ramp over the pairs), as for long contexts."""
    half = case["rot"] // 2 if "rot" in case else case["d"] // 2
    i = torch.arange(half, dtype=torch.float64)
    f = 10000.0 ** (-i / half)
    far = max(1.0, case.get("max_pos", 0) / 32768.0)
    ramp = (i / max(1, half - 1)).clamp(0.0, 1.0)
    return (f * (1 - ramp) + f / far * ramp).to(DEV)


def _pool(rows, hkv, d, kv8, gen):
    """A page pool's rows: values as a cache of normalised keys or values holds them."""
    if not kv8:
        return torch.randn(rows, hkv, d, generator=gen, device=DEV, dtype=torch.bfloat16), None
    codes = torch.empty(rows, hkv, d, device=DEV, dtype=torch.float8_e4m3fn)
    scale = torch.empty(rows, hkv, device=DEV, dtype=torch.uint8)
    step = max(1, (1 << 28) // (hkv * d))
    for a in range(0, rows, step):
        x = torch.randn(min(step, rows - a), hkv, d, generator=gen, device=DEV)
        c, s = _quantise(x)
        codes[a:a + step], scale[a:a + step] = c, s
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case)}
    if op == "rope":
        T, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        if case["fused"]:
            qkv = torch.randn(T, (hq + 2 * hkv) * d, generator=gen, device=DEV).to(_dtype(case))
            st["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
            st["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        else:
            st["q"] = torch.randn(T, hq, d, generator=gen, device=DEV).to(_dtype(case))
            st["k"] = torch.randn(T, hkv, d, generator=gen, device=DEV).to(_dtype(case))
        top = case["max_pos"]
        if T > 1024:  # one prompt that ends at the last position
            st["positions"] = torch.arange(max(0, top - T), max(0, top - T) + T, device=DEV, dtype=torch.int32)
        else:
            st["positions"] = torch.randint(0, top, (T,), generator=gen, device=DEV, dtype=torch.int32)
        st["inv_freq"] = _frequencies(case)
        return st

    new, kv = _lengths(case)
    T, B = sum(new), case["batch"]
    st["max_new"], st["max_kv"], st["total"] = max(new), max(kv), T
    st["cu"] = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device=DEV)
    if op == "packed":
        hq, hkv = case["hq"], case["hkv"]
        for name, h in (("q", hq), ("k", hkv), ("v", hkv)):
            st[name] = torch.randn(T, h, 128, generator=gen, device=DEV, dtype=torch.bfloat16)
    else:
        P, hkv, d = case["page"], case["hkv"], case.get("d", 128)
        need = [-(-n // P) for n in kv]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=gen, device=DEV, dtype=torch.int32)
        most = max(need)
        table = torch.full((B, most), -1, dtype=torch.int32)
        host = order.cpu()
        at = 0
        for b in range(B):
            table[b, :need[b]] = host[at:at + need[b]]
            at += need[b]
        st["table"] = table.to(DEV)
        st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
        for name in ("k", "v"):
            rows, scale = _pool(pages * P, hkv, d, case["kv8"], gen)
            st[name + "_pages"] = rows.view(pages, P, hkv, d)
            st[name + "_scale"] = None if scale is None else scale.view(pages, P, hkv).transpose(1, 2).contiguous()
        if op == "write":
            for name in ("k", "v"):
                st[name] = torch.randn(T, hkv, d, generator=gen, device=DEV).to(_dtype(case))
            if case["dtype"] == "f32" and not case["kv8"]:
                for name in ("k_pages", "v_pages"):
                    st[name] = st[name].float()
            st["inv_freq"] = _frequencies(case) if case["rope"] else None
        if op == "chunk":
            st["q"] = torch.randn(T, case["hq"], 128, generator=gen, device=DEV, dtype=torch.bfloat16)
    if op in ("packed", "chunk"):  # scratch that a serving loop keeps (zeroed once)
        st["ws"] = torch.zeros(128 << 20, dtype=torch.uint8, device=DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _rotate(x, positions, inv_freq, interleaved, inverse=False):
    """x [T, H, d] in 32 bits, the first 2 * len(inv_freq) of d rotated; angles in 64 bits."""
    half = inv_freq.numel()
    angle = positions.double()[:, None] * inv_freq[None, :]
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    if inverse:
        s = -s
    x = x.float()
    rest = x[..., 2 * half:]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack((a * c - b * s, b * c + a * s), dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat((a * c - b * s, b * c + a * s), dim=-1)
    return torch.cat((turned, rest), dim=-1)


def _quantise(x):
    """Rows of 32-bit x to 8-bit floats under the smallest power of two that holds the row's largest
    magnitude: x ~ codes * 2**(scale - 127)."""
    m, e = torch.frexp(x.abs().amax(-1))
    top = torch.where(m == 0, torch.zeros_like(e), e - 9 + (m > 0.875).to(e.dtype)).clamp(-126, 127)
    return torch.ldexp(x, -top[..., None]).to(torch.float8_e4m3fn), (top + 127).to(torch.uint8)


def _widen(codes, scale):
    """8-bit rows with their powers of two -> 32 bits; other rows are only widened."""
    if scale is None:
        return codes.float()
    return codes.float() * (scale.int() << 23).view(torch.float32)[..., None]


def _places(cu, total):
    """For each packed row: its sequence and its place there."""
    t = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous().long(), t, right=True)
    return seq, t - cu.long()[seq]


def _pages_at(table, seq, pos, page):
    return table[seq, pos // page].long(), pos % page


def _attend(q, k, v, new, kv, scale):
    """q [B, Lq, Hq, d], k and v [B, Lk, Hkv, d], 32 bits, padded at their ends; token i of
    sequence b at position kv[b] - new[b] + i sees the keys up to its own."""
    B, Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qg = q.view(B, Lq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Lq, d)
    s = torch.matmul(qg, k.permute(0, 2, 3, 1)).view(B, Hkv, G, Lq, Lk).mul_(scale)
    at = (kv - new).long()[:, None] + torch.arange(Lq, device=q.device)[None]
    unseen = torch.arange(Lk, device=q.device)[None, None, :] > at[:, :, None]
    s.masked_fill_(unseen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-1e30)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * Lq, Lk), v.permute(0, 2, 1, 3)).view(B, Hkv, G, Lq, d)
    o = o / total.clamp(min=1e-37)
    lse = (m + total.log())[..., 0]
    return o.permute(0, 3, 1, 2, 4).reshape(B, Lq, Hq, d), lse.reshape(B, Hq, Lq)


def _padded(x, cu, new, longest):
    j = torch.arange(longest, device=x.device)
    at = cu.long()[:-1, None] + j[None]
    there = j[None] < new.long()[:, None]
    return x.float()[torch.where(there, at, 0)] * there[..., None, None]


def _plain(st):
    op, case = st["op"], st["case"]
    if op == "rope":
        dt = st["q"].dtype
        return tuple(_rotate(x, st["positions"], st["inv_freq"], case["interleaved"], case["inverse"]).to(dt)
                     for x in (st["q"], st["k"]))
    cu, total = st["cu"], st["total"]
    new = cu[1:] - cu[:-1]
    seq, at = _places(cu, total)
    if op == "packed":
        n = st["max_new"]
        o, lse = _attend(*(_padded(st[x], cu, new, n) for x in ("q", "k", "v")), new, new, 128 ** -0.5)
        return o[seq, at].to(torch.bfloat16), lse[seq, :, at].t().contiguous()

    page = case["page"]
    if op == "read":
        where, row = _pages_at(st["table"], seq, at, page)
        got = []
        for x in ("k", "v"):
            rows, scale = st[x + "_pages"], st[x + "_scale"]
            if scale is None:
                got.append(_widen(rows[where, row], None).to(torch.bfloat16))
            else:
                got.append(_widen(rows.view(torch.uint8)[where, row].view(torch.float8_e4m3fn),
                                  scale[where, :, row]).to(torch.bfloat16))
        return tuple(got)

    if op == "write":
        pos = (st["kv_len"] - new).long()[seq] + at
        where, row = _pages_at(st["table"], seq, pos, page)
        for x in ("k", "v"):
            rows = st[x].float()
            if x == "k" and st["inv_freq"] is not None:
                rows = _rotate(rows, pos, st["inv_freq"], False)
            if st[x + "_scale"] is None:
                st[x + "_pages"][where, row] = rows.to(st[x + "_pages"].dtype)
            else:
                codes, scale = _quantise(rows)
                st[x + "_pages"].view(torch.uint8)[where, row] = codes.view(torch.uint8)
                st[x + "_scale"][where, :, row] = scale
        return tuple(st[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale") if st[x] is not None)

    # chunk: the sequences' rows gathered from their pages, then attention
    B, Lk = st["table"].shape[0], st["max_kv"]
    j = torch.arange(Lk, device=cu.device)
    there = j[None] < st["kv_len"].long()[:, None]
    where = torch.where(there, st["table"][:, j // page].long(), 0)
    row = torch.where(there, (j % page)[None], 0)
    wide = []
    for x in ("k", "v"):
        rows, scale = st[x + "_pages"], st[x + "_scale"]
        if scale is None:
            wide.append(_widen(rows[where, row], None))
        else:
            wide.append(_widen(rows.view(torch.uint8)[where, row].view(torch.float8_e4m3fn),
                               scale[where, :, row]))
    o, lse = _attend(_padded(st["q"], cu, new, st["max_new"]), wide[0], wide[1], new, st["kv_len"], 128 ** -0.5)
    return o[seq, at].to(torch.bfloat16), lse[seq, :, at].t().contiguous()


def run(st):
    if not own:
        return _plain(st)
    import hybrid_sparse_attention_tcgen05_b200 as hs
    op, case = st["op"], st["case"]
    if op == "rope":
        return hs.rope(st["q"], st["positions"], st["inv_freq"], k=st["k"], interleaved=case["interleaved"],
                       inverse=case["inverse"])
    if op == "packed":
        return hs.packed_attn(st["q"], st["k"], st["v"], st["cu"], max_len=st["max_new"], ws=st["ws"])
    if op == "read":
        return hs.cache_read(st["k_pages"], st["v_pages"], st["cu"], st["table"], total=st["total"],
                             k_scale=st["k_scale"], v_scale=st["v_scale"], dtype=torch.bfloat16)
    if op == "write":
        hs.cache_write(st["k"], st["v"], st["k_pages"], st["v_pages"], st["cu"], st["kv_len"], st["table"],
                       k_scale=st["k_scale"], v_scale=st["v_scale"], inv_freq=st["inv_freq"])
        return tuple(st[x] for x in ("k_pages", "v_pages", "k_scale", "v_scale") if st[x] is not None)
    return hs.chunk_attn_paged(st["q"], st["k_pages"], st["v_pages"], st["cu"], st["kv_len"], st["table"],
                               max_q=st["max_new"], max_len=st["max_kv"], k_scale=st["k_scale"],
                               v_scale=st["v_scale"], ws=st["ws"])


# ------------------------------------------------------------------ work and definitions

def work(case):
    op = case["op"]
    if op == "rope":
        es = 4 if case["dtype"] == "f32" else 2
        heads = case["hq"] + case["hkv"]
        return {"bytes": case["tokens"] * (heads * case["d"] * es * 2 + 4) + case["rot"] * 4,
                "flops": 3 * case["tokens"] * heads * case["rot"]}
    new, kv = _lengths(case)
    T, rows = sum(new), sum(kv)
    if op == "packed":
        pairs = sum(n * (n + 1) // 2 for n in new)
        return {"bytes": T * (2 * (case["hq"] + case["hkv"]) * 256 + case["hq"] * 4),
                "flops": 4 * 128 * case["hq"] * pairs}
    hkv, d = case["hkv"], case.get("d", 128)
    es = 4 if case.get("dtype") == "f32" else 2
    if op == "read":
        return {"bytes": 2 * T * hkv * ((d + 1 if case["kv8"] else 2 * d) + 2 * d), "flops": 0}
    if op == "write":
        return {"bytes": 2 * T * hkv * (es * d + (d + 1 if case["kv8"] else es * d)), "flops": 0}
    pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, kv))
    return {"bytes": T * case["hq"] * (2 * 256 + 4) + 2 * rows * hkv * (129 if case["kv8"] else 256),
            "flops": 4 * 128 * case["hq"] * pairs}


def _turn64(x, pos, f, interleaved, sign):
    y = x.double().clone()
    n = f.numel()
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        t = pos.double() * f[i]
        c, s = torch.cos(t)[:, None], sign * torch.sin(t)[:, None]
        y[..., a] = x[..., a].double() * c - x[..., b].double() * s
        y[..., b] = x[..., a].double() * s + x[..., b].double() * c
    return y


def _e4m3_64(y):
    """Nearest 8-bit floats (ties to even) of 64-bit rows, and the exponents of their rows' scales."""
    top = y.abs().amax(-1)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448.0)), torch.zeros_like(top))
    e = torch.where((top > 0) & (top <= 448.0 * torch.exp2(e - 1)), e - 1, e)
    e = torch.where((top > 0) & (top > 448.0 * torch.exp2(e)), e + 1, e).clamp(-126, 127)
    z = y * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / step) * step, e


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        sign = -1.0 if case["inverse"] else 1.0
        if case["tokens"] * (case["hq"] + case["hkv"]) * case["d"] > 1 << 30:
            return None
        return tuple(_turn64(st[x], st["positions"], st["inv_freq"], case["interleaved"], sign) for x in ("q", "k"))
    new, kv = _lengths(case)
    B = case["batch"]
    starts = [sum(new[:b]) for b in range(B)]

    def rows_of(x, b, first, last):
        """The 64-bit cache rows first .. last - 1 of sequence b."""
        j = torch.arange(first, last, device=DEV)
        page = st["table"][b].long()[j // case["page"]]
        r = st[x + "_pages"].view(torch.uint8)[page, j % case["page"]] if case["kv8"] else \
            st[x + "_pages"][page, j % case["page"]]
        if case["kv8"]:
            e = st[x + "_scale"][page, :, j % case["page"]].double() - 127.0
            return r.view(torch.float8_e4m3fn).float().double() * torch.exp2(e)[..., None]
        return r.double()

    if op == "read":
        return tuple(torch.cat([rows_of(x, b, 0, new[b]) for b in range(B)]) for x in ("k", "v"))
    if op == "write":
        got = [st[x].float().double() for x in ("k_pages", "v_pages")]
        for n, x in enumerate(("k", "v")):
            for b in range(B):
                pos = torch.arange(kv[b] - new[b], kv[b], device=DEV)
                y = st[x][starts[b]:starts[b] + new[b]].double()
                if n == 0 and st["inv_freq"] is not None:
                    y = _turn64(y, pos, st["inv_freq"], False, 1.0)
                if case["kv8"]:
                    y, _ = _e4m3_64(y)
                got[n][st["table"][b].long()[pos // case["page"]], pos % case["page"]] = y
        return tuple(got) + ((None, None) if case["kv8"] else ())

    hq, hkv = case["hq"], case["hkv"]
    pairs = sum(n * m for n, m in zip(new, kv))
    if pairs * hq > 1 << 35:
        return None
    outs, lses = [], []
    for b in range(B):
        n, m = new[b], kv[b]
        part = slice(starts[b], starts[b] + n)
        if op == "packed":
            k, v = st["k"][part].double(), st["v"][part].double()
        else:
            k, v = rows_of("k", b, 0, m), rows_of("v", b, 0, m)
        q = st["q"][part].double()
        o = torch.empty(n, hq, 128, dtype=torch.float64, device=DEV)
        lse = torch.empty(hq, n, dtype=torch.float64, device=DEV)
        late = torch.arange(m, device=DEV)[None, :] > torch.arange(m - n, m, device=DEV)[:, None]
        for h in range(hq):
            g = h // (hq // hkv)
            s = (q[:, h] @ k[:, g].t()) / math.sqrt(128.0)
            s = s.masked_fill(late, -math.inf)
            lse[h] = torch.logsumexp(s, -1)
            o[:, h] = torch.exp(s - lse[h][:, None]) @ v[:, g]
        outs.append(o)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses, 1)
