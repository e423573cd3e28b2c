"""Plain 64-bit definitions of the ragged-batch calls, one sequence at a time
on the host (test infrastructure, no package code)."""
import math

import torch


def rope(x, positions, inv_freq, interleaved=False, inverse=False, factor=1.0):
    """x [T, H, d] -> float64."""
    y = x.double().clone()
    n = inv_freq.numel()
    a = positions.double()[:, None] * inv_freq.double()[None]
    c, s = torch.cos(a)[:, None] * factor, torch.sin(a)[:, None] * factor * (-1.0 if inverse else 1.0)
    i0 = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    i1 = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    u, w = x[..., i0].double(), x[..., i1].double()
    y[..., i0] = u * c - w * s
    y[..., i1] = w * c + u * s
    return y


def e4m3(rows):
    """(values under the row scale as float64 on the 8-bit grid, scale bytes) of float64 rows."""
    top = rows.abs().amax(-1)
    byte = torch.full(top.shape, 127, dtype=torch.int64)
    for i in range(top.numel()):
        t = float(top.view(-1)[i])
        if t > 0:
            m, e = math.frexp(t)            # t = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
            byte.view(-1)[i] = max(e - 9 + (1 if m > 0.875 else 0), -126) + 127
    z = rows * torch.exp2(-(byte.double() - 127))[..., None]
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / step) * step, byte


def widen(codes, byte):
    """What 8-bit rows stand for."""
    return codes.float().double() * torch.exp2(byte.double() - 127)[..., None]


def rows_of(pages, table, first, last, scale=None):
    """Positions first .. last - 1 of one sequence (table: its pages), float64 [n, Hkv, d]."""
    P = pages.shape[1]
    out = []
    for j in range(first, last):
        row = pages[int(table[j // P]), j % P]
        if scale is None:
            out.append(row.double())
        else:
            out.append(widen(row, scale[int(table[j // P]), :, j % P]))
    return torch.stack(out) if out else torch.zeros(0, *pages.shape[2:], dtype=torch.float64)


def attend(q, k, v, scale, dropped=()):
    """q [n, Hq, d] at the last n of the m positions of k, v [m, Hkv, d]: (out, lse [Hq, n]) in 64
    bits; a row that sees nothing gives zeros and -inf.  dropped: positions that are not there."""
    n, Hq, d = q.shape
    m, Hkv = k.shape[:2]
    out = torch.zeros(n, Hq, d, dtype=torch.float64)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64)
    keep = torch.ones(m, dtype=torch.bool)
    for j in dropped:
        keep[j] = False
    for i in range(n):
        pos = m - n + i
        if pos < 0:
            continue
        see = keep[:pos + 1].nonzero()[:, 0]
        if see.numel() == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            s = (k[see, g].double() @ q[i, h].double()) * scale
            lse[h, i] = torch.logsumexp(s, 0)
            out[i, h] = torch.exp(s - lse[h, i]) @ v[see, g].double()
    return out, lse


def make_table(gen, need, extra=2, first=0):
    """Shuffled pages for sequences needing need[b] pages each: (table [B, most], number of pages)."""
    total = sum(need) + extra
    order = torch.randperm(total, generator=gen)
    table = torch.full((len(need), max(max(need), 1)), -1, dtype=torch.int32)
    at = first
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    return table, total


def cu_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)
