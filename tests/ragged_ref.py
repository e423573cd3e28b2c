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
    """q [n, Hq, d] at the last n of the m positions of k, v [m, Hkv, d]: (out, lse [Hq, n],
    sum_j p_j |v_j|) in 64 bits; a row that sees nothing gives zeros and -inf.  dropped: positions
    that are not there."""
    n, Hq, d = q.shape
    m, Hkv = k.shape[:2]
    out = torch.zeros(n, Hq, d, dtype=torch.float64)
    size = torch.zeros(n, Hq, d, dtype=torch.float64)
    lse = torch.full((Hq, n), -math.inf, dtype=torch.float64)
    if n == 0 or m == 0:
        return out, lse, size
    see = torch.arange(m)[None] <= torch.arange(m - n, m)[:, None]
    see[:, list(dropped)] = False
    for h in range(Hq):
        g = h // (Hq // Hkv)
        s = (q[:, h].double() @ k[:, g].double().t()) * scale
        s = s.masked_fill(~see, -math.inf)
        lse[h] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[h].clamp(min=-1e300)[:, None])
        out[:, h] = p @ v[:, g].double()
        size[:, h] = p @ v[:, g].double().abs()
    return out, lse, size


def check_attend(name, out, lse, want, slack=0.0):
    """out, lse of one sequence's rows against attend()'s.  The probabilities are rounded to bf16 before
    they meet v (2^-8 of each term p |v|), the result to bf16 (2^-8 of it); a score is a sum of 128
    products in fp32, off by at most 128 * 2^-24 * sum |q k| * scale, which for entries of size ~1 is
    under 1e-4, and moves each probability by that relative amount (twice: its own and the sum's)."""
    o, l, size = want
    tol = (2.0 ** -8 + 2e-4 + slack) * size + 2.0 ** -8 * o.abs() + 1e-30
    err = (out.double().cpu() - o).abs()
    assert bool(torch.isfinite(out.float()).all()), f"{name}: not finite"
    assert bool((err <= tol).all()), f"{name}: off by {float((err - tol).max())} past the bound, error {float(err.max())}"
    none = torch.isinf(l)
    assert torch.equal(torch.isinf(lse.cpu()) & (lse.cpu() < 0), none), f"{name}: rows that see nothing"
    e = (lse.double().cpu() - l)[~none].abs()
    assert e.numel() == 0 or float(e.max()) <= 1e-4 + slack, f"{name}: lse off by {float(e.max())}"


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
