"""Attention over packed prompts and paged caches with scores that rise along the keys by more than
the running reference lets pass without moving: between the halves of a key tile, between tiles,
between 16-key blocks, and in one late step.  Values shrink as the scores rise (in half of the KV
heads), so that early and late keys weigh alike and a wrong rescale of what came before shows.
Rows of one warp move their references at different steps.  Compared with the 64-bit definition."""
import math

import pytest
import torch

import hybrid_sparse_attention_tcgen05_b200 as hs
from hybrid_sparse_attention_tcgen05_b200 import _lib
import ragged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
SCALE = 1 / math.sqrt(128)
HKV = 4


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _levels(m):
    """Score of each of m keys in log2 units, for the four KV heads."""
    j = torch.arange(m)
    return torch.stack([10 * (j // 64).clamp(max=9), 12 * (j // 128).clamp(max=7), 9 * ((j // 16) % 11),
                        30 * (j >= (3 * m) // 4)], 1).double()


def _rows(gen, new, kv, hq):
    """q of the new rows and k, v of all positions, sequence after sequence (bf16)."""
    G = hq // HKV
    e = torch.where(torch.rand(128, generator=gen) < 0.5, -1.0, 1.0)
    unit = math.log(2) / (128 * SCALE)
    q, k, v = [], [], []
    for n, m in zip(new, kv):
        level = _levels(m)
        k.append(0.3 * torch.randn(m, HKV, 128, generator=gen) + (level * unit).float()[..., None] * e)
        size = torch.where(torch.arange(HKV) < 2, torch.exp2(-level), torch.ones(())).float()
        v.append(torch.randn(m, HKV, 128, generator=gen) * size[..., None])
        c = 1.0 - 0.5 * ((torch.arange(n)[:, None] + torch.arange(hq)[None] % G) % 3)     # 1, a half, 0
        q.append(0.3 * torch.randn(n, hq, 128, generator=gen) + c[..., None] * e)
    return [torch.cat(x).to(BF) for x in (q, k, v)]


def _check(name, q, k, v, out, lse, v_byte=None):
    """One sequence.  As ragged_ref.check_attend, with a score's bound taken from the rows (128 products
    summed in fp32: 128 * 2^-24 * sum |q k| * scale; it moves a probability twice, by itself and by the
    sum).  8-bit rows: probabilities below 2^-14 of the largest product of probability and row scale may
    be held to 2^-25 of that product, times codes of up to 448."""
    want, wl, size = ref.attend(q, k, v, SCALE)
    G = q.shape[1] // HKV
    slack = 0.0
    for h in range(q.shape[1]):
        slack = max(slack, float((q[:, h].double().abs() @ k[:, h // G].double().abs().t()).max()))
    slack *= 2 * 128 * 2.0 ** -24 * SCALE
    tol = (2.0 ** -8 + 2e-4 + slack) * size + 2.0 ** -8 * want.abs() + 1e-30
    if v_byte is not None:
        n, m = q.shape[0], k.shape[0]
        see = torch.arange(m)[None] <= torch.arange(m - n, m)[:, None]
        for h in range(q.shape[1]):
            s = (q[:, h].double() @ k[:, h // G].double().t() * SCALE).masked_fill(~see, -math.inf)
            ps = torch.exp(s - wl[h][:, None]) * torch.exp2(v_byte[:, h // G].double() - 127)
            tol[:, h] += 2.0 ** -25 * 448 * m * ps.amax(1, keepdim=True)
    err = (out.double().cpu() - want).abs()
    assert bool(torch.isfinite(out.float()).all()) and bool(torch.isfinite(lse).all()), f"{name}: not finite"
    assert bool((err <= tol).all()), f"{name}: {float((err / tol).max())} of the bound"
    assert float((lse.double().cpu() - wl).abs().max()) <= 1e-4 + slack, f"{name}: lse"


def _same_each_time(call):
    first = [x.clone() for x in call()]
    for _ in range(4):
        again = call()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    return first


# The last rows of a prompt fill one row tile or less, over 3, 5, 7 and 4 key tiles, beside whole items
# of two row tiles.
@pytest.mark.parametrize("hq,lens", [(16, [340, 586]), (16, [864, 453, 33]), (4, [356, 512 + 7, 768 + 70]),
                                     (64, [323, 577, 70]), (12, [90 + 300])])
def test_packed_rising_scores(hq, lens):
    gen = torch.Generator().manual_seed(sum(lens))
    q, k, v = _rows(gen, lens, lens, hq)
    cu = ref.cu_of(lens)
    dq, dk, dv = q.to(DEV), k.to(DEV), v.to(DEV)
    out, lse = _same_each_time(lambda: hs.packed_attn(dq, dk, dv, cu.to(DEV), max_len=max(lens)))
    for b, n in enumerate(lens):
        part = slice(int(cu[b]), int(cu[b]) + n)
        _check(f"seq {b}", q[part], k[part], v[part], out[part], lse[:, part])


# One row tile over 3, 5, 7, 2 and 4 key tiles, two row tiles, keys split over pieces, and the few rows
# that the decode kernel takes.
@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq,new,kv", [(16, [20, 31, 12], [330, 600, 870]), (16, [20, 32, 30], [200, 500, 385]),
                                       (4, [100, 70], [380, 641]), (64, [8, 7], [380, 897]), (16, [60, 64], [700, 850]),
                                       (16, [30], [4500]), (16, [9, 300], [3000, 1700]),
                                       (16, [1, 1, 1], [300, 900, 17]), (16, [4, 2], [700, 130]), (64, [1], [3000]),
                                       (4, [8, 5], [900, 260])])
def test_chunk_rising_scores(hq, new, kv, pool):
    gen = torch.Generator().manual_seed(sum(kv) + hq)
    q, k, v = _rows(gen, new, kv, hq)
    P = 32
    table, pages = ref.make_table(gen, [-(-m // P) for m in kv])
    dt, cu, all_rows = table.to(DEV), ref.cu_of(new), ref.cu_of(kv).to(DEV)
    dtype = BF if pool == "bf16" else torch.float8_e4m3fn
    pk, pv = (torch.zeros(pages, P, HKV, 128, device=DEV).to(dtype) for _ in range(2))
    sc = {} if pool == "bf16" else {n: torch.zeros(pages, HKV, P, dtype=torch.uint8, device=DEV)
                                    for n in ("k_scale", "v_scale")}
    hs.cache_write(k.to(DEV), v.to(DEV), pk, pv, all_rows, _int(kv), dt, **sc)
    k, v = (x.cpu() for x in hs.cache_read(pk, pv, all_rows, dt, total=sum(kv), dtype=torch.float32, **sc))
    ws = torch.zeros(hs.ragged_workspace_size(len(new), sum(new), hq, HKV, 128, max(new), max(kv)), dtype=torch.uint8,
                     device=DEV)
    out, lse = _same_each_time(lambda: hs.chunk_attn_paged(q.to(DEV), pk, pv, cu.to(DEV), _int(kv), dt, max_q=max(new),
                                                           max_len=max(kv), ws=ws, **sc))
    assert hs.workspace_status(ws) == _lib.HS_OK
    for b, (n, m) in enumerate(zip(new, kv)):
        part, rows = slice(int(cu[b]), int(cu[b]) + n), slice(sum(kv[:b]), sum(kv[:b]) + m)
        byte = None
        if pool == "e4m3":
            byte = torch.stack([sc["v_scale"].cpu()[int(table[b, j // P]), :, j % P] for j in range(m)])
        _check(f"seq {b}", q[part], k[rows], v[rows], out[part], lse[:, part], byte)
