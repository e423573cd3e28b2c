"""Attention over packed prompts and paged caches where it can go wrong quietly."""
import math

import pytest
import torch

import hybrid_sparse_attention_tcgen05_b200 as hs
from hybrid_sparse_attention_tcgen05_b200 import _lib
import ragged_ref as ref
from test_gpu_ragged_attn import BF, DEV, SCALE, _check_all, _chunk, _int, _paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [1, 2, 4, 8, 32, 128])
def test_every_third_page_outside_the_pool(P, pool):
    """Flags of lost keys in most key tiles, changing from tile to tile, in items of one and of two row
    tiles; the same bits each time."""
    gen = torch.Generator().manual_seed(P)
    new, old, hq, hkv = [30, 140, 7], [900, 500, 1300], 8, 2
    kv = [a + b for a, b in zip(new, old)]
    table, got = _paged(gen, kv, P, hkv, pool)
    dropped = []
    for b, n in enumerate(kv):
        gone = [i for i in range(-(-n // P)) if (i + i // 7) % 3 == b % 3]
        for i in gone:
            table[b, i] = [-1, got["k"][0].shape[0], 2 ** 31 - 1][i % 3]
        dropped.append(sorted(j for i in gone for j in range(i * P, min((i + 1) * P, n))))
    q = torch.randn(sum(new), hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new)
    ws = torch.zeros(hs.ragged_workspace_size(3, sum(new), hq, hkv, 128, 140, max(kv)), dtype=torch.uint8, device=DEV)
    first = None
    for _ in range(5):
        out, lse = _chunk(q, got, cu, kv, table, max_q=140, max_len=max(kv), ws=ws)
        assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_INDEX
        first = first or (out.clone(), lse.clone())
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    _check_all(f"P {P}", q, got, cu, new, out, lse, dropped=dropped)


HUGE = 1e38


@pytest.mark.parametrize("new,old", [([200, 90], [0, 0]), ([140, 20], [300, 700]), ([20, 3], [2000, 900]), ([4, 2], [500, 31])])
@pytest.mark.parametrize("pool", ["packed", "bf16", "e4m3"])
def test_huge_values_behind_a_row_do_not_reach_it(pool, new, old):
    """Finite values near the type's largest at positions that a row does not see: its result is the
    definition's, wherever in a tile they lie.  (Rows that do see one are not looked at: their sums in
    fp32 may overflow before the division.)"""
    gen = torch.Generator().manual_seed(sum(new) + len(pool))
    if pool == "packed":
        old = [0, 0]
    hq, hkv, P = 8, 2, 16
    kv, cu, T = [a + b for a, b in zip(new, old)], ref.cu_of(new), sum(new)
    q = torch.randn(T, hq, 128, generator=gen).to(BF)
    k, v = (torch.randn(sum(kv), hkv, 128, generator=gen).to(BF) for _ in range(2))
    at = [range(m - n + 1, m) for n, m in zip(new, kv)]          # all but the first new row
    first = ref.cu_of(kv)
    table, pages = ref.make_table(gen, [-(-m // P) for m in kv])
    dt = table.to(DEV)
    sc = {}
    if pool == "e4m3":
        sc = {n: torch.zeros(pages, hkv, P, dtype=torch.uint8, device=DEV) for n in ("k_scale", "v_scale")}
    dtype = torch.float8_e4m3fn if pool == "e4m3" else BF
    pk, pv = (torch.zeros(pages, P, hkv, 128, device=DEV).to(dtype) for _ in range(2))
    for step in (1, 3, 16, 37):                                  # huge from a row on: every step-th new position
        vx = v.clone()
        lim = []
        for b in range(2):
            hit = list(at[b])[step - 1::step][:40]
            for i, j in enumerate(hit):
                vx[int(first[b]) + j] = HUGE * (-1) ** i
            lim.append(min(hit) - (kv[b] - new[b]) if hit else new[b])     # new rows that see none of them
        if pool == "packed":
            out, lse = hs.packed_attn(q.to(DEV), k.to(DEV), vx.to(DEV), cu.to(DEV), max_len=max(new))
            rk, rv = k, vx
        else:
            hs.cache_write(k.to(DEV), vx.to(DEV), pk, pv, first.to(DEV), _int(kv), dt, **sc)
            out, lse = hs.chunk_attn_paged(q.to(DEV), pk, pv, cu.to(DEV), _int(kv), dt, max_q=max(new), max_len=max(kv), **sc)
            rk, rv = (x.cpu() for x in hs.cache_read(pk, pv, first.to(DEV), dt, total=sum(kv), dtype=torch.float32, **sc))
        for b in range(2):
            r0, n = int(cu[b]), lim[b]
            rows = slice(int(first[b]), int(first[b]) + kv[b] - new[b] + n)
            ref.check_attend(f"step {step} seq {b}", out[r0:r0 + n], lse[:, r0:r0 + n],
                             ref.attend(q[r0:r0 + n], rk[rows], rv[rows], SCALE))


@pytest.mark.parametrize("new", [1, 3])
def test_keys_far_below_the_maximum_give_nothing(new):
    """Probabilities below the smallest float are 0, also beside huge values."""
    gen = torch.Generator().manual_seed(new)
    hq, hkv, m = 8, 2, 300
    e = torch.where(torch.rand(128, generator=gen) < 0.5, -1.0, 1.0)
    for rows in (new, 90):
        q = (0.1 * torch.randn(rows, hq, 128, generator=gen) + e).to(BF)
        k = 0.1 * torch.randn(m, hkv, 128, generator=gen)
        v = torch.randn(m, hkv, 128, generator=gen)
        low = torch.arange(m) % 5 != 0
        k[low] -= 20.0 * e                    # 20 * 128 / sqrt(128) = 226 below, in natural units
        v[low] = HUGE
        k, v = k.to(BF), v.to(BF)
        table = _int([list(range(5))])
        pk, pv = (torch.zeros(5, 64, hkv, 128, dtype=BF, device=DEV) for _ in range(2))
        hs.cache_write(k.to(DEV), v.to(DEV), pk, pv, _int([0, m]), _int([m]), table)
        out, lse = hs.chunk_attn_paged(q.to(DEV), pk, pv, _int([0, rows]), _int([m]), table, max_q=rows, max_len=m)
        # scores of up to 226: 128 * 2^-24 * 226 * 2
        ref.check_attend(f"{rows} rows", out, lse, ref.attend(q, k, v, SCALE), slack=4e-3)


@pytest.mark.parametrize("size", [1.0, 1e-3, 1e-6, 1e-12])
@pytest.mark.parametrize("new", [1, 4, 40])
def test_8bit_rows_of_zeros_beside_small_values(new, size):
    """A value row of zeros has the scale 2^0; where its key has the largest score, small values beside
    it keep their bits."""
    gen = torch.Generator().manual_seed(new)
    hq, hkv, P, m = 8, 2, 16, 200
    q = torch.randn(new, hq, 128, generator=gen).to(BF)
    k, v = torch.randn(m, hkv, 128, generator=gen), torch.randn(m, hkv, 128, generator=gen) * size
    v[::7] = 0
    v[3::7] = -0.0
    k[5] = 1.5 * q.float().view(new, hkv, hq // hkv, 128)[0].mean(1)      # above the others for the first row
    v[5] = 0
    table = _int([list(range(13))])
    pk, pv = (torch.zeros(13, P, hkv, 128, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    sc = {n: torch.zeros(13, hkv, P, dtype=torch.uint8, device=DEV) for n in ("k_scale", "v_scale")}
    hs.cache_write(k.to(DEV), v.to(DEV), pk, pv, _int([0, m]), _int([m]), table, **sc)
    assert bool((sc["v_scale"][0, :, 5] == 127).all())
    rk, rv = (x.cpu() for x in hs.cache_read(pk, pv, _int([0, m]), table, total=m, dtype=torch.float32, **sc))
    out, lse = hs.chunk_attn_paged(q.to(DEV), pk, pv, _int([0, new]), _int([m]), table, max_q=new, max_len=m, **sc)
    ref.check_attend(f"{new} rows", out, lse, ref.attend(q, rk, rv, SCALE))


@pytest.mark.parametrize("hq,hkv", [(8, 2), (6, 2), (7, 1)])
@pytest.mark.parametrize("fill", [math.nan, 3e38, 0.0])
def test_rows_of_others_in_a_tile_change_nothing(hq, hkv, fill):
    """Whatever lies in a row tile beside a sequence's own rows, its rows are the same bits: rows of nobody
    between sequences that hold NaN, huge numbers or zeros, and group sizes that do not fill a tile."""
    gen = torch.Generator().manual_seed(hq)
    lens, gap, T = [70, 5, 33, 130], 40, 4 * 170
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(BF) for h in (hq, hkv, hkv))
    # every second sequence has no keys and is the gap behind the one before it; its rows hold `fill`
    cu, kv, at = [], [], 0
    for n in lens:
        cu += [at, at + n]
        kv += [n + 600, 0]
        at += n + gap
    cu.append(at)
    table, got = _paged(gen, kv, 32, hkv, "bf16")
    plain = q.clone()
    for i in range(len(lens)):
        q[cu[2 * i + 1]:cu[2 * i + 2]] = fill
    dcu = _int(cu)
    first = None
    for x in (plain, q):
        out, lse = hs.chunk_attn_paged(x.to(DEV), got["k"][0], got["v"][0], dcu, _int(kv), table.to(DEV), max_q=130,
                                       max_len=max(kv))
        rows = torch.cat([torch.arange(cu[2 * i], cu[2 * i + 1]) for i in range(len(lens))]).to(DEV)
        first = first or (out[rows], lse[:, rows])
        assert torch.equal(out[rows], first[0]) and torch.equal(lse[:, rows], first[1])
    for i, n in enumerate(lens):
        part = slice(cu[2 * i], cu[2 * i] + n)
        ref.check_attend(f"seq {i}", out[part], lse[:, part],
                         ref.attend(plain[part], got["k"][2][2 * i], got["v"][2][2 * i], SCALE))


@pytest.mark.parametrize("T", [1, 40])
def test_workspace_sized_without_lengths(T):
    """The size for no stated lengths serves calls that state none."""
    gen = torch.Generator().manual_seed(T)
    hq, hkv, n = 4, 1, 6000
    table, got = _paged(gen, [n], 64, hkv, "bf16")
    q = torch.randn(T, hq, 128, generator=gen).to(BF)
    ws = torch.zeros(hs.ragged_workspace_size(1, T, hq, hkv), dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(max_len=0), dict(max_q=0, max_len=0)):
        for w in (ws, None):
            out, lse = _chunk(q, got, ref.cu_of([T]), [n], table, ws=w, **kw)
            _check_all(str(kw), q, got, ref.cu_of([T]), [T], out, lse)
    assert hs.workspace_status(ws) == _lib.HS_OK
    k = torch.randn(T, hkv, 128, generator=gen).to(BF)
    for kw in (dict(), dict(max_len=0)):
        for w in (ws, None):
            out, lse = hs.packed_attn(q.to(DEV), k.to(DEV), k.to(DEV), _int([0, T]), ws=w, **kw)
            ref.check_attend(str(kw), out, lse, ref.attend(q, k, k, SCALE))


@pytest.mark.parametrize("by", [1, 10])
def test_malformed_bounds_are_reported_each_time(by):
    """Every kind of bad bound is reported by the call that met it, and sequences whose own bounds are
    right are the definition's; few rows a sequence, and more."""
    gen = torch.Generator().manual_seed(1)
    hq, hkv, P, kv, T = 2, 1, 16, [40 * by, 33 * by, 20 * by], 7 * by
    table, got = _paged(gen, kv, P, hkv, "bf16", stale=False)
    q = torch.randn(T, hq, 128, generator=gen).to(BF)
    a, b, c, d = 0, 2 * by, 5 * by, 7 * by
    for longest in (max(kv), 64 * max(kv)):
        n = hs.ragged_workspace_size(3, T, hq, hkv, 128, 3 * by, longest)
        for rows, good in (([a, b, c, 900], (0, 1)), ([-4, b, c, d], (1, 2)), ([a, b, 2 ** 31 - 1, d], (0,)),
                           ([-2 ** 31, b, c, d], (1, 2)), ([a, b, c, d + 1], (0, 1))):
            ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
            out, lse = hs.chunk_attn_paged(q.to(DEV), got["k"][0], got["v"][0], _int(rows), _int(kv), table.to(DEV),
                                           max_q=3 * by, max_len=longest, ws=ws)
            assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_ARG, rows
            for i in good:
                part = slice(rows[i], rows[i + 1])
                ref.check_attend(f"{rows} seq {i}", out[part], lse[:, part],
                                 ref.attend(q[part], got["k"][2][i], got["v"][2][i], SCALE))


def test_more_rows_than_announced_are_reported_by_each_kernel():
    gen = torch.Generator().manual_seed(3)
    hq, hkv, P, kv = 2, 1, 16, [40, 33, 20]
    table, got = _paged(gen, kv, P, hkv, "bf16", stale=False)
    q = torch.randn(600, hq, 128, generator=gen).to(BF)
    # 9 tokens of 2 heads where a tile of 8 rows is planned; 3 + 2 items of 128 tokens where one a sequence is
    for most, lens in ((1, [9, 0, 0]), (30, [300, 200, 0])):
        cu = ref.cu_of(lens)
        ws = torch.zeros(hs.ragged_workspace_size(3, sum(lens), hq, hkv, 128, most, 48), dtype=torch.uint8, device=DEV)
        _chunk(q[:sum(lens)], got, cu, kv, table, max_q=most, max_len=48, ws=ws)
        assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_ARG, most
    ws = torch.zeros(hs.ragged_workspace_size(1, 600, hq, 1, 128, 200, 200), dtype=torch.uint8, device=DEV)
    k = torch.randn(600, 1, 128, generator=gen).to(BF)
    hs.packed_attn(q.to(DEV), k.to(DEV), k.to(DEV), _int([0, 600]), max_len=200, ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_ARG
