"""Attention over packed prompts and over paged caches on the GPU, against the
64-bit definition (bounds: ragged_ref.check_attend)."""
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


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ packed prompts

@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (5, 1), (32, 8), (28, 4), (16, 1), (32, 1)])
@pytest.mark.parametrize("lens", [[1], [3, 0, 1, 130], [128], [129, 127, 1], [300, 64, 63, 65, 0], [513]])
def test_packed_matches_definition(lens, hq, hkv):
    """Rows before the first and behind the last sequence hold NaN and must reach nothing."""
    gen = torch.Generator().manual_seed(len(lens) * 1000 + hq)
    lead, tail = 3, 140
    T = lead + sum(lens) + tail
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(BF) for h in (hq, hkv, hkv))
    for x in (q, k, v):
        x[:lead] = math.nan
        x[T - tail:] = math.nan
    cu = ref.cu_of(lens) + lead
    out = torch.full((T, hq, 128), 5.0, dtype=BF, device=DEV)
    lse = torch.full((hq, T), 5.0, device=DEV)
    ws = torch.zeros(hs.ragged_workspace_size(len(lens), T, hq, hkv, 128, max(lens), max(lens)), dtype=torch.uint8,
                     device=DEV)
    hs.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), max_len=max(lens), out=out, lse=lse, ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_OK
    for b, n in enumerate(lens):
        part = slice(int(cu[b]), int(cu[b]) + n)
        ref.check_attend(f"seq {b}", out[part], lse[:, part], ref.attend(q[part], k[part], v[part], SCALE))
    for rest in (slice(0, lead), slice(T - tail, T)):
        assert bool((out[rest] == 5).all()) and bool((lse[:, rest] == 5).all())


def test_packed_sequences_do_not_touch_each_other():
    """NaN and infinities in one sequence's rows stay in that sequence: the rows beside it are those of
    a call without it, bit for bit."""
    gen = torch.Generator().manual_seed(2)
    lens, hq, hkv = [70, 200, 57], 8, 2
    T = sum(lens)
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(BF).to(DEV) for h in (hq, hkv, hkv))
    cu = ref.cu_of(lens).to(DEV)
    clean, clean_lse = hs.packed_attn(q, k, v, cu)
    for x in (k, v):
        x[70:270] = math.nan
        x[100] = math.inf
    out, lse = hs.packed_attn(q, k, v, cu)
    for part in (slice(0, 70), slice(270, T)):
        assert torch.equal(out[part], clean[part]) and torch.equal(lse[:, part], clean_lse[:, part])


def test_packed_slices_of_one_projection_and_scale():
    gen = torch.Generator().manual_seed(4)
    lens, hq, hkv = [33, 90, 5], 6, 3
    T = sum(lens)
    qkv = torch.randn(T, hq + 2 * hkv, 128, generator=gen).to(BF).to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    cu = ref.cu_of(lens).to(DEV)
    out, lse = hs.packed_attn(q, k, v, cu, max_len=90, scale=0.3)
    o2, l2 = hs.packed_attn(q.contiguous(), k.contiguous(), v.contiguous(), cu, scale=0.3)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    for b, n in enumerate(lens):
        part = slice(sum(lens[:b]), sum(lens[:b]) + n)
        # a larger scale makes larger scores: their error bound grows with it
        ref.check_attend(f"seq {b}", out[part], lse[:, part],
                         ref.attend(q[part].cpu(), k[part].cpu(), v[part].cpu(), 0.3), slack=1e-3)


def test_packed_many_sequences():
    """More sequences than one warp looks at in one go, empty ones among them."""
    gen = torch.Generator().manual_seed(6)
    lens = [int(x) for x in torch.randint(0, 9, (300,), generator=gen)]
    lens[200] = 150
    hq, hkv, T = 4, 2, sum(lens)
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(BF) for h in (hq, hkv, hkv))
    cu = ref.cu_of(lens)
    out, lse = hs.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), max_len=150)
    for b, n in enumerate(lens):
        part = slice(int(cu[b]), int(cu[b]) + n)
        ref.check_attend(f"seq {b}", out[part], lse[:, part], ref.attend(q[part], k[part], v[part], SCALE))


@pytest.mark.parametrize("B", [33, 64, 1100, 2500])
def test_packed_more_sequences_than_lanes(B):
    """Batches whose items are found in two steps, with runs of empty sequences, and several items in
    some sequences; rows of a few sequences against the definition, all of them finite."""
    gen = torch.Generator().manual_seed(B)
    lens = [0 if r < 3 else r for r in torch.randint(0, 12, (B,), generator=gen).tolist()]
    lens[B // 2:B // 2 + 40] = [0] * min(40, B - B // 2)
    lens[-1], lens[B // 3], lens[5] = 200, 131, 64
    hq, hkv, T = 4, 1, sum(lens)
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(BF) for h in (hq, hkv, hkv))
    cu = ref.cu_of(lens)
    out = torch.full((T, hq, 128), math.nan, dtype=BF, device=DEV)
    _, lse = hs.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu.to(DEV), max_len=200, out=out)
    assert bool(torch.isfinite(out.float()).all())
    for b in [0, 1, 5, 31, 32, B // 3, B // 2 - 1, min(B // 2 + 40, B - 1), B - 2, B - 1]:
        part = slice(int(cu[b]), int(cu[b]) + lens[b])
        ref.check_attend(f"seq {b}", out[part], lse[:, part], ref.attend(q[part], k[part], v[part], SCALE))


def test_packed_equals_full_layer():
    """Equal prompts: the full layer of the hybrid block, prompt by prompt, to rounding (both round P
    and the output to bf16: twice check_attend's terms)."""
    gen = torch.Generator().manual_seed(8)
    B, L, hq, hkv = 3, 256, 8, 2
    q, k, v = (torch.randn(B, L, h, 128, generator=gen).to(BF).to(DEV) for h in (hq, hkv, hkv))
    full, full_lse, _ = hs.full_attn_scores(q, k, v, want_scores=False)
    out, lse = hs.packed_attn(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), _int([0, L, 2 * L, 3 * L]), max_len=L)
    size = torch.stack([ref.attend(q[b].cpu(), k[b].cpu(), v[b].cpu(), SCALE)[2] for b in range(B)])
    err = (out.view(B, L, hq, 128).double() - full.double()).abs().cpu()
    assert bool((err <= (2 * 2.0 ** -8 + 4e-4) * size + 2 * 2.0 ** -8 * full.double().abs().cpu()).all())
    assert float((lse.view(hq, B, L).transpose(0, 1) - full_lse).abs().max()) <= 2e-4


# ------------------------------------------------------------------ paged caches

def _paged(gen, kv, P, hkv, pool, stale=True):
    """Pools holding kv[b] random rows a sequence; rows behind them (and pages of nobody) are NaN."""
    table, pages = ref.make_table(gen, [-(-n // P) for n in kv])
    got = {}
    for name in ("k", "v"):
        if pool == "bf16":
            pg, sc = torch.full((pages, P, hkv, 128), math.nan if stale else 0.0, dtype=BF), None
        else:
            pg = torch.full((pages, P, hkv, 128), 0x7f if stale else 0, dtype=torch.uint8).view(torch.float8_e4m3fn)
            sc = torch.full((pages, hkv, P), 254 if stale else 127, dtype=torch.uint8)
        rows = []
        for b, n in enumerate(kv):
            x = torch.randn(n, hkv, 128, generator=gen)
            if pool == "e4m3":
                x = x * torch.exp2(torch.randint(-1, 2, (n, 1, 1), generator=gen).float())
                m, e = torch.frexp(x.abs().amax(-1))
                byte = (e - 9 + (m > 0.875).int() + 127) if n else torch.zeros(0, hkv, dtype=torch.int32)
                codes = torch.ldexp(x, -(byte - 127)[..., None]).to(torch.float8_e4m3fn)
                x = codes.float() * torch.exp2(byte.float() - 127)[..., None]
            else:
                x = x.to(BF).float()
            rows.append(x)
            for j in range(n):
                pi, r = int(table[b, j // P]), j % P
                if pool == "e4m3":
                    pg.view(torch.uint8)[pi, r] = codes[j].view(torch.uint8)
                    sc[pi, :, r] = byte[j].to(torch.uint8)
                else:
                    pg[pi, r] = x[j].to(BF)
        got[name] = (pg.to(DEV), None if sc is None else sc.to(DEV), rows)
    return table, got


def _chunk(q, got, cu, kv, table, **kw):
    return hs.chunk_attn_paged(q.to(DEV), got["k"][0], got["v"][0], cu.to(DEV), _int(kv), table.to(DEV),
                               k_scale=got["k"][1], v_scale=got["v"][1], **kw)


def _check_all(name, q, got, cu, new, out, lse, dropped=None):
    for b, n in enumerate(new):
        part = slice(int(cu[b]), int(cu[b]) + n)
        want = ref.attend(q[part], got["k"][2][b], got["v"][2][b], SCALE, dropped=() if dropped is None else dropped[b])
        ref.check_attend(f"{name} seq {b}", out[part], lse[:, part], want)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [16, 64, 128, 256, 8, 4, 2, 1])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 1), (7, 1)])
def test_chunk_matches_definition(hq, hkv, P, pool):
    """One token, none, chunks within and over a tile, a first chunk with nothing cached."""
    gen = torch.Generator().manual_seed(P * 10 + hq)
    new = [1, 0, 5, 40, 1, 129, 1]
    old = [0, 50, 123, 200, 127, 0, 300]
    kv = [a + b for a, b in zip(new, old)]
    table, got = _paged(gen, kv, P, hkv, pool)
    T = sum(new) + 2
    q = torch.randn(T, hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new) + 1
    out = torch.full((T, hq, 128), 5.0, dtype=BF, device=DEV)
    lse = torch.full((hq, T), 5.0, device=DEV)
    ws = torch.zeros(hs.ragged_workspace_size(len(new), T, hq, hkv, 128, max(new), max(kv)), dtype=torch.uint8, device=DEV)
    _chunk(q, got, cu, kv, table, max_q=max(new), max_len=max(kv), out=out, lse=lse, ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_OK
    _check_all(f"P {P}", q, got, cu, new, out, lse)
    assert bool((out[0] == 5).all()) and bool((out[-1] == 5).all()) and bool((lse[:, [0, T - 1]] == 5).all())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [64, 16, 8, 4, 2, 1])
@pytest.mark.parametrize("hq,hkv,most", [(8, 2, 1), (3, 1, 2), (16, 1, 1), (5, 5, 3), (7, 1, 2), (32, 8, 4), (64, 2, 1),
                                         (8, 2, 16), (12, 4, 7)])
def test_chunk_few_rows_match_definition(hq, hkv, most, P, pool):
    """Decode steps and short chunks: few rows a sequence, one and several 16-row tiles of them, caches
    that end before, at and behind a 16-key block, empty sequences and caches shorter than the chunk."""
    gen = torch.Generator().manual_seed(P * 100 + hq + most)
    new = [most, 0, 1, most, 1, min(2, most), most]
    kv = [most, 5, 16, 33 + most, 17, 1, 300 + most]
    table, got = _paged(gen, kv, P, hkv, pool)
    T = sum(new) + 2
    q = torch.randn(T, hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new) + 1
    out = torch.full((T, hq, 128), 5.0, dtype=BF, device=DEV)
    lse = torch.full((hq, T), 5.0, device=DEV)
    ws = torch.zeros(hs.ragged_workspace_size(len(new), T, hq, hkv, 128, most, 4096), dtype=torch.uint8, device=DEV)
    _chunk(q, got, cu, kv, table, max_q=most, max_len=4096, out=out, lse=lse, ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_OK
    _check_all(f"P {P}", q, got, cu, new, out, lse)
    assert bool((out[0] == 5).all()) and bool((out[-1] == 5).all()) and bool((lse[:, [0, T - 1]] == 5).all())
    assert bool(torch.isfinite(out.float()).all())


@pytest.mark.parametrize("new", [[1, 1], [90, 1]])
def test_chunk_8bit_scales_far_apart(new):
    """Scales over the whole range in one cache: keys whose scores vanish beside others', values a
    million times larger than their neighbours' on keys that count and on keys that do not.  Queries
    from 2^-30 to 2^30 of the usual size meet keys scaled the other way."""
    gen = torch.Generator().manual_seed(5)
    hq, hkv, P, old = 4, 2, 16, [400, 333]
    kv = [a + b for a, b in zip(new, old)]
    table, pages = ref.make_table(gen, [-(-n // P) for n in kv])
    pools = {}
    for name in ("k", "v"):
        codes = torch.randn(pages, P, hkv, 128, generator=gen).mul_(8).to(torch.float8_e4m3fn)
        byte = torch.full((pages, hkv, P), 124, dtype=torch.uint8)
        if name == "v":
            pick = torch.randint(0, 60, byte.shape, generator=gen)
            byte[pick == 0] = 144                  # 2^20 above
            byte[pick == 1] = 100
            byte[pick == 2] = 1
        else:
            pick = torch.randint(0, 60, byte.shape, generator=gen)
            byte[pick == 0] = 1
            byte[pick == 1] = 90
        pools[name] = (codes, byte)
    for shift in (0, -30, 30):
        q = (torch.randn(sum(new), hq, 128, generator=gen) * 2.0 ** shift).to(BF)
        got, rows = {}, {}
        for name, (codes, byte) in pools.items():
            b = (byte.int() - shift).clamp(1, 254).to(torch.uint8) if name == "k" else byte
            got[name] = (codes.to(DEV), b.to(DEV), [ref.rows_of(codes, table[i], 0, n, b) for i, n in enumerate(kv)])
        cu = ref.cu_of(new)
        out, lse = _chunk(q, got, cu, kv, table, max_q=max(new), max_len=max(kv))
        for b, n in enumerate(new):
            part = slice(int(cu[b]), int(cu[b]) + n)
            ref.check_attend(f"shift {shift} seq {b}", out[part], lse[:, part],
                             ref.attend(q[part], got["k"][2][b], got["v"][2][b], SCALE), slack=1e-4)


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("new,old", [([1], [5000]), ([1, 1, 1], [3000, 0, 40]), ([40], [4100]), ([300, 2], [1500, 3500]),
                                     ([1], [16383])])
def test_chunk_long_caches_split(new, old, pool):
    """Few rows, many keys: the keys are split over CTAs and the pieces joined.  How they are split is
    planned from max_len; a cache longer than planned for is still right."""
    gen = torch.Generator().manual_seed(sum(old))
    hq, hkv, P = 8, 2, 64
    kv = [a + b for a, b in zip(new, old)]
    table, got = _paged(gen, kv, P, hkv, pool)
    q = torch.randn(sum(new), hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new)
    for longest in (max(kv), max(kv) // 3, 16 * max(kv)):
        n = hs.ragged_workspace_size(len(new), sum(new), hq, hkv, 128, max(new), longest)
        ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
        out, lse = _chunk(q, got, cu, kv, table, max_q=max(new), max_len=longest, ws=ws)
        assert hs.workspace_status(ws) == _lib.HS_OK
        _check_all(f"planned for {longest}", q, got, cu, new, out, lse)
    assert hs.ragged_workspace_size(len(new), sum(new), hq, hkv, 128, max(new), max(kv)) > 256


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_chunk_rows_that_see_nothing(pool):
    """A cache shorter than the chunk: the first rows see nothing and give zeros and -inf; an empty
    cache gives only such rows."""
    gen = torch.Generator().manual_seed(12)
    new, kv, hq, hkv = [6, 3, 140], [4, 0, 139], 4, 2
    table, got = _paged(gen, kv, 16, hkv, pool)
    q = torch.randn(sum(new), hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new)
    for longest in (max(kv), 8192):
        out, lse = _chunk(q, got, cu, kv, table, max_q=140, max_len=longest)
        _check_all("short cache", q, got, cu, new, out, lse)
    assert bool((out[:2] == 0).all()) and bool((out[6:9] == 0).all()) and bool(torch.isinf(lse[:, 6:9]).all())


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [2, 16, 128])
def test_chunk_drops_pages_outside_the_pool(P, pool):
    gen = torch.Generator().manual_seed(P)
    new, old, hq, hkv = [1, 30, 2], [700, 200, 60], 4, 2
    kv = [a + b for a, b in zip(new, old)]
    table, got = _paged(gen, kv, P, hkv, pool)
    dropped = [set(), set(), set()]
    for b, pg, bad in ((0, 1, -1), (0, 170 // P, 2 ** 31 - 1), (1, 0, got["k"][0].shape[0]), (2, 30 // P, -7)):
        table[b, pg] = bad
        dropped[b] |= set(range(pg * P, min((pg + 1) * P, kv[b])))
    q = torch.randn(sum(new), hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new)
    ws = torch.zeros(hs.ragged_workspace_size(3, sum(new), hq, hkv, 128, 30, max(kv)), dtype=torch.uint8, device=DEV)
    out, lse = _chunk(q, got, cu, kv, table, max_q=30, max_len=max(kv), ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_INDEX
    _check_all("bad pages", q, got, cu, new, out, lse, dropped=[sorted(d) for d in dropped])


def test_chunk_bad_lengths_are_reported():
    """Lengths that would leave the buffers are clamped and reported; the sequences beside them are
    right."""
    gen = torch.Generator().manual_seed(1)
    new, kv, hq, hkv, P = [2, 3, 2], [40, 33, 20], 2, 1, 16
    table, got = _paged(gen, kv, P, hkv, "bf16", stale=False)
    q = torch.randn(sum(new), hq, 128, generator=gen).to(BF)
    cu = ref.cu_of(new)
    ws = torch.zeros(hs.ragged_workspace_size(3, 7, hq, hkv, 128, 3, 48), dtype=torch.uint8, device=DEV)
    for bad in (1000, -5, 2 ** 31 - 1, -2 ** 31):
        out, lse = _chunk(q, got, cu, [bad, 33, 20], table, max_q=3, max_len=48, ws=ws)
        assert hs.workspace_status(ws) in ((_lib.HS_ERR_INVALID_ARG, _lib.HS_ERR_INVALID_INDEX))
        for b in (1, 2):
            part = slice(int(cu[b]), int(cu[b]) + new[b])
            ref.check_attend(f"beside {bad}", out[part], lse[:, part],
                             ref.attend(q[part], got["k"][2][b], got["v"][2][b], SCALE))
    for rows in ([0, 2, 5, 900], [0, 2, 5, -3], [0, 2 ** 31 - 1, 5, 7], [-4, 2, 5, 7], [0, 5, 2, 7]):
        out, lse = hs.chunk_attn_paged(q.to(DEV), got["k"][0], got["v"][0], _int(rows), _int(kv), table.to(DEV), max_q=3,
                                       max_len=48, ws=ws)
        hs.workspace_status(ws)
    # more rows in a sequence than the call said: reported
    _chunk(q, got, ref.cu_of([7, 0, 0]), kv, table, max_q=1, max_len=48, ws=ws)
    small = torch.randn(600, hq, 128, generator=gen).to(BF)
    hs.packed_attn(small.to(DEV), small[:, :1].to(DEV), small[:, :1].to(DEV), _int([0, 600]), max_len=200, ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_ARG


def test_attention_on_another_stream_and_in_a_graph():
    """The same bits on another stream and from a captured graph replayed over new contents (its
    lengths too: they live on the device)."""
    gen = torch.Generator().manual_seed(31)
    new, hq, hkv, P = [1, 1, 1, 1], 8, 2, 32
    kv = [2000, 77, 1, 900]
    table, got = _paged(gen, [2048] * 4, P, hkv, "bf16", stale=False)
    q = torch.randn(4, hq, 128, generator=gen).to(BF).to(DEV)
    cu, dkv, dt = ref.cu_of(new).to(DEV), _int(kv), table.to(DEV)
    ws = torch.zeros(hs.ragged_workspace_size(4, 4, hq, hkv, 128, 1, 2048), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(hq, 4, device=DEV)

    def go(o, l):
        return hs.chunk_attn_paged(q, got["k"][0], got["v"][0], cu, dkv, dt, max_q=1, max_len=2048, out=o, lse=l, ws=ws)
    go(out, lse)
    first = out.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o2, l2 = go(torch.empty_like(out), torch.empty_like(lse))
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(out, lse)
    for lens in ([3, 2048, 500, 129], [1, 1, 1, 1]):
        dkv.copy_(_int(lens))
        q.copy_(torch.randn(4, hq, 128, generator=gen))
        g.replay()
        got_o, got_l = out.clone(), lse.clone()
        go(out, lse)
        assert torch.equal(got_o, out) and torch.equal(got_l, lse)
        for b in range(4):
            ref.check_attend(f"replay seq {b}", got_o[b:b + 1], got_l[:, b:b + 1],
                             ref.attend(q[b:b + 1].cpu(), got["k"][2][b][:lens[b]], got["v"][2][b][:lens[b]], SCALE))
    assert hs.workspace_status(ws) == _lib.HS_OK and not torch.equal(first, out)


def test_wait_limit_marks_lse(monkeypatch):
    """A wait that gives up (the limit set to nothing) is reported and its rows' lse is NaN."""
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(300, h, 128, generator=gen).to(BF).to(DEV) for h in (4, 1, 1))
    ws = torch.zeros(hs.ragged_workspace_size(1, 300, 4, 1, 128, 300, 300), dtype=torch.uint8, device=DEV)
    monkeypatch.setenv("HYSPARSE_WAIT_LIMIT_NS", "0")
    _, lse = hs.packed_attn(q, k, v, _int([0, 300]), ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_ERR_TIMEOUT and bool(torch.isnan(lse).any())
    monkeypatch.delenv("HYSPARSE_WAIT_LIMIT_NS")
    _, lse = hs.packed_attn(q, k, v, _int([0, 300]), ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_OK and bool(torch.isfinite(lse).all())


# ------------------------------------------------------------------ used together

def test_prompt_in_chunks_then_decode_over_the_same_pages():
    """Two prompts rotated, written and attended chunk by chunk over their pages equal their packed
    prefill (to rounding), and block_paged then decodes over the same pages: its full layer is the
    one-token chunk's."""
    gen = torch.Generator().manual_seed(77)
    hq, hkv, P, lens, k_top, window = 8, 2, 16, [150, 61], 32, 16
    T = sum(lens)
    f, _ = hs.rope_frequencies(128, device=DEV)
    qkv = torch.randn(T, hq + 2 * hkv, 128, generator=gen).to(BF).to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(DEV)
    rq, rk = hs.rope(q, pos, f, k=k)
    want, want_lse = hs.packed_attn(rq, rk, v, ref.cu_of(lens).to(DEV), max_len=max(lens))
    table, pages = ref.make_table(gen, [-(-(n + 1) // P) for n in lens])
    dt = table.to(DEV)
    pk, pv = (torch.zeros(pages, P, hkv, 128, dtype=BF, device=DEV) for _ in range(2))
    done = [0, 0]
    size = torch.cat([ref.attend(rq[a:a + n].cpu(), rk[a:a + n].cpu(), v[a:a + n].cpu(), SCALE)[2]
                      for a, n in ((0, lens[0]), (lens[0], lens[1]))])
    for step in ([64, 61], [50, 0], [36, 0]):
        rows = torch.cat([torch.arange(sum(lens[:b]) + done[b], sum(lens[:b]) + done[b] + n) for b, n in enumerate(step)])
        done = [a + b for a, b in zip(done, step)]
        cu, kv = ref.cu_of(step).to(DEV), _int(done)
        hs.cache_write(k[rows], v[rows], pk, pv, cu, kv, dt, inv_freq=f)
        out, lse = hs.chunk_attn_paged(rq[rows], pk, pv, cu, kv, dt, max_q=max(step))
        err = (out.double() - want[rows].double()).abs().cpu()
        assert bool((err <= (2 * 2.0 ** -8 + 4e-4) * size[rows] + 2 * 2.0 ** -8 * want[rows].double().abs().cpu()).all())
        assert float((lse - want_lse[:, rows]).abs().max()) <= 2e-4
    back_k, back_v = hs.cache_read(pk, pv, ref.cu_of(lens).to(DEV), dt, total=T)
    assert torch.equal(back_k, rk) and torch.equal(back_v, v.contiguous())
    # one decode step: the new token's key and value, then the hybrid block over the pages
    x = torch.randn(2, hq + 2 * hkv, 128, generator=gen).to(BF).to(DEV)
    kv = _int([n + 1 for n in lens])
    cu = _int([0, 1, 2])
    hs.cache_write(x[:, hq:hq + hkv], x[:, hq + hkv:], pk, pv, cu, kv, dt, inv_freq=f)
    dq = hs.rope(x[:, :hq], _int(lens), f)
    one, one_lse = hs.chunk_attn_paged(dq, pk, pv, cu, kv, dt, max_q=1)
    qs = [torch.randn(2, 1, hq, 128, generator=gen).to(BF).to(DEV)]
    gate = [torch.randn(2, 1, hq, generator=gen).to(DEV)]
    full, full_lse, _, _ = hs.block_paged(dq.view(2, 1, hq, 128), pk, pv, qs, gate, k_top, window, kv, dt)
    for b in range(2):
        n = lens[b] + 1
        rows = [ref.rows_of(pg.cpu(), table[b], 0, n) for pg in (pk, pv)]
        w = ref.attend(dq[b:b + 1].cpu(), rows[0], rows[1], SCALE)
        ref.check_attend(f"chunk {b}", one[b:b + 1], one_lse[:, b:b + 1], w)
        ref.check_attend(f"block {b}", full[b], full_lse[b], w)


# ------------------------------------------------------------------ NaN in what is seen

@pytest.mark.parametrize("where", ["k", "q", "v"])
@pytest.mark.parametrize("new", [[2, 1, 2], [150, 3, 1], [1, 1, 1]])
@pytest.mark.parametrize("pool", ["bf16", "e4m3", "packed"])
def test_nan_reaches_the_rows_that_see_it_and_no_others(pool, new, where):
    """One NaN in sequence 0: a key's makes the rows from its position on NaN, a query's its own row and
    head, a value's its column (8-bit: all of them) in those rows.  Earlier rows are as ever (but for that column, within a tile),
    and so are the other sequences'."""
    gen = torch.Generator().manual_seed(77 + len(where) + sum(new))
    hq, hkv, P = 8, 2, 16
    old = [0, 0, 0] if pool == "packed" else [300, 20, 129]
    kv = [a + b for a, b in zip(new, old)]
    g, row, head, col = 1, new[0] // 2, 5, 37            # head 5 belongs to KV head 1
    at = old[0] + row                                    # the position hit
    T, cu = sum(new), ref.cu_of(new)
    q = torch.randn(T, hq, 128, generator=gen).to(BF)
    if pool == "packed":
        rows = {n: torch.randn(T, hkv, 128, generator=gen).to(BF) for n in "kv"}
        got = {n: (None, None, [rows[n][int(cu[b]):int(cu[b + 1])].float() for b in range(3)]) for n in "kv"}
    else:
        table, got = _paged(gen, kv, P, hkv, pool)
    qx = q.clone()
    if where == "q":
        qx[row, head, col] = math.nan
    elif pool == "packed":
        rows[where][at, g, col] = math.nan
    elif pool == "bf16":
        got[where][0][int(table[0, at // P]), at % P, g, col] = math.nan
    else:
        got[where][0].view(torch.uint8)[int(table[0, at // P]), at % P, g] = 0x7f     # a row of NaN
        got[where][1][int(table[0, at // P]), g, at % P] = 255
    if pool == "packed":
        out, lse = hs.packed_attn(qx.to(DEV), rows["k"].to(DEV), rows["v"].to(DEV), cu.to(DEV), max_len=max(new))
    else:
        out, lse = _chunk(qx, got, cu, kv, table, max_q=max(new), max_len=max(kv))
    out, lse = out.cpu(), lse.cpu()
    want = [ref.attend(q[int(cu[b]):int(cu[b + 1])], got["k"][2][b], got["v"][2][b], SCALE) for b in range(3)]
    for b in (1, 2):
        part = slice(int(cu[b]), int(cu[b + 1]))
        ref.check_attend(f"seq {b}", out[part], lse[:, part], want[b])
    n = new[0]
    heads = [head] if where == "q" else list(range(g * 4, g * 4 + 4))
    hit = torch.zeros(n, hq, dtype=torch.bool)
    for h in heads:
        hit[row:(row + 1 if where == "q" else n), h] = True
    if where == "v":
        cols = slice(col, col + 1) if pool != "e4m3" else slice(0, 128)
        assert bool(torch.isnan(out[:n, :, cols][hit]).all())
        got_o = out[:n].clone()
        got_o[:, heads, cols] = want[0][0][:, heads, cols].to(BF)
        ref.check_attend("other columns", got_o, lse[:, :n], want[0])
        return
    assert bool(torch.isnan(out[:n][hit]).all()) and bool(torch.isnan(lse[:, :n].t()[hit]).all())
    o, l = out[:n].clone(), lse[:, :n].clone()
    o[hit] = want[0][0][hit].to(BF)
    l.t()[hit] = want[0][1].t()[hit].float()
    ref.check_attend("rows that do not see it", o, l, want[0])


# ------------------------------------------------------------------ calls at their limits

@pytest.mark.parametrize("pool,new", [("e4m3", [90, 40]), ("e4m3", [20, 12]), ("bf16", [20, 12])])
def test_wait_limit_marks_lse_of_chunks(monkeypatch, pool, new):
    """As test_wait_limit_marks_lse, for two row tiles, for one that both warpgroups share, and for 8-bit pages."""
    gen = torch.Generator().manual_seed(6)
    kv = [n + 700 for n in new]
    table, got = _paged(gen, kv, 64, 2, pool)
    cu, T = ref.cu_of(new), sum(new)
    q = torch.randn(T, 8, 128, generator=gen).to(BF)
    ws = torch.zeros(hs.ragged_workspace_size(2, T, 8, 2, 128, max(new), max(kv)), dtype=torch.uint8, device=DEV)
    monkeypatch.setenv("HYSPARSE_WAIT_LIMIT_NS", "0")
    _, lse = _chunk(q, got, cu, kv, table, max_q=max(new), max_len=max(kv), ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_ERR_TIMEOUT and bool(torch.isnan(lse).any())
    monkeypatch.delenv("HYSPARSE_WAIT_LIMIT_NS")
    out, lse = _chunk(q, got, cu, kv, table, max_q=max(new), max_len=max(kv), ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_OK
    _check_all("after", q, got, cu, new, out, lse)


def test_two_threads_call_at_once():
    """Each on a stream of its own, the library called without the interpreter's lock."""
    import threading
    gen = torch.Generator().manual_seed(8)
    new, old, hq, hkv = [1, 30, 1], [400, 90, 2000], 8, 2
    kv = [a + b for a, b in zip(new, old)]
    table, got = _paged(gen, kv, 16, hkv, "e4m3")
    cu, T = ref.cu_of(new), sum(new)
    q = [torch.randn(T, hq, 128, generator=gen).to(BF).to(DEV) for _ in range(2)]
    dcu, dkv, dt = cu.to(DEV), _int(kv), table.to(DEV)

    def go(i):
        return hs.chunk_attn_paged(q[i], got["k"][0], got["v"][0], dcu, dkv, dt, max_q=max(new), max_len=max(kv),
                                   k_scale=got["k"][1], v_scale=got["v"][1])
    want = [go(i) for i in range(2)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            for _ in range(50):
                out, lse = go(i)
                st.synchronize()
                if not (torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])):
                    bad.append(i)
                    return
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("pool", ["bf16", "e4m3"])
def test_pools_past_32_bits(pool):
    """Pools of more than 2^32 elements, their last and first pages in use."""
    gen = torch.Generator().manual_seed(9)
    hq, hkv, P, pages, n = 8, 8, 64, 66000, 300
    assert pages * P * hkv * 128 > 1 << 32
    dtype = BF if pool == "bf16" else torch.float8_e4m3fn
    pk, pv = (torch.empty(pages, P, hkv, 128, dtype=dtype, device=DEV) for _ in range(2))
    sc = {} if pool == "bf16" else {x: torch.zeros(pages, hkv, P, dtype=torch.uint8, device=DEV)
                                    for x in ("k_scale", "v_scale")}
    table = _int([[pages - 1, 0, pages - 2, 65537, pages - 3]])
    k, v = (torch.randn(n, hkv, 128, generator=gen).to(BF) for _ in range(2))
    hs.cache_write(k.to(DEV), v.to(DEV), pk, pv, _int([0, n]), _int([n]), table, **sc)
    bk, bv = (x.cpu() for x in hs.cache_read(pk, pv, _int([0, n]), table, total=n, **sc))
    for got, x in ((bk, k), (bv, v)):
        if pool == "bf16":
            assert torch.equal(got, x)
        else:
            codes, byte = ref.e4m3(x.double())
            assert torch.equal(got.double(), codes * torch.exp2(byte.double() - 127)[..., None])
    for rows in (1, 5, 100):
        q = torch.randn(rows, hq, 128, generator=gen).to(BF)
        out, lse = hs.chunk_attn_paged(q.to(DEV), pk, pv, _int([0, rows]), _int([n]), table, max_q=rows, max_len=n, **sc)
        ref.check_attend(f"{rows} rows", out, lse, ref.attend(q, bk, bv, SCALE))


def test_rows_past_32_bits():
    """Packed rows of more than 2^31 elements: rotated in place, attended, the last sequences checked."""
    gen = torch.Generator().manual_seed(10)
    hq, hkv, n, B = 256, 8, 97, 700
    T = n * B
    assert T * hq * 128 > 1 << 31
    f, _ = hs.rope_frequencies(128, device=DEV)
    q = torch.zeros(T, hq, 128, dtype=BF, device=DEV)
    k, v = (torch.zeros(T, hkv, 128, dtype=BF, device=DEV) for _ in range(2))
    part = slice(T - 2 * n, T)
    tail = [torch.randn(2 * n, h, 128, generator=gen).to(BF) for h in (hq, hkv, hkv)]
    for x, y in zip((q, k, v), tail):
        x[part] = y.to(DEV)
    pos = torch.arange(n, dtype=torch.int32).repeat(B).to(DEV)
    wq, wk = hs.rope(q[part].clone(), pos[part].contiguous(), f, k=k[part].clone())
    hs.rope(q, pos, f, k=k, out=q, out_k=k)
    assert torch.equal(q[part], wq) and torch.equal(k[part], wk)
    out, lse = hs.packed_attn(q, k, v, torch.arange(B + 1, dtype=torch.int32, device=DEV) * n, max_len=n)
    heads = list(range(0, hq, 51))
    for b in range(2):
        rows = slice(b * n, (b + 1) * n)
        want = ref.attend(wq[rows].cpu(), wk[rows].cpu(), tail[2][rows], SCALE)
        at = slice(T - 2 * n + b * n, T - 2 * n + (b + 1) * n)
        ref.check_attend(f"seq {B - 2 + b}", out[at][:, heads], lse[heads][:, at],
                         (want[0][:, heads], want[1][heads], want[2][:, heads]))


def test_binding_refusals():
    """Shapes, types and strides that the calls do not take raise before anything runs."""
    q, k, v = (torch.zeros(6, h, 128, dtype=BF, device=DEV) for h in (4, 2, 2))
    cu, kv, table = _int([0, 4, 6]), _int([4, 2]), _int([[0, 1], [2, 3]])
    pk, pv = (torch.zeros(4, 16, 2, 128, dtype=BF, device=DEV) for _ in range(2))
    f, _ = hs.rope_frequencies(128, device=DEV)
    p8, s8 = torch.zeros(4, 16, 2, 128, device=DEV).to(torch.float8_e4m3fn), torch.ones(4, 2, 16, dtype=torch.uint8, device=DEV)
    pos = _int(list(range(6)))
    wrong = (TypeError, ValueError)
    for call in (
            lambda: hs.rope(q, pos.long(), f), lambda: hs.rope(q, pos[:5], f), lambda: hs.rope(q, pos, f.float()),
            lambda: hs.rope(q.half(), pos, f), lambda: hs.rope(q[0], pos, f), lambda: hs.rope(q, pos, f, k=k[:5]),
            lambda: hs.rope(q, pos, f, out=q[:, :2]), lambda: hs.rope(q, pos, f, out_k=k),
            lambda: hs.rope(q[:, ::2], pos, f), lambda: hs.rope(q[..., :64], pos, f), lambda: hs.rope(q, pos.cpu(), f),
            lambda: hs.rope(q, pos, f, factor="a"), lambda: hs.rope(None, pos, f),
            lambda: hs.cache_write(k, v[:5], pk, pv, cu, kv, table), lambda: hs.cache_write(k, v.float(), pk, pv, cu, kv, table),
            lambda: hs.cache_write(k, v, pk, pv[:3], cu, kv, table), lambda: hs.cache_write(k, v, pk, pv, cu[:2], kv, table),
            lambda: hs.cache_write(k, v, pk, pv, cu, kv.long(), table), lambda: hs.cache_write(k, v, pk, pv, cu, kv, table[0]),
            lambda: hs.cache_write(k, v, p8, p8, cu, kv, table), lambda: hs.cache_write(k, v, pk, pv, cu, kv, table, k_scale=s8),
            lambda: hs.cache_write(k, v, p8, p8, cu, kv, table, k_scale=s8, v_scale=s8[:, :, :8]),
            lambda: hs.cache_write(k, v, pk.transpose(1, 2), pv.transpose(1, 2), cu, kv, table),
            lambda: hs.cache_write(k, v, pk, pv, cu, kv, table, ws=torch.zeros(8, device=DEV)),
            lambda: hs.cache_write(k, v, pk, pv, cu, kv, table, inv_freq=torch.cat([f, f])),
            lambda: hs.cache_read(pk, pv, cu, table, total=-1), lambda: hs.cache_read(pk, pv, cu, table, total=6, dtype=torch.half),
            lambda: hs.cache_read(pk, pv, cu, table, total=6, start=_int([0])), lambda: hs.cache_read(pk, pv, cu, table, total=2 ** 40),
            lambda: hs.cache_read(pk, pv, cu, table, total=6, out_k=torch.zeros(6, 2, 128, device=DEV)),
            lambda: hs.packed_attn(q.float(), k, v, cu), lambda: hs.packed_attn(q, k.float(), v.float(), cu),
            lambda: hs.packed_attn(q, k[:5], v[:5], cu), lambda: hs.packed_attn(q, k, v, cu[:1]),
            lambda: hs.packed_attn(q, k, v, cu, max_len=2 ** 35), lambda: hs.packed_attn(q, k, v, cu, out=q.float()),
            lambda: hs.packed_attn(q, k, v, cu, lse=torch.zeros(6, 4, device=DEV)), lambda: hs.packed_attn(q, k, v, cu.cpu()),
            lambda: hs.chunk_attn_paged(q.float(), pk, pv, cu, kv, table), lambda: hs.chunk_attn_paged(q[..., :64], pk, pv, cu, kv, table),
            lambda: hs.chunk_attn_paged(q, p8, p8, cu, kv, table), lambda: hs.chunk_attn_paged(q, pk, pv, cu, kv[:1], table),
            lambda: hs.chunk_attn_paged(q, pk, pv, cu, kv, table, out=q[:5])):
        with pytest.raises(wrong):
            call()
    for call in (lambda: hs.packed_attn(q, k, v, cu, out=q), lambda: hs.packed_attn(q, k, v, cu, max_len=-1),
                 lambda: hs.packed_attn(q, k, v, cu, ws=torch.zeros(256, dtype=torch.uint8, device=DEV)[1:]),
                 lambda: hs.chunk_attn_paged(q, pk.float(), pv.float(), cu, kv, table),
                 lambda: hs.rope(q, pos, f, factor=math.inf)):
        with pytest.raises(hs.HysparseError):
            call()


def test_no_rows():
    """Batches of no rows at all, and of sequences without rows."""
    q, k = torch.zeros(0, 4, 128, dtype=BF, device=DEV), torch.zeros(0, 2, 128, dtype=BF, device=DEV)
    pk, pv = (torch.full((3, 16, 2, 128), 5.0, dtype=BF, device=DEV) for _ in range(2))
    cu, kv, table = _int([0, 0, 0]), _int([0, 7]), _int([[0], [1]])
    f, _ = hs.rope_frequencies(128, device=DEV)
    rq, rk = hs.rope(q, _int([]), f, k=k)
    assert rq.shape == q.shape and rk.shape == k.shape
    hs.cache_write(k, k, pk, pv, cu, kv, table, inv_freq=f)
    back = hs.cache_read(pk, pv, cu, table, total=0)
    assert back[0].shape == (0, 2, 128)
    for out, lse in (hs.packed_attn(q, k, k, cu), hs.chunk_attn_paged(q, pk, pv, cu, kv, table)):
        assert out.shape == q.shape and lse.shape == (4, 0)
    # rows that belong to no sequence only
    q, k = torch.zeros(9, 4, 128, dtype=BF, device=DEV), torch.zeros(9, 2, 128, dtype=BF, device=DEV)
    out, lse = torch.full_like(q, 3.0), torch.full((4, 9), 3.0, device=DEV)
    hs.cache_write(k, k, pk, pv, cu, kv, table, inv_freq=f)
    for most in (1, 9):
        hs.chunk_attn_paged(q, pk, pv, cu, kv, table, max_q=most, out=out, lse=lse)
    hs.packed_attn(q, k, k, cu, out=out, lse=lse)
    assert bool((pk == 5).all()) and bool((out == 3).all()) and bool((lse == 3).all())
