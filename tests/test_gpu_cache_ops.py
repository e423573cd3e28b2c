"""Rotary positions and the paged cache's write and read on the GPU, against
their definitions in 64 bits.

Tolerances.  A rotated element is fl(fl(x c) - fl(y s)) with c and s rounded
to fp32 (and by the amplitude's product once more): four roundings of at most
2^-24 on each term, so |error| <= 4 * 2^-24 * (|x| + |y|) * factor, the angle
itself being good to 1e-9 at these positions (64-bit product, whole turns
taken out).  A bf16 result adds half a bf16 step, 2^-8 of the value.  8-bit
codes of rows that were not rotated are exact: dividing by a power of two is,
and the rounding to the nearest code is the operation's definition."""
import math

import pytest
import torch

import hybrid_sparse_attention_tcgen05_b200 as hs
from hybrid_sparse_attention_tcgen05_b200 import _lib
import ragged_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _close_rope(got, x, want, n, interleaved, factor, dtype):
    amax = x.double().abs()
    i0 = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    i1 = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    tol = torch.zeros_like(want)
    pair = (amax[..., i0] + amax[..., i1]) * (4 * 2.0 ** -24 + 1e-9) * abs(factor)
    tol[..., i0] = pair
    tol[..., i1] = pair
    if dtype == "bf16":
        tol[..., :2 * n] += want[..., :2 * n].abs() * 2.0 ** -8 * (1 + 1e-6) + 1e-38
    bad = (got.double().cpu() - want).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} elements off, worst {float((got.double().cpu() - want).abs().max())}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot", [(1, 1, 1, 8, 2), (3, 4, 1, 64, 64), (65, 5, 5, 96, 24), (17, 32, 8, 128, 128),
                                            (33, 2, 1, 128, 70), (5, 3, 1, 256, 64), (4099, 2, 1, 64, 48)])
def test_rope_matches_definition(T, Hq, Hkv, d, rot, interleaved, dtype):
    gen = torch.Generator().manual_seed(T * 131 + d + rot)
    q = torch.randn(T, Hq, d, generator=gen).to(DT[dtype])
    k = torch.randn(T, Hkv, d, generator=gen).to(DT[dtype])
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen, dtype=torch.int32)
    pos[-1] = (1 << 31) - 1 if T > 3 else 0
    f, _ = hs.rope_frequencies(rot, device=DEV)
    for inverse, factor in ((False, 1.0), (True, 1.3466)):
        oq, ok = hs.rope(q.to(DEV), pos.to(DEV), f, k=k.to(DEV), interleaved=interleaved, inverse=inverse, factor=factor)
        for got, x in ((oq, q), (ok, k)):
            # the last position is past what the tolerance's angle error allows for
            want = ref.rope(x, pos, f.cpu(), interleaved, inverse, torch.tensor(factor).float().double().item())
            n = T - 1 if T > 3 else T
            _close_rope(got[:n], x[:n], want[:n], rot // 2, interleaved, factor, dtype)
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])
            assert bool(torch.isfinite(got.float()).all())


def test_rope_in_place_slices_and_streams():
    """Slices of one projection, turned in place, equal the packed call; v's part of the projection
    and nothing else stays as it was; another stream than the default one gives the same bits."""
    T, Hq, Hkv, d = 77, 6, 2, 128
    qkv = torch.randn(T, (Hq + 2 * Hkv) * d, device=DEV).to(torch.bfloat16)
    before = qkv.clone()
    q = qkv[:, :Hq * d].unflatten(1, (Hq, d))
    k = qkv[:, Hq * d:(Hq + Hkv) * d].unflatten(1, (Hkv, d))
    pos = torch.arange(1000, 1000 + T, device=DEV, dtype=torch.int32)
    for rot in (d, 32):
        f, _ = hs.rope_frequencies(rot, device=DEV)
        qkv.copy_(before)
        wq, wk = hs.rope(q.contiguous(), pos, f, k=k.contiguous())
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            hs.rope(q, pos, f, k=k, out=q, out_k=k)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(q, wq) and torch.equal(k, wk)
        assert torch.equal(qkv[:, (Hq + Hkv) * d:], before[:, (Hq + Hkv) * d:])
        only_q = hs.rope(before[:, :Hq * d].unflatten(1, (Hq, d)), pos, f)
        assert torch.equal(only_q, wq)
    empty = hs.rope(torch.empty(0, Hq, d, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), f)
    assert tuple(empty.shape) == (0, Hq, d)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(interleaved):
    """The inverse call is the transposed map: <R x, w> = <x, R^T w>, and it agrees with central
    differences of <R x, w>, which is linear in x, so that a difference over a step of 1 is its
    derivative up to rounding: 2 * d products of size ~1 in fp32, summed in 64 bits."""
    T, H, d, rot = 9, 2, 64, 48
    gen = torch.Generator().manual_seed(3)
    x, w = torch.randn(T, H, d, generator=gen), torch.randn(T, H, d, generator=gen)
    pos = torch.randint(0, 5000, (T,), generator=gen, dtype=torch.int32).to(DEV)
    f, amp = hs.rope_frequencies(rot, scaling="parts", factor=8.0, original_len=512, device=DEV)
    run = lambda y, inv=False: hs.rope(y.to(DEV), pos, f, interleaved=interleaved, inverse=inv, factor=amp).double().cpu()
    grad = run(w, True)
    # each side is a sum of T * H * d products of roundings 4 * 2^-24 on terms up to amp * (|x| + |y|) |w|
    tol = 8 * 2.0 ** -24 * amp * float(x.abs().max() * w.abs().sum())
    assert abs(float((run(x) * w.double()).sum() - (x.double() * grad).sum())) <= tol
    for t, h, e in ((0, 0, 0), (4, 1, 23), (8, 0, 47), (3, 1, 63), (5, 0, 24)):
        up, dn = x.clone(), x.clone()
        up[t, h, e] += 0.5
        dn[t, h, e] -= 0.5
        step = up[t, h, e].double() - dn[t, h, e].double()
        diff = float(((run(up) - run(dn)) * w.double()).sum() / step)
        # two changed elements, each of two rounded results of size up to 2 * amp * |x|max
        assert abs(diff - float(grad[t, h, e])) <= 32 * 2.0 ** -24 * amp * float(x.abs().max() + 1) * float(w.abs().max())


def test_rope_frequencies_scalings():
    base, amp = hs.rope_frequencies(64, device="cpu")
    assert amp == 1.0 and base.dtype == torch.float64
    assert torch.equal(base, 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64))
    lin, _ = hs.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, base / 4, rtol=1e-15)
    ntk, _ = hs.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert ntk[0] == 1.0 and math.isclose(float(ntk[-1]), float(base[-1]) / 4, rel_tol=1e-12)
    for kind in ("parts", "bands"):
        f, a = hs.rope_frequencies(64, scaling=kind, factor=4.0, original_len=8192, device="cpu")
        r = f / base
        assert r[0] == 1.0 and math.isclose(float(r[-1]), 0.25, rel_tol=1e-12) and bool((r[1:] <= r[:-1] + 1e-15).all())
        assert a == (0.1 * math.log(4.0) + 1.0 if kind == "parts" else 1.0)


def _batch(gen, new, old, P, Hkv, d, dtype, lead=0, tail=0):
    kv = [a + b for a, b in zip(new, old)]
    table, pages = ref.make_table(gen, [-(-n // P) for n in kv])
    T = lead + sum(new) + tail
    cu = ref.cu_of(new) + lead
    k = torch.randn(T, Hkv, d, generator=gen).to(dtype)
    v = (torch.randn(T, Hkv, d, generator=gen) * 10).to(dtype)
    return kv, table, pages, cu, k, v


NEW = [5, 0, 1, 17, 3, 0]
OLD = [0, 9, 30, 2, 15, 0]


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("pool", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("P,Hkv,d", [(16, 2, 128), (1, 1, 64), (64, 3, 96), (4, 8, 16), (256, 1, 256)])
def test_cache_write_then_read(P, Hkv, d, pool, src):
    gen = torch.Generator().manual_seed(P + d)
    kv, table, pages, cu, k, v = _batch(gen, NEW, OLD, P, Hkv, d, DT[src], lead=2, tail=3)
    k[3] = 0.0                                # a row of zeros
    k[4] *= 2.0 ** -120 if src == "f32" else 2.0 ** -100
    v[5] *= 2.0 ** 100
    if pool == "e4m3":
        pk = torch.zeros(pages, P, Hkv, d, dtype=torch.uint8).fill_(0x2a).view(torch.float8_e4m3fn)
        sk = torch.full((pages, Hkv, P), 99, dtype=torch.uint8)
    else:
        pk, sk = torch.full((pages, P, Hkv, d), 7.0, dtype=DT[pool]), None
    dk, dv = pk.to(DEV), pk.to(DEV).clone()
    dsk, dsv = (None, None) if sk is None else (sk.to(DEV), sk.to(DEV).clone())
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    args = (cu.to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV), table.to(DEV))
    hs.cache_write(k.to(DEV), v.to(DEV), dk, dv, *args, k_scale=dsk, v_scale=dsv, ws=ws)
    assert hs.workspace_status(ws) == _lib.HS_OK
    touched = torch.zeros(pages, P, dtype=torch.bool)
    for b, n in enumerate(NEW):
        for i in range(n):
            pos = OLD[b] + i
            page, row = int(table[b, pos // P]), pos % P
            touched[page, row] = True
            for got, gs, x in ((dk, dsk, k), (dv, dsv, v)):
                r = x[2 + sum(NEW[:b]) + i]
                if pool == "e4m3":
                    code, byte = ref.e4m3(r.double())
                    assert torch.equal(gs[page, :, row].cpu().long(), byte)
                    assert torch.equal(got[page, row].float().double().cpu(), code)
                else:
                    assert torch.equal(got[page, row].cpu(), r.to(DT[pool]))
    for got, was in ((dk, pk), (dv, pk)):
        assert torch.equal(got.view(torch.uint8).cpu()[~touched], was.view(torch.uint8)[~touched])
    if sk is not None:
        assert torch.equal(dsk.cpu().transpose(1, 2)[~touched], sk.transpose(1, 2)[~touched])

    # read back: every new row, from its own start
    start = torch.tensor(OLD, dtype=torch.int32, device=DEV)
    T = k.shape[0]
    for out in ("bf16", "f32"):
        rk = torch.full((T, Hkv, d), -3.0, dtype=DT[out], device=DEV)
        rv = rk.clone()
        hs.cache_read(dk, dv, args[0], args[2], total=T, start=start, k_scale=dsk, v_scale=dsv, dtype=DT[out],
                      out_k=rk, out_v=rv, ws=ws)
        assert hs.workspace_status(ws) == _lib.HS_OK
        for b, n in enumerate(NEW):
            part = slice(2 + sum(NEW[:b]), 2 + sum(NEW[:b]) + n)
            for got, pg, sc in ((rk, dk, dsk), (rv, dv, dsv)):
                want = ref.rows_of(pg.cpu(), table[b], OLD[b], OLD[b] + n, None if sc is None else sc.cpu())
                assert torch.equal(got[part].cpu(), want.to(DT[out]))
        for got in (rk, rv):                  # rows of no sequence
            assert bool((got[:2] == -3).all()) and bool((got[T - 3:] == -3).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("pool", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("rot", [128, 64, 24])
def test_cache_write_rotates_keys(rot, pool, interleaved):
    gen = torch.Generator().manual_seed(rot)
    P, Hkv, d = 8, 2, 128
    kv, table, pages, cu, k, v = _batch(gen, NEW, OLD, P, Hkv, d, torch.bfloat16)
    dt = torch.float8_e4m3fn if pool == "e4m3" else DT[pool]
    dk = torch.zeros(pages, P, Hkv, d, dtype=torch.float32, device=DEV).to(dt)
    dv = dk.clone()
    sc = [torch.zeros(pages, Hkv, P, dtype=torch.uint8, device=DEV) for _ in range(2)] if pool == "e4m3" else [None, None]
    f, _ = hs.rope_frequencies(rot, device=DEV)
    qkv = torch.cat((k, v), 1).to(DEV)        # strided rows
    hs.cache_write(qkv[:, :Hkv], qkv[:, Hkv:], dk, dv, cu.to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV),
                   table.to(DEV), k_scale=sc[0], v_scale=sc[1], inv_freq=f, interleaved=interleaved)
    for b, n in enumerate(NEW):
        x = k[sum(NEW[:b]):sum(NEW[:b]) + n]
        pos = torch.arange(OLD[b], OLD[b] + n, dtype=torch.int32)
        want = ref.rope(x, pos, f.cpu(), interleaved)
        got = ref.rows_of(dk.cpu(), table[b], OLD[b], OLD[b] + n, None if sc[0] is None else sc[0].cpu())
        if n == 0:
            continue
        gv = ref.rows_of(dv.cpu(), table[b], OLD[b], OLD[b] + n, None if sc[1] is None else sc[1].cpu())
        xv = v[sum(NEW[:b]):sum(NEW[:b]) + n].double()
        if pool == "e4m3":
            code, byte_v = ref.e4m3(xv)
            xv = code * torch.exp2(byte_v.double() - 127)[..., None]
        assert torch.equal(gv, xv)             # values are never turned
        slack = 4 * 2.0 ** -24 * 2 * x.double().abs().amax(-1, keepdim=True)
        if pool == "e4m3":
            # half a step of the 8-bit grid under the row's scale (at least the subnormal step 2^-9)
            byte = torch.stack([sc[0].cpu()[int(table[b, p // P]), :, int(p) % P] for p in pos]).double()
            unit = torch.exp2(byte - 127)[..., None]
            half = torch.maximum(want.abs() * 2.0 ** -4, unit * 2.0 ** -10)
            top = want.abs().amax(-1, keepdim=True)
            assert bool((top <= 448 * unit * (1 + 1e-6)).all()) and bool((top > 224 * unit * (1 - 1e-6)).all())
        elif pool == "bf16":
            half = want.abs() * 2.0 ** -8
        else:
            half = 0.0
        assert bool(((got - want).abs() <= half + slack).all())
        # the same turn as rope's own, bit for bit, where nothing is rounded to 8 bits
        if pool != "e4m3":
            r = hs.rope(x.to(DEV).float() if pool == "f32" else x.to(DEV), pos.to(DEV), f, interleaved=interleaved)
            assert torch.equal(got.to(DT[pool]), r.cpu())


def test_cache_calls_report_bad_lengths_and_pages():
    """Lengths and pages that would leave the pools are skipped and reported; nothing else changes."""
    P, Hkv, d = 4, 1, 64
    new = [2, 2, 2]
    cu = ref.cu_of(new).to(DEV)
    k = torch.ones(6, Hkv, d, device=DEV)
    table = torch.tensor([[0, 1], [2, 9], [3, -1]], dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def write(kv):
        pk, pv = (torch.zeros(4, P, Hkv, d, device=DEV) for _ in range(2))
        hs.cache_write(k, k, pk, pv, cu, torch.tensor(kv, dtype=torch.int32, device=DEV), table, ws=ws)
        return pk, hs.workspace_status(ws)

    pk, st = write([2, 3, 4])
    assert st == _lib.HS_OK and int((pk != 0).sum()) == 6 * d
    pk, st = write([2, 5, 4])                       # sequence 1's second row falls on page 9
    assert st == _lib.HS_ERR_INVALID_INDEX and int((pk != 0).sum()) == 5 * d
    pk, st = write([2, 3, 5])                       # sequence 2's second row falls on page -1
    assert st == _lib.HS_ERR_INVALID_INDEX and int((pk != 0).sum()) == 5 * d
    for bad, rows in (([9, 3, 4], 5), ([1, 3, 4], 5), ([2 ** 31 - 1, 3, 4], 4), ([-2 ** 31, 3, 4], 4)):
        pk, st = write(bad)
        assert st == _lib.HS_ERR_INVALID_ARG and int((pk != 0).sum()) == rows * d
    pool = torch.ones(4, P, Hkv, d, device=DEV)
    out = torch.zeros(6, Hkv, d, device=DEV)
    start = torch.tensor([0, 3, 7], dtype=torch.int32, device=DEV)
    hs.cache_read(pool, pool, cu, table, total=6, start=start, dtype=torch.float32, out_k=out, out_v=out.clone(), ws=ws)
    assert int((out != 0).sum()) == 3 * d           # page 9, page -1 and position 8 are left out
    assert hs.workspace_status(ws) == _lib.HS_ERR_INVALID_ARG


def test_cache_ops_in_a_graph():
    """Captured once and replayed over new contents: the results follow the inputs."""
    P, Hkv, d = 16, 2, 128
    gen = torch.Generator().manual_seed(0)
    kv, table, pages, cu, k, v = _batch(gen, NEW, OLD, P, Hkv, d, torch.bfloat16)
    pk = torch.zeros(pages, P, Hkv, d, dtype=torch.float8_e4m3fn, device=DEV)
    pv = pk.clone()
    sk, sv = (torch.zeros(pages, Hkv, P, dtype=torch.uint8, device=DEV) for _ in range(2))
    f, _ = hs.rope_frequencies(d, device=DEV)
    dk, dv, dcu, dkv, dt = k.to(DEV), v.to(DEV), cu.to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV), table.to(DEV)
    start = torch.tensor(OLD, dtype=torch.int32, device=DEV)

    def go():
        hs.cache_write(dk, dv, pk, pv, dcu, dkv, dt, k_scale=sk, v_scale=sv, inv_freq=f)
        return hs.cache_read(pk, pv, dcu, dt, total=k.shape[0], start=start, k_scale=sk, v_scale=sv)
    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = go()
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        dk.copy_(torch.randn(k.shape, generator=gen))
        dv.copy_(torch.randn(v.shape, generator=gen))
        g.replay()
        got = [x.clone() for x in out]
        want = go()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("d", [128, 48])
@pytest.mark.parametrize("pool", ["bf16", "f32", "e4m3"])
def test_cache_write_nan_and_infinity(pool, d):
    """A NaN stays where it is, or (8-bit) makes its row and head one of NaN; an infinity stays, or becomes
    448 * 2^120 beside codes under that row's scale.  Other rows are not touched by either."""
    gen = torch.Generator().manual_seed(5)
    T, Hkv, P = 9, 3, 4
    k = torch.randn(T, Hkv, d, generator=gen).to(torch.bfloat16)
    bad = k.clone()
    bad[2, 1, d - 3] = math.nan
    bad[4, 0, 7] = math.inf
    bad[4, 2, 8] = -math.inf
    bad[7] = math.nan
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    args = (torch.tensor([0, T], dtype=torch.int32, device=DEV), torch.tensor([T], dtype=torch.int32, device=DEV), table)
    if pool == "e4m3":
        pools = [torch.zeros(3, P, Hkv, d, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.zeros(3, Hkv, P, dtype=torch.uint8, device=DEV) for _ in range(2)]
    else:
        pools = [torch.zeros(3, P, Hkv, d, dtype=DT[pool], device=DEV) for _ in range(2)]
        scales = [None, None]
    hs.cache_write(k.to(DEV), bad.to(DEV), *pools, *args, k_scale=scales[0], v_scale=scales[1])
    clean, got = hs.cache_read(*pools, args[0], table, total=T, k_scale=scales[0], v_scale=scales[1], dtype=torch.float32)
    clean, got = clean.cpu(), got.cpu()
    want = clean.clone()
    if pool == "e4m3":
        want[2, 1] = math.nan
        want[4, [0, 2]] = 0.0                             # beside 448 * 2^120, which fp32 has as infinity
        want[4, 0, 7], want[4, 2, 8] = math.inf, -math.inf
        assert int((scales[1] == 255).sum()) == 1 + Hkv and int((scales[0] == 255).sum()) == 0
    else:
        want[2, 1, d - 3], want[4, 0, 7], want[4, 2, 8] = math.nan, math.inf, -math.inf
    want[7] = math.nan
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0)) and bool(torch.isfinite(clean).all())
