"""Host-side checks of the ragged-batch calls (no GPU): bad arguments are
refused with the documented status before anything is launched.  Pointers
are fake device addresses: argument checking never dereferences them, and
every call below is refused (or has no rows)."""
import ctypes

import pytest

from hybrid_sparse_attention_tcgen05_b200 import _lib, build as hs_build

A = 0x7f0000000000
P = lambda i, off=0: ctypes.c_void_p(A + 0x100000 * i + off)
BAD, UNS, OK = _lib.HS_ERR_INVALID_ARG, _lib.HS_ERR_UNSUPPORTED, _lib.HS_OK


@pytest.fixture(scope="module")
def L():
    hs_build.build()
    return _lib.lib()


def cache(**kw):
    a = dict(cu=P(20), kv=P(21), table=P(22), B=2, page=16, max_pages=8, num_pages=100, dtype=_lib.HS_BF16, k=P(23),
             v=P(24), ks=None, vs=None)
    a.update(kw)
    val = lambda x: x.value if isinstance(x, ctypes.c_void_p) else x
    return _lib.HsPagedCache(val(a["cu"]), val(a["kv"]), val(a["table"]), a["B"], a["page"], a["max_pages"],
                             a["num_pages"], a["dtype"], val(a["k"]), val(a["v"]), val(a["ks"]), val(a["vs"]))


BAD_CACHES = [(dict(cu=None), BAD), (dict(cu=P(20, 2)), BAD), (dict(table=None), BAD), (dict(table=P(22, 1)), BAD),
              (dict(B=0), BAD), (dict(page=0), BAD), (dict(page=24), BAD), (dict(page=1 << 17), BAD),
              (dict(max_pages=0), BAD), (dict(num_pages=0), BAD), (dict(page=1 << 16, num_pages=1 << 15), BAD),
              (dict(page=1 << 16, max_pages=1 << 15), BAD), (dict(dtype=3), BAD), (dict(dtype=-1), BAD),
              (dict(k=None), BAD), (dict(v=P(24, 8)), BAD), (dict(dtype=_lib.HS_E4M3), BAD),
              (dict(dtype=_lib.HS_E4M3, ks=P(25)), BAD)]


def test_rope_rejects(L):
    def f(T=4, Hq=2, Hkv=1, d=64, dt=_lib.HS_F32, q=P(1), ldq=128, k=P(2), ldk=64, pos=P(3), fr=P(4), rot=64, flags=0,
          factor=1.0, oq=P(5), ldoq=128, ok=P(6), ldok=64):
        return L.hysparse_rope(T, Hq, Hkv, d, dt, q, ldq, k, ldk, pos, fr, rot, flags, factor, oq, ldoq, ok, ldok, None)
    assert f(T=0) == OK
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=-1), dict(Hq=5000), dict(dt=2), dict(dt=7), dict(q=None), dict(q=P(1, 8)),
               dict(k=None), dict(ok=None), dict(ok=P(6, 4)), dict(oq=None), dict(pos=None), dict(pos=P(3, 2)),
               dict(fr=None), dict(fr=P(4, 4)), dict(rot=0), dict(rot=63), dict(rot=66), dict(rot=-2), dict(flags=4),
               dict(factor=float("nan")), dict(factor=float("inf")), dict(ldq=127), dict(ldq=129), dict(ldq=0),
               dict(ldk=60), dict(ldoq=130), dict(ldok=8), dict(oq=P(1), ldoq=132), dict(ok=P(2), ldok=68)):
        assert f(**kw) == BAD, kw
    for kw in (dict(d=60, rot=60, ldq=120, ldk=60, ldoq=120, ldok=60), dict(d=520, ldq=1040, ldk=520, ldoq=1040, ldok=520)):
        assert f(**kw) == UNS, kw


def test_cache_write_rejects(L):
    def f(c=None, T=4, H=2, d=128, dt=_lib.HS_BF16, k=P(1), ldk=256, v=P(2), ldv=256, fr=None, rot=0, flags=0,
          factor=1.0, ws=None):
        c = c or cache()
        return L.hysparse_cache_write(ctypes.byref(c), T, H, d, dt, k, ldk, v, ldv, fr, rot, flags, factor, ws, None)
    assert f(T=0) == OK
    for kw, want in BAD_CACHES + [(dict(kv=None), BAD), (dict(kv=P(21, 2)), BAD)]:
        assert f(c=cache(**kw)) == want, kw
    for kw in (dict(T=-1), dict(H=0), dict(dt=2), dict(k=None), dict(v=P(2, 8)), dict(ldk=255), dict(ldv=257), dict(ldk=0),
               dict(fr=P(3, 4), rot=64), dict(fr=P(3), rot=0), dict(fr=P(3), rot=130), dict(fr=P(3), rot=31),
               dict(fr=P(3), rot=64, factor=float("nan")), dict(flags=2), dict(ws=P(9, 4))):
        assert f(**kw) == BAD, kw
    for d in (8, 72, 272):
        assert f(d=d, ldk=2 * d, ldv=2 * d) == UNS
    assert L.hysparse_cache_write(None, 4, 2, 128, 1, P(1), 256, P(2), 256, None, 0, 0, 1.0, None, None) == BAD


def test_cache_read_rejects(L):
    def f(c=None, start=None, total=4, H=2, d=128, dt=_lib.HS_BF16, k=P(1), v=P(2), ws=None):
        c = c or cache(kv=None)
        return L.hysparse_cache_read(ctypes.byref(c), start, total, H, d, dt, k, v, ws, None)
    assert f(total=0) == OK
    for kw, want in BAD_CACHES:
        assert f(c=cache(**kw)) == want, kw
    for kw in (dict(total=-1), dict(H=0), dict(dt=2), dict(k=None), dict(v=P(2, 4)), dict(start=P(3, 2)), dict(ws=P(9, 8))):
        assert f(**kw) == BAD, kw
    assert f(d=40) == UNS
    assert L.hysparse_cache_read(None, None, 4, 2, 128, 1, P(1), P(2), None, None) == BAD


def test_binding_refuses():
    """Shapes, types and places that the binding checks before the library does."""
    import torch
    import hybrid_sparse_attention_tcgen05_b200 as hs
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        hs.rope(q, torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))       # CPU tensors
    for kw in (dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=8, scaling="other"), dict(rot_dim=8, factor=0.5),
               dict(rot_dim=8, scaling="parts", factor=2.0), dict(rot_dim=2, scaling="base", factor=2.0),
               dict(rot_dim=8, scaling="bands", original_len=10, slow=2.0, fast=1.0)):
        with pytest.raises(ValueError):
            hs.rope_frequencies(**kw, device="cpu")


def test_ragged_workspace_size(L):
    f = L.hysparse_ragged_workspace_size
    assert f(1, 0, 8, 2, 128, 0, 0) == 256 and f(4, 100000, 32, 8, 128, 100000, 100000) == 256   # enough rows: no pieces
    few = f(1, 1, 8, 2, 128, 1, 32768)
    assert few > 256 and few % 256 == 0                           # one row, many keys: partial results
    for a in ((1, 1, 8, 2, 128, 1, 1 << 24), (64, 64, 32, 8, 128, 1, 32768), (3, 700, 64, 4, 128, 300, 1 << 20),
              (1, 5000, 128, 1, 128, 5000, 1 << 20)):
        n = f(*a) if a[2] // a[3] <= 32 else 256
        assert 256 <= n <= 94 << 20
    for bad in ((0, 1, 8, 2, 128, 1, 1), (1, -1, 8, 2, 128, 1, 1), (1, 1, 0, 2, 128, 1, 1), (1, 1, 8, 3, 128, 1, 1),
                (1, 1, 8, 0, 128, 1, 1), (1, 1, 8, 2, 64, 1, 1), (1, 1, 33, 1, 128, 1, 1), (1, 1, 8, 2, 128, -1, 1),
                (1, 1, 8, 2, 128, 1, -1)):
        assert f(*bad) == 0, bad


def test_packed_attn_rejects(L):
    def f(cu=P(1), B=2, T=64, Hq=8, Hkv=2, d=128, max_len=0, scale=0.0, q=P(2), ldq=1024, k=P(3), ldk=256, v=P(4), ldv=256,
          out=P(5), lse=P(6), ws=P(7), wsb=1 << 30):
        return L.hysparse_packed_attn(cu, B, T, Hq, Hkv, d, max_len, scale, q, ldq, k, ldk, v, ldv, out, lse, ws, wsb, None)
    assert f(T=0) == OK
    for kw in (dict(cu=None), dict(cu=P(1, 2)), dict(B=0), dict(T=-1), dict(Hq=0), dict(Hkv=3), dict(max_len=-1),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(q=P(2, 8)), dict(k=None),
               dict(v=P(4, 2)), dict(ldq=1023), dict(ldq=1028), dict(ldk=0), dict(ldv=260), dict(out=None),
               dict(out=P(5, 8)), dict(lse=None), dict(lse=P(6, 2)), dict(ws=None), dict(ws=P(7, 16))):
        assert f(**kw) == BAD, kw
    assert f(d=64) == UNS and f(Hq=66, Hkv=2, ldq=66 * 128) == UNS
    assert f(wsb=255) == _lib.HS_ERR_WORKSPACE
    need = L.hysparse_ragged_workspace_size(2, 64, 8, 2, 128, 4096, 4096)
    assert need > 256 and f(max_len=4096, wsb=need - 1) == _lib.HS_ERR_WORKSPACE


def test_chunk_attn_paged_rejects(L):
    def f(c=None, T=64, Hq=8, Hkv=2, d=128, max_q=0, max_len=0, scale=0.0, q=P(2), ldq=1024, out=P(5), lse=P(6), ws=P(7),
          wsb=1 << 30):
        c = c or cache()
        return L.hysparse_chunk_attn_paged(ctypes.byref(c), T, Hq, Hkv, d, max_q, max_len, scale, q, ldq, out, lse, ws, wsb,
                                           None)
    assert f(T=0) == OK
    for kw, want in BAD_CACHES + [(dict(kv=None), BAD), (dict(kv=P(21, 2)), BAD), (dict(dtype=_lib.HS_F32), UNS)]:
        assert f(c=cache(**kw)) == want, kw
    for kw in (dict(T=-1), dict(Hq=0), dict(Hkv=3), dict(max_q=-1), dict(max_len=-1), dict(scale=float("nan")), dict(q=None),
               dict(q=P(2, 4)), dict(ldq=1000), dict(ldq=1028), dict(out=None), dict(out=P(5, 8)), dict(lse=P(6, 1)),
               dict(ws=None), dict(ws=P(7, 128))):
        assert f(**kw) == BAD, kw
    assert f(d=64) == UNS and f(Hq=66, ldq=66 * 128) == UNS
    need = L.hysparse_ragged_workspace_size(2, 64, 8, 2, 128, 64, 128)
    assert f(max_q=64, wsb=need - 1) == _lib.HS_ERR_WORKSPACE
    assert L.hysparse_chunk_attn_paged(None, 64, 8, 2, 128, 0, 0, 0.0, P(2), 1024, P(5), P(6), P(7), 1 << 30, None) == BAD


def test_attention_results_may_not_replace_inputs(L):
    a = (2, 64, 8, 2, 128, 0, 0.0, P(2), 1024, P(3), 256, P(4), 256)
    for out in (P(2), P(3), P(4)):
        assert L.hysparse_packed_attn(P(1), *a, out, P(6), P(7), 1 << 30, None) == BAD
    c = cache()
    assert L.hysparse_chunk_attn_paged(ctypes.byref(c), 64, 8, 2, 128, 0, 0, 0.0, P(2), 1024, P(2), P(6), P(7), 1 << 30,
                                       None) == BAD


def test_binding_shares_the_cpp_runtime(L):
    """The native binding and torch format messages and throw through one libstdc++: a copy of its own
    crashed where a refusal prints a shape."""
    import subprocess
    needs = subprocess.run(["ldd", hs_build.BINDING], capture_output=True, text=True, check=True).stdout
    assert "libstdc++" in needs


@pytest.mark.parametrize("rot,base,length,factor", [(128, 1e4, 131072, 4.0), (128, 1e4, 65536, 4.0), (64, 1e4, 1 << 20, 8.0),
                                                    (128, 1e4, 32768, 4.0), (128, 5e5, 131072, 8.0), (64, 1e4, 8192, 4.0)])
def test_rope_frequencies_parts_ramp(rot, base, length, factor):
    """The ramp from kept to divided pairs is linear in the pair's index between the indices that make 32
    turns and one turn over the trained length (rounded outwards), also where the latter lies
    beyond the last pair: that pair, which makes more than one turn, is then not divided wholly."""
    import math

    import hybrid_sparse_attention_tcgen05_b200 as hs
    f, amp = hs.rope_frequencies(rot, base, scaling="parts", factor=factor, original_len=length, device="cpu")

    def index(turns):            # the pair whose angle makes that many turns: base^(-2 i / rot) length = 2 pi turns
        return rot / 2 * math.log(length / (2 * math.pi * turns), base)
    lo, hi = max(math.floor(index(32)), 0), min(math.ceil(index(1)), rot - 1)
    for i in range(rot // 2):
        plain = base ** (-2 * i / rot)
        mix = min(max((i - lo) / (hi - lo), 0), 1)                # 0: kept, 1: divided
        assert abs(float(f[i]) / (plain * (1 - mix) + plain / factor * mix) - 1) < 1e-12, i
        turns = length * plain / (2 * math.pi)
        if i < lo:
            assert float(f[i]) == plain
        if turns > 1:
            assert float(f[i]) > plain / factor, i
    assert abs(amp - (0.1 * math.log(factor) + 1)) < 1e-15


def test_library_is_built_where_the_binding_cannot_be(L, monkeypatch, tmp_path):
    """The C library needs nvcc only: without the headers of torch and Python it is built all the same,
    and then the binding's failure is raised."""
    def no_headers():
        raise RuntimeError("no headers")
    lib = tmp_path / "libhysparse.so"
    monkeypatch.setattr(hs_build, "LIB", str(lib))
    monkeypatch.setattr(hs_build, "_binding_stale", lambda: True)
    monkeypatch.setattr(hs_build, "_build_binding", no_headers)
    with pytest.raises(RuntimeError, match="no headers"):
        hs_build.build()
    assert ctypes.CDLL(str(lib)).hysparse_version is not None


def test_binding_raises_what_a_flag_raises():
    """A flag that has no truth value is an error of its own, not a call with the flag set."""
    import torch

    import hybrid_sparse_attention_tcgen05_b200 as hs
    both = torch.ones(2)
    q, pos, f = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    pages = torch.zeros(2, 16, 2, 64)
    for call in (lambda: hs.rope(q, pos, f, interleaved=both), lambda: hs.rope(q, pos, f, inverse=both),
                 lambda: hs.cache_write(q, q, pages, pages, pos, pos, pos, interleaved=both)):
        with pytest.raises(RuntimeError, match="Boolean value"):
            call()


def test_ragged_workspace_size_for_any_length(L):
    """max_len 0 (any length) is enough for every length, as the calls take it."""
    f = L.hysparse_ragged_workspace_size
    for B, T, Hq, Hkv, most in ((1, 1, 8, 2, 1), (64, 64, 32, 8, 1), (3, 700, 64, 4, 300), (1, 40, 32, 1, 40),
                                (16, 16, 64, 64, 1), (7, 30, 28, 4, 8), (1, 8192, 64, 4, 8192), (2, 64, 8, 2, 0)):
        any_len = f(B, T, Hq, Hkv, 128, most, 0)
        assert 256 <= any_len <= 94 << 20
        for length in [1, 100, 999, 4096, 12345, 1 << 17, 1 << 20, 1 << 24] + [1 << i for i in range(31)]:
            assert f(B, T, Hq, Hkv, 128, most, length) <= any_len, (B, T, Hq, Hkv, most, length)
