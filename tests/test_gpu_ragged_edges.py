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
