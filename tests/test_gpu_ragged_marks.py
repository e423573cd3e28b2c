"""What the ragged-batch calls tell torch about the tensors that they write."""
import pytest
import torch

import hybrid_sparse_attention_tcgen05_b200 as hs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _args():
    f, _ = hs.rope_frequencies(128, device=DEV)
    return _int(list(range(6))), f, _int([0, 4, 6]), _int([4, 2]), _int([[0, 1], [2, 3]])


def test_backward_notices_what_was_written_over():
    pos, f, *_ = _args()
    leaf = torch.randn(6, 4, 128, device=DEV).to(BF).requires_grad_()
    x = leaf * 1.0
    y = (x * x).sum()                                 # saves x
    hs.rope(x.detach(), pos, f, out=x.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_written_tensors_count_as_changed():
    pos, f, cu, kv, table = _args()
    q, k, v = (torch.randn(6, h, 128, device=DEV).to(BF) for h in (4, 2, 2))
    pk, pv = (torch.zeros(4, 16, 2, 128, dtype=BF, device=DEV) for _ in range(2))
    p8 = [torch.zeros(4, 16, 2, 128, device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    s8 = [torch.zeros(4, 2, 16, dtype=torch.uint8, device=DEV) for _ in range(2)]
    out, ok, lse = torch.empty_like(q), torch.empty_like(k), torch.empty(4, 6, device=DEV)
    bk, bv = torch.empty_like(k), torch.empty_like(v)
    for call, written in ((lambda: hs.rope(q, pos, f, k=k, out=out, out_k=ok), (out, ok)),
                          (lambda: hs.cache_write(k, v, pk, pv, cu, kv, table), (pk, pv)),
                          (lambda: hs.cache_write(k, v, *p8, cu, kv, table, k_scale=s8[0], v_scale=s8[1]), (*p8, *s8)),
                          (lambda: hs.cache_read(pk, pv, cu, table, total=6, out_k=bk, out_v=bv), (bk, bv)),
                          (lambda: hs.packed_attn(q, k, v, cu, out=out, lse=lse), (out, lse)),
                          (lambda: hs.chunk_attn_paged(q, pk, pv, cu, kv, table, out=out, lse=lse), (out, lse))):
        read = [x for x in (q, k, v, cu, kv, table, f, pos)]
        before, kept = [x._version for x in written], [x._version for x in read]
        call()
        assert all(x._version > n for x, n in zip(written, before))
        assert [x._version for x in read] == kept


def test_tensors_of_inference_mode():
    """Written in and outside of inference mode, and results of inputs that require gradients."""
    pos, f, cu, *_ = _args()
    with torch.inference_mode():
        x = torch.randn(6, 4, 128, device=DEV).to(BF)
        hs.rope(x, pos, f, out=x)
    want = hs.rope(x, pos, f)
    hs.rope(x, pos, f, out=x)
    assert torch.equal(x, want)
    q = torch.randn(6, 4, 128, device=DEV).to(BF).requires_grad_()
    assert not hs.rope(q, pos, f).requires_grad
    assert not hs.packed_attn(q, q, q, cu)[0].requires_grad
