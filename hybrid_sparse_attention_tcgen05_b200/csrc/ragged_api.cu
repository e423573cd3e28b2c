// C-ABI entry points over ragged batches and paged caches: argument checks on
// the host and dispatch.  See include/hysparse.h for the contract of every
// call.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "hysparse.h"
#include "internal.h"

namespace hs {
namespace {

bool aligned(const void *p, unsigned n) { return p != nullptr && ((uintptr_t)p & (n - 1)) == 0; }

size_t elem_bytes(int dtype) { return dtype == HS_F32 ? 4 : 2; }

// A row stride in elements: at least one row, and whole 16-byte units.
bool row_stride_ok(long long ld, int H, int d, int dtype) {
    return ld >= (long long)H * d && ld < (1ll << 40) && (ld * (long long)elem_bytes(dtype)) % 16 == 0;
}

constexpr int kMaxHeads = 4096;

int check_rows(int T, int H, int d, int dtype) {
    if (T < 0 || H < 1 || H > kMaxHeads || d < 1) return HS_ERR_INVALID_ARG;
    if (dtype != HS_F32 && dtype != HS_BF16) return HS_ERR_INVALID_ARG;
    return HS_OK;
}

int check_rot(int rot, int d, float factor) {
    if (rot < 2 || rot > d || (rot & 1) != 0 || !isfinite(factor)) return HS_ERR_INVALID_ARG;
    return HS_OK;
}

int resolve_cache(const hs_paged_cache *in, bool need_kv_len, int Hkv, int d, PagedCache *out) {
    if (in == nullptr) return HS_ERR_INVALID_ARG;
    const hs_paged_cache &c = *in;
    if (c.B < 1 || !aligned(c.cu_rows, 4) || (need_kv_len && !aligned(c.kv_len, 4)) || !aligned(c.block_table, 4))
        return HS_ERR_INVALID_ARG;
    const int ps = c.page_size;
    if (ps < 1 || ps > (1 << 16) || (ps & (ps - 1)) != 0) return HS_ERR_INVALID_ARG;
    if (c.max_pages < 1 || c.num_pages < 1) return HS_ERR_INVALID_ARG;
    if ((long long)c.max_pages * ps > 0x7fffffffLL) return HS_ERR_INVALID_ARG;   // positions in int32
    if ((long long)c.num_pages * ps > 0x7fffffffLL) return HS_ERR_INVALID_ARG;   // pool rows in int32
    if (c.cache_dtype != HS_F32 && c.cache_dtype != HS_BF16 && c.cache_dtype != HS_E4M3) return HS_ERR_INVALID_ARG;
    if (!aligned(c.k_pages, 16) || !aligned(c.v_pages, 16)) return HS_ERR_INVALID_ARG;
    if (c.cache_dtype == HS_E4M3 && (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))) return HS_ERR_INVALID_ARG;
    if (Hkv < 1 || Hkv > kMaxHeads) return HS_ERR_INVALID_ARG;
    if (d < 16 || d > 256 || d % 16 != 0) return HS_ERR_UNSUPPORTED;
    out->cu_rows = c.cu_rows;
    out->kv_len = c.kv_len;
    out->block_table = c.block_table;
    out->B = c.B;
    out->page_shift = __builtin_ctz((unsigned)ps);
    out->max_pages = c.max_pages;
    out->num_pages = c.num_pages;
    out->dtype = c.cache_dtype;
    out->k_pages = c.k_pages;
    out->v_pages = c.v_pages;
    out->k_scale = c.k_scale;
    out->v_scale = c.v_scale;
    return HS_OK;
}

// What both attention calls and the workspace size share.
int resolve_attn(int B, int T, int Hq, int Hkv, int d, int max_q, int max_len, float scale, RaggedCall *a) {
    if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || Hq > kMaxHeads || Hq % Hkv != 0) return HS_ERR_INVALID_ARG;
    if (max_q < 0 || max_len < 0 || !(scale == scale) || isinf(scale)) return HS_ERR_INVALID_ARG;
    if (d != 128 || Hq / Hkv > 32) return HS_ERR_UNSUPPORTED;
    a->B = B;
    a->T = T;
    a->Hq = Hq;
    a->Hkv = Hkv;
    a->max_q = max_q > 0 ? max_q : T;
    a->max_len = max_len;
    a->scale = scale > 0.f ? scale : 1.0f / sqrtf((float)d);
    return HS_OK;
}

int run_attn(const RaggedCall &a, void *ws, size_t ws_bytes, hs_stream_t stream) {
    if (a.T == 0) return HS_OK;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.lse, 4) || !row_stride_ok(a.ld_q, a.Hq, 128, HS_BF16))
        return HS_ERR_INVALID_ARG;
    if (!aligned(ws, 256)) return HS_ERR_INVALID_ARG;
    // other rows' work items still read these when the first results are written
    if (a.out == a.q || a.out == a.k || a.out == a.v) return HS_ERR_INVALID_ARG;
    const RaggedPlan pl = ragged_plan(a);
    if (ws_bytes < pl.bytes) return HS_ERR_WORKSPACE;
    const cudaError_t e = ragged_attn_launch(a, pl, ws, wait_limit_ns(), (cudaStream_t)stream);
    return e == cudaSuccess ? HS_OK : HS_ERR_CUDA;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? HS_OK : HS_ERR_CUDA; }

}  // namespace
}  // namespace hs

using namespace hs;

extern "C" {

int hysparse_rope(int T, int Hq, int Hkv, int d, int dtype, const void *q, long long ld_q, const void *k,
                  long long ld_k, const int32_t *positions, const double *inv_freq, int rot, int flags, float factor,
                  void *out_q, long long ld_oq, void *out_k, long long ld_ok, hs_stream_t stream) {
    int rc = check_rows(T, Hq, d, dtype);
    if (rc != HS_OK) return rc;
    if (Hkv < 0 || Hkv > kMaxHeads || (flags & ~(HS_ROPE_INTERLEAVED | HS_ROPE_INVERSE)) != 0)
        return HS_ERR_INVALID_ARG;
    if (d % 8 != 0 || d > 512) return HS_ERR_UNSUPPORTED;
    rc = check_rot(rot, d, factor);
    if (rc != HS_OK) return rc;
    if (T == 0) return HS_OK;
    if (!aligned(q, 16) || !aligned(out_q, 16) || !aligned(positions, 4) || !aligned(inv_freq, 8))
        return HS_ERR_INVALID_ARG;
    if (!row_stride_ok(ld_q, Hq, d, dtype) || !row_stride_ok(ld_oq, Hq, d, dtype)) return HS_ERR_INVALID_ARG;
    if (Hkv > 0 && (!aligned(k, 16) || !aligned(out_k, 16) || !row_stride_ok(ld_k, Hkv, d, dtype) ||
                    !row_stride_ok(ld_ok, Hkv, d, dtype)))
        return HS_ERR_INVALID_ARG;
    // turned in place, a row has to be where it was
    if ((out_q == q && ld_oq != ld_q) || (Hkv > 0 && out_k == k && ld_ok != ld_k)) return HS_ERR_INVALID_ARG;
    RopeCall a{};
    a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.d = d; a.rot = rot; a.dtype = dtype;
    a.interleaved = (flags & HS_ROPE_INTERLEAVED) != 0;
    a.inverse = (flags & HS_ROPE_INVERSE) != 0;
    a.factor = factor;
    a.q = q; a.k = k; a.out_q = out_q; a.out_k = out_k;
    a.ld_q = ld_q; a.ld_k = ld_k; a.ld_oq = ld_oq; a.ld_ok = ld_ok;
    a.positions = positions; a.inv_freq = inv_freq;
    return cuda_status(rope_launch(a, (cudaStream_t)stream));
}

int hysparse_cache_write(const hs_paged_cache *cache, int T, int Hkv, int d, int dtype, const void *k, long long ld_k,
                         const void *v, long long ld_v, const double *inv_freq, int rot, int flags, float factor,
                         void *ws, hs_stream_t stream) {
    PagedCache c;
    int rc = check_rows(T, Hkv, d, dtype);
    if (rc != HS_OK) return rc;
    rc = resolve_cache(cache, true, Hkv, d, &c);
    if (rc != HS_OK) return rc;
    if ((flags & ~HS_ROPE_INTERLEAVED) != 0) return HS_ERR_INVALID_ARG;
    if (inv_freq != nullptr) {
        rc = check_rot(rot, d, factor);
        if (rc != HS_OK) return rc;
        if (!aligned(inv_freq, 8)) return HS_ERR_INVALID_ARG;
    }
    if (ws != nullptr && !aligned(ws, 16)) return HS_ERR_INVALID_ARG;
    if (T == 0) return HS_OK;
    if (!aligned(k, 16) || !aligned(v, 16) || !row_stride_ok(ld_k, Hkv, d, dtype) ||
        !row_stride_ok(ld_v, Hkv, d, dtype))
        return HS_ERR_INVALID_ARG;
    return cuda_status(cache_write_launch(c, T, Hkv, d, dtype, k, ld_k, v, ld_v, inv_freq, rot,
                                          (flags & HS_ROPE_INTERLEAVED) != 0, factor, (unsigned int *)ws,
                                          (cudaStream_t)stream));
}

int hysparse_cache_read(const hs_paged_cache *cache, const int32_t *start, int total, int Hkv, int d, int dtype,
                        void *k, void *v, void *ws, hs_stream_t stream) {
    PagedCache c;
    int rc = check_rows(total, Hkv, d, dtype);
    if (rc != HS_OK) return rc;
    rc = resolve_cache(cache, false, Hkv, d, &c);
    if (rc != HS_OK) return rc;
    if (start != nullptr && !aligned(start, 4)) return HS_ERR_INVALID_ARG;
    if (ws != nullptr && !aligned(ws, 16)) return HS_ERR_INVALID_ARG;
    if (total == 0) return HS_OK;
    if (!aligned(k, 16) || !aligned(v, 16)) return HS_ERR_INVALID_ARG;
    return cuda_status(cache_read_launch(c, start, total, Hkv, d, dtype, k, v, (unsigned int *)ws,
                                         (cudaStream_t)stream));
}

size_t hysparse_ragged_workspace_size(int B, int T, int Hq, int Hkv, int d, int max_q, int max_len) {
    RaggedCall a{};
    if (resolve_attn(B, T, Hq, Hkv, d, max_q, max_len, 0.f, &a) != HS_OK) return 0;
    if (max_len == 0) return ragged_most_bytes(a);
    size_t n = ragged_plan(a).bytes;   // whichever call and pool it is for
    for (int dtype : {(int)HS_BF16, (int)HS_E4M3}) {
        a.paged = true;
        a.cache.dtype = dtype;
        const size_t m = ragged_plan(a).bytes;
        n = n > m ? n : m;
    }
    return n;
}

int hysparse_packed_attn(const int32_t *cu_rows, int B, int T, int Hq, int Hkv, int d, int max_len, float scale,
                         const void *q, long long ld_q, const void *k, long long ld_k, const void *v, long long ld_v,
                         void *out, float *lse, void *ws, size_t ws_bytes, hs_stream_t stream) {
    RaggedCall a{};
    const int rc = resolve_attn(B, T, Hq, Hkv, d, max_len, max_len > 0 ? max_len : T, scale, &a);
    if (rc != HS_OK) return rc;
    if (!aligned(cu_rows, 4)) return HS_ERR_INVALID_ARG;
    if (T > 0 && (!aligned(k, 16) || !aligned(v, 16) || !row_stride_ok(ld_k, Hkv, d, HS_BF16) ||
                  !row_stride_ok(ld_v, Hkv, d, HS_BF16)))
        return HS_ERR_INVALID_ARG;
    a.paged = false;
    a.cache.cu_rows = cu_rows;
    a.cache.B = B;
    a.q = q; a.k = k; a.v = v; a.ld_q = ld_q; a.ld_k = ld_k; a.ld_v = ld_v;
    a.out = out; a.lse = lse;
    return run_attn(a, ws, ws_bytes, stream);
}

int hysparse_chunk_attn_paged(const hs_paged_cache *cache, int T, int Hq, int Hkv, int d, int max_q, int max_len,
                              float scale, const void *q, long long ld_q, void *out, float *lse, void *ws,
                              size_t ws_bytes, hs_stream_t stream) {
    if (cache == nullptr) return HS_ERR_INVALID_ARG;
    RaggedCall a{};
    int rc = resolve_attn(cache->B, T, Hq, Hkv, d, max_q, max_len, scale, &a);
    if (rc != HS_OK) return rc;
    rc = resolve_cache(cache, true, Hkv, d, &a.cache);
    if (rc != HS_OK) return rc;
    if (a.cache.dtype == HS_F32) return HS_ERR_UNSUPPORTED;
    a.paged = true;
    if (max_len == 0) a.max_len = cache->max_pages * cache->page_size;
    a.q = q; a.ld_q = ld_q;
    a.out = out; a.lse = lse;
    return run_attn(a, ws, ws_bytes, stream);
}

}  // extern "C"
