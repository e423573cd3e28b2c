// Attention of few new rows per sequence over a paged cache (decode steps,
// short speculative chunks): 8 or 16 rows (token x query head of one KV
// group) to a warp, on the warp-level MMAs.
//
// Bound: HBM.  Each K and V row of the cache is read once per 16 rows and
// used for 2 * 16 * 128 multiply-adds, far below what the tensor cores could
// do, so what matters is bytes in flight and few instructions per byte.
// Every warp streams its own 16-key blocks through a private ring of shared
// memory (cp.async, `depth` blocks deep, no barrier between warps); warps of
// a CTA take the blocks of one piece of a sequence's keys in turn and join
// their partial results at the end, and a second kernel joins the pieces.
//
// Keys are the MMA's 16-row side and query rows its 8-column side (S^T = K
// Q^T, O^T = V^T P^T), so that eight rows - a decode step of a group of up to
// eight heads - fill it.  The contraction indices may be permuted as long as
// both operands agree, and so may the output rows, which lets every lane read
// whole 16-byte chunks from shared memory:
//   S^T  lane (g, c) = (lane / 4, lane % 4) holds 32 of the 128 dimensions of
//        keys g and g + 8; MMA step kk takes its elements 4 kk .. 4 kk + 3.
//   O^T  lane (g, c) holds 16 dimensions of the keys 2 c, 2 c + 1, 2 c + 8,
//        2 c + 9; byte permutes pair the keys.  P^T gets from the scores'
//        fragment to the operand's by two 8 x 8 transposes.
// 8-bit caches: a code widens to fp16 exactly (one conversion per two codes)
// and the MMAs run in fp16.  The rows' scales stay out of the operands: the
// key's power of two joins the score, the value's joins the probability, whose
// running reference is 2^-7 of the largest probability x scale among rows that
// are not all zeros (a row of zeros has whatever scale its writer gave it), so
// that products stay below 2^15 and lose bits only from 2^-21 of the largest
// down: each is off by 2^-11 of itself or 2^-32 of the largest.  The sum of
// probabilities keeps a reference of its own.  Queries are scaled to [1, 2) by a power of two per row, which
// makes their fp16 form exact for elements within 2^-14 of the row's largest
// (2^-25 of that element's size below).  fp16 probabilities are rounded by
// 2^-11; for bf16 caches they are rounded to bf16 (2^-8), the type of V.
#include <algorithm>
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "ragged.cuh"
#include "tc_util.cuh"

namespace hs {
namespace rows {
namespace {

constexpr int kWarps = 4;          // per CTA
constexpr int kBlock = 16;         // keys a warp takes at a time
// Reference of a row that has seen no key: finite, so that differences with
// it need no special case, and below every score but the last float's.
constexpr float kNone = -3.4e38f;
// How far below a row's maximum (log2 units) a new reference is put, and how
// far above it a score may rise before it moves.
template <bool F8> struct Ref {
    static constexpr float below = F8 ? 7.f : 0.f, above = F8 ? 15.f : 8.f;
};

template <bool F8> struct Cfg {
    static constexpr int row = F8 ? 128 : 256;                     // bytes of a K or V row
    static constexpr int slot = 2 * kBlock * row + (F8 ? 32 : 0);  // K, V, scale bytes
    static constexpr int depth = F8 ? 4 : 3;
    static constexpr int ring = kWarps * depth * slot;
    static constexpr int smem = ring + kWarps * 16 * 3 * 4;        // + (mx, my, l) per warp and row
    // the rows' partial results (16 x 128 fp32 per warp) take the ring's place at the end
    static_assert(kWarps * 16 * 128 * 4 <= ring, "partial results fit the ring");
};

struct Params {
    PagedCache c;
    int T, Hq, Hkv, G, tiles;      // tiles: 8- or 16-row tiles of a sequence and KV head
    int splits, chunk;             // pieces of a sequence; blocks of 16 keys per piece
    float scale_log2;
    const __nv_bfloat16 *q;
    long long ld_q;
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;                 // as in ragged_attn_tc.cu
    float2 *part_ml;
    unsigned int *status;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    // a source size of 0 writes zeros and reads nothing
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Four codes to two pairs of fp16 numbers, exactly.
__device__ __forceinline__ uint2 widen4(uint32_t codes) {
    uint2 r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(codes));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool F8, int NB>
__global__ void __launch_bounds__(32 * kWarps, F8 ? 3 : 2) ragged_rows(const Params p) {
    using C = Cfg<F8>;
    constexpr int ROWS = 8 * NB;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gl = lane >> 2, c = lane & 3;
    int id = blockIdx.x;
    const int g = id % p.Hkv;
    id /= p.Hkv;
    const int tile = id % p.tiles;
    id /= p.tiles;
    const int piece = id % p.splits;
    const int b = id / p.splits;

    const int raw0 = __ldg(p.c.cu_rows + b), raw1 = __ldg(p.c.cu_rows + b + 1), raw_kv = __ldg(p.c.kv_len + b);
    const int q0 = clamp_row(raw0, p.T);
    const int ql = max(clamp_row(raw1, p.T) - q0, 0);
    const int kvl = min(max(raw_kv, 0), p.c.max_pages << p.c.page_shift);
    if (threadIdx.x == 0 && piece == 0 && tile == 0 && ql > 0 &&
        (raw0 < 0 || raw1 > p.T || raw_kv != kvl || (long long)ql * p.G > (long long)ROWS * p.tiles))
        report(p.status, HS_ERR_INVALID_ARG);
    if ((long long)ql * p.G <= ROWS * tile) return;
    const int nrows = (int)min((long long)ql * p.G - ROWS * tile, (long long)ROWS);
    const int off = kvl - ql;                                       // position of the first new row
    const int last = off + (ROWS * tile + nrows - 1) / p.G;
    const int blocks = last < 0 ? 0 : last / kBlock + 1;            // key blocks that any row sees
    const bool partial = blocks > p.chunk;
    const int b0 = min(piece * p.chunk, blocks);
    // (the last piece also takes keys past the length the plan was made for)
    const int nb = piece == p.splits - 1 ? blocks - b0 : min(blocks - b0, p.chunk);
    if (!partial && piece > 0) return;

    uint8_t *ring = smem + warp * C::depth * C::slot;
    float *stat = reinterpret_cast<float *>(smem + C::ring);        // [3][kWarps][ROWS]

    const int32_t *table = p.c.block_table + (size_t)b * p.c.max_pages;
    const size_t stride = (size_t)p.Hkv * C::row;                   // pool row to pool row
    constexpr int chunks = C::row / 16;                             // 16-byte chunks of a row: 8 or 16
    constexpr int per = 32 / chunks;                                // rows that one copy of a warp covers
    const int lr = lane / chunks, lch = lane % chunks;
    const uint8_t *kp = (const uint8_t *)p.c.k_pages + (size_t)g * C::row + lch * 16;
    const uint8_t *vp = (const uint8_t *)p.c.v_pages + (size_t)g * C::row + lch * 16;
    const int n = nb > warp ? (nb - warp + kWarps - 1) / kWarps : 0;   // blocks of this warp
    const int key_first = (b0 + warp) * kBlock;                     // key 0 of its first block; next ones kWarps blocks on

    // Page of key lane % 16 of this warp's i-th block (read one block ahead of
    // its copies, which need it).
    auto page_of = [&](int i) -> int {
        const int key = key_first + i * (kWarps * kBlock) + (lane & 15);
        return i < n && key < kvl ? __ldg(table + (key >> p.c.page_shift)) : -1;
    };
    int page_ahead = page_of(0);
    // Starts the copies of the i-th block; returns which of its keys are not
    // there (behind the sequence's end, or on a page outside the pool).  Their
    // rows are filled with zeros and nothing is read for them.
    auto fetch = [&](int i, int slot) -> unsigned {
        unsigned gone = 0;
        const int page = page_ahead;
        page_ahead = page_of(i + 1);
        if (i < n) {
            const uint32_t dst = tc::smem_u32(ring + slot * C::slot);
            const int key0 = key_first + i * (kWarps * kBlock);
            const int key = key0 + (lane & 15);
            const int mask = (1 << p.c.page_shift) - 1;
            int row = -1;
            if (key < kvl) {
                if (page >= 0 && page < p.c.num_pages) row = (page << p.c.page_shift) | (key & mask);
                else report(p.status, HS_ERR_INVALID_INDEX);
            }
            gone = __ballot_sync(0xffffffffu, row < 0) & 0xffffu;
            // chunks lie where the lanes that read them together find them in
            // different banks
            if (p.c.page_shift >= 4 && gone == 0) {
                // sixteen neighbouring rows of one page
                const size_t at = (size_t)((page << p.c.page_shift) | (key0 & mask)) * stride + lr * stride;
                const uint8_t *ks = kp + at, *vs = vp + at;
#pragma unroll
                for (int r0 = 0; r0 < kBlock; r0 += per) {
                    const int r = r0 + lr;
                    cp16(dst + r * C::row + ((lch ^ (F8 ? (r & 1) : (r & 1) * 4)) << 4), ks, true);
                    cp16(dst + (kBlock + r) * C::row + ((lch ^ (r & 6)) << 4), vs, true);
                    ks += per * stride;
                    vs += per * stride;
                }
            } else {
#pragma unroll
                for (int r0 = 0; r0 < kBlock; r0 += per) {
                    const int r = r0 + lr;
                    const int pr = __shfl_sync(0xffffffffu, row, r);
                    const size_t at = pr < 0 ? 0 : (size_t)pr * stride;
                    cp16(dst + r * C::row + ((lch ^ (F8 ? (r & 1) : (r & 1) * 4)) << 4), kp + at, pr >= 0);
                    cp16(dst + (kBlock + r) * C::row + ((lch ^ (r & 6)) << 4), vp + at, pr >= 0);
                }
            }
            if (F8) {
                const uint32_t sdst = dst + 2 * kBlock * C::row;
                if (p.c.page_shift >= 2) {
                    // four keys of a page at a time: lanes 0-3 of K, 4-7 of V
                    const int pr = __shfl_sync(0xffffffffu, row, (lane & 3) * 4);
                    if (lane < 8) {
                        const uint8_t *s = lane < 4 ? p.c.k_scale : p.c.v_scale;
                        cp4(sdst + lane * 4, s + (pr < 0 ? 0 : scale_index(p.c, pr, p.Hkv, g)), pr >= 0);
                    }
                } else {
                    const uint8_t *s = lane < 16 ? p.c.k_scale : p.c.v_scale;
                    ring[slot * C::slot + 2 * kBlock * C::row + lane] =
                        row < 0 ? 0 : __ldg(s + scale_index(p.c, row, p.Hkv, g));
                }
            }
        }
        cp_commit();
        return gone;
    };
    unsigned gone_ring[C::depth - 1];
#pragma unroll
    for (int s = 0; s < C::depth - 1; ++s) gone_ring[s] = fetch(s, s);

    // Q^T as the B operand: row gl of each 8-row tile, this lane's dimensions
    uint32_t qf[NB][8][2];
    float cs[NB][2];      // rows 2 c, 2 c + 1 of each tile: score -> log2 units
    int pos[NB][2];       // and their positions
#pragma unroll
    for (int t = 0; t < NB; ++t) {
        const int r = min(8 * t + gl, nrows - 1) + ROWS * tile;
        const int tok = r / p.G;
        const __nv_bfloat16 *qrow = p.q + (long long)(q0 + tok) * p.ld_q + (size_t)(g * p.G + r % p.G) * 128;
        float inv = 1.f;
        int a = 127;      // the row's power of two, 2^(a - 127)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const uint4 u = *reinterpret_cast<const uint4 *>(qrow + (F8 ? 32 * c + 8 * v : 8 * (c + 4 * v)));
            qf[t][2 * v][0] = u.x;
            qf[t][2 * v][1] = u.y;
            qf[t][2 * v + 1][0] = u.z;
            qf[t][2 * v + 1][1] = u.w;
        }
        if (F8) {
            float top = 0.f;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qf[t][kk][e]));
                    top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // rows of zeros and the ends of the range stay within normal factors
            a = min(max((int)(__float_as_uint(top) >> 23), 2), 252);
            inv = __uint_as_float((uint32_t)(254 - a) << 23);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&qf[t][kk][e]));
                    qf[t][kk][e] = pack_f16(f.x * inv, f.y * inv);
                }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rc = 2 * c + e;
            cs[t][e] = p.scale_log2;
            if (F8) cs[t][e] *= __uint_as_float((uint32_t)__shfl_sync(0xffffffffu, a, rc * 4) << 23);
            pos[t][e] = off + (min(8 * t + rc, nrows - 1) + ROWS * tile) / p.G;
        }
    }

    float o[NB][8][4];
    float mx[NB][2], my[NB][2], l[NB][2];
#pragma unroll
    for (int t = 0; t < NB; ++t) {
#pragma unroll
        for (int d = 0; d < 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][d][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            mx[t][e] = my[t][e] = kNone;
            l[t][e] = 0.f;
        }
    }

    int slot = 0;
    for (int i = 0; i < n; ++i) {
        cp_wait<C::depth - 2>();
        __syncwarp();
        const uint8_t *blk = ring + slot * C::slot;
        const unsigned gone = gone_ring[0];
        const int key0 = key_first + i * (kWarps * kBlock);
        // scores: keys gl (elements 0, 1 of a fragment) and gl + 8 (2, 3) against rows
        // 2 c, 2 c + 1; two chains of four MMAs each
        float s[NB][2][4];
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[t][e >> 2][e & 3] = 0.f;
#pragma unroll
        for (int v = 0; v < C::row / 64; ++v) {
            const int ch = F8 ? (2 * c + v) ^ (gl & 1) : (c + 4 * v) ^ ((gl & 1) * 4);
            const uint4 x = *reinterpret_cast<const uint4 *>(blk + gl * C::row + (ch << 4));
            const uint4 y = *reinterpret_cast<const uint4 *>(blk + (gl + 8) * C::row + (ch << 4));
            const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
            if constexpr (F8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int kk = 4 * v + q;
                    const uint2 xa = widen4(xw[q]), ya = widen4(yw[q]);
                    const uint4 a = make_uint4(xa.x, ya.x, xa.y, ya.y);
#pragma unroll
                    for (int t = 0; t < NB; ++t) mma<true>(s[t][kk & 1], a, qf[t][kk][0], qf[t][kk][1]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int kk = 2 * v + q;
                    const uint4 a = make_uint4(xw[2 * q], yw[2 * q], xw[2 * q + 1], yw[2 * q + 1]);
#pragma unroll
                    for (int t = 0; t < NB; ++t) mma<false>(s[t][kk & 1], a, qf[t][kk][0], qf[t][kk][1]);
                }
            }
        }
        float ks[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f};
        if (F8) {
            const uint8_t *sc = blk + 2 * kBlock * C::row + gl;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                ks[k] = __uint_as_float((uint32_t)sc[8 * k] << 23);
                // byte - 127 as a float: 2^23 + byte, less 2^23 + 127
                ev[k] = __uint_as_float(0x4b000000u | sc[kBlock + 8 * k]) - 8388735.f;
            }
        }
        uint32_t pb[NB][2];       // P^T as the B operand: row gl, keys 2 c, 2 c + 1 / 2 c + 8, 2 c + 9
        bool grow = false;
        float x[NB][4], y[NB][4];     // [2 * key + row]: score in log2 units; with the value's exponent
#pragma unroll
        for (int t = 0; t < NB; ++t) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x[t][2 * k + e] = (s[t][0][2 * k + e] + s[t][1][2 * k + e]) * (F8 ? ks[k] * cs[t][e] : cs[t][e]);
        }
        // keys that a row must not see: only near the sequence's end, or on lost pages
        if (key0 + kBlock - 1 > off || gone != 0) {
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (key0 + gl + 8 * k > pos[t][e] || ((gone >> (gl + 8 * k)) & 1u)) x[t][2 * k + e] = -INFINITY;
        }
#pragma unroll
        for (int t = 0; t < NB; ++t) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e) y[t][2 * k + e] = F8 ? x[t][2 * k + e] + ev[k] : x[t][2 * k + e];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                grow = grow || fmaxf(y[t][e], y[t][2 + e]) > my[t][e] + Ref<F8>::above;
                if (F8) grow = grow || fmaxf(x[t][e], x[t][2 + e]) > mx[t][e] + 8.f;
            }
        }
        // the references move only when a row's maximum grows by more than 8
        if (__any_sync(0xffffffffu, grow)) {
            if (F8) {
                // value rows of zeros give nothing: their scales move no reference
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 *vr = reinterpret_cast<const uint4 *>(blk + (kBlock + gl + 8 * k) * C::row + 32 * c);
                    const uint4 u = vr[0], w = vr[1];
                    uint32_t any = (u.x | u.y | u.z | u.w | w.x | w.y | w.z | w.w) & 0x7f7f7f7fu;
                    any |= __shfl_xor_sync(0xffffffffu, any, 1);
                    any |= __shfl_xor_sync(0xffffffffu, any, 2);
                    if (any == 0) {                  // (NaN and infinity stay: they make the row NaN)
#pragma unroll
                        for (int t = 0; t < NB; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (y[t][2 * k + e] < INFINITY) y[t][2 * k + e] = -INFINITY;
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float ty = fmaxf(y[t][e], y[t][2 + e]), tx = fmaxf(x[t][e], x[t][2 + e]);
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) {
                        ty = fmaxf(ty, __shfl_xor_sync(0xffffffffu, ty, d));
                        if (F8) tx = fmaxf(tx, __shfl_xor_sync(0xffffffffu, tx, d));
                    }
                    if (!F8) tx = ty;
                    const float ny = fmaxf(my[t][e], ty - Ref<F8>::below), nx = fmaxf(mx[t][e], tx);
                    const float cy = ex2(my[t][e] - ny);
                    l[t][e] *= ex2(mx[t][e] - nx);
                    my[t][e] = ny;
                    mx[t][e] = nx;
#pragma unroll
                    for (int d = 0; d < 8; ++d) {
                        o[t][d][e] *= cy;
                        o[t][d][2 + e] *= cy;
                    }
                }
        }
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            float pr[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ry = my[t][e], rx = mx[t][e];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    pr[2 * k + e] = ex2(y[t][2 * k + e] - ry);
                    l[t][e] += F8 ? ex2(x[t][2 * k + e] - rx) : pr[2 * k + e];
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                pb[t][k] = tc::movm_t(F8 ? pack_f16(pr[2 * k], pr[2 * k + 1]) : tc::pack_bf16(pr[2 * k], pr[2 * k + 1]));
        }
        // O^T += V^T P^T
#pragma unroll
        for (int half = 0; half < C::row / 128; ++half) {
            uint4 v[4];           // keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9; 16 (8) dimensions of each
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 2 * c + (k & 1) + 8 * (k >> 1);
                v[k] = *reinterpret_cast<const uint4 *>(blk + (kBlock + r) * C::row + (((gl + 8 * half) ^ (2 * c)) << 4));
            }
            const uint32_t *v0 = reinterpret_cast<const uint32_t *>(&v[0]), *v1 = reinterpret_cast<const uint32_t *>(&v[1]);
            const uint32_t *v2 = reinterpret_cast<const uint32_t *>(&v[2]), *v3 = reinterpret_cast<const uint32_t *>(&v[3]);
            if constexpr (F8) {
#pragma unroll
                for (int d = 0; d < 8; ++d) {        // dimensions 2 d, 2 d + 1: codes (k0 d, k1 d, k0 d+1, k1 d+1)
                    const uint32_t sel = (d & 1) ? 0x7362 : 0x5140;
                    const uint2 lo = widen4(__byte_perm(v0[d / 2], v1[d / 2], sel));
                    const uint2 hi = widen4(__byte_perm(v2[d / 2], v3[d / 2], sel));
                    const uint4 a = make_uint4(lo.x, lo.y, hi.x, hi.y);
#pragma unroll
                    for (int t = 0; t < NB; ++t) mma<true>(o[t][d], a, pb[t][0], pb[t][1]);
                }
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const uint4 a = make_uint4(__byte_perm(v0[d], v1[d], 0x5410), __byte_perm(v0[d], v1[d], 0x7632),
                                               __byte_perm(v2[d], v3[d], 0x5410), __byte_perm(v2[d], v3[d], 0x7632));
#pragma unroll
                    for (int t = 0; t < NB; ++t) mma<false>(o[t][4 * half + d], a, pb[t][0], pb[t][1]);
                }
            }
        }
        __syncwarp();                                            // the slot's readers are done
        const int next = slot == 0 ? C::depth - 1 : slot - 1;    // the slot of the block before this one
#pragma unroll
        for (int d = 0; d < C::depth - 2; ++d) gone_ring[d] = gone_ring[d + 1];
        gone_ring[C::depth - 2] = fetch(i + C::depth - 1, next);
        slot = slot + 1 == C::depth ? 0 : slot + 1;
    }
    cp_wait<0>();
    __syncthreads();                                             // the rings become the partial results

    // join the warps: references, then the weighted sums
    float *po = reinterpret_cast<float *>(smem) + warp * ROWS * 128;
#pragma unroll
    for (int t = 0; t < NB; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], d);
            const int r = 8 * t + 2 * c + e;
            if (gl == 0) {
                stat[(0 * kWarps + warp) * ROWS + r] = mx[t][e];
                stat[(1 * kWarps + warp) * ROWS + r] = my[t][e];
                stat[(2 * kWarps + warp) * ROWS + r] = l[t][e];
            }
            // fragment d, elements e and 2 + e: dimensions 2 d, 2 d + 1 of the
            // lane's 16 (8-bit: 16 gl + .., bf16: 8 gl + .. in each half); rotated
            // by the row, so that a store's rows do not meet in one bank
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const int dim = F8 ? 16 * gl + 2 * d : 8 * gl + 2 * (d & 3) + 64 * (d >> 2);
                *reinterpret_cast<float2 *>(po + r * 128 + ((dim + 8 * r) & 127)) = make_float2(o[t][d][e], o[t][d][2 + e]);
            }
        }
    __syncthreads();
    // eight threads a row, 16 dimensions each
    const int r = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * 16;
    if (r >= nrows) return;
    float Mx = kNone, My = kNone, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        Mx = fmaxf(Mx, stat[w * ROWS + r]);
        My = fmaxf(My, stat[(kWarps + w) * ROWS + r]);
    }
    float acc[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) acc[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float ax = stat[w * ROWS + r], ay = stat[(kWarps + w) * ROWS + r];
        const float lw = stat[(2 * kWarps + w) * ROWS + r];
        if (lw == 0.f) continue;                                 // saw nothing
        L += lw * exp2f(ax - Mx);
        const float f = exp2f(ay - My);
        const float *src = reinterpret_cast<const float *>(smem) + (w * ROWS + r) * 128;
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
            const float4 z = *reinterpret_cast<const float4 *>(src + ((d0 + k + 8 * r) & 127));
            acc[k] += f * z.x;
            acc[k + 1] += f * z.y;
            acc[k + 2] += f * z.z;
            acc[k + 3] += f * z.w;
        }
    }
    const int gr = ROWS * tile + r, tok = gr / p.G, h = g * p.G + gr % p.G;
    const size_t row = (size_t)q0 + tok;
    // O is in units of 2^My, the sum in units of 2^Mx
    const float unit = Mx == kNone ? 0.f : exp2f(My - Mx);
    if (partial) {
        const size_t pr = ((size_t)piece * p.T + row) * p.Hq + h;
        if (d0 == 0) p.part_ml[pr] = make_float2(L == 0.f ? -INFINITY : Mx, L);
#pragma unroll
        for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4 *>(p.part_o + pr * 128 + d0 + k) =
                make_float4(acc[k] * unit, acc[k + 1] * unit, acc[k + 2] * unit, acc[k + 3] * unit);
        return;
    }
    if (d0 == 0) {
        if (p.splits > 1) p.part_ml[row * p.Hq + h] = make_float2(0.f, -1.f);
        p.lse[(size_t)h * p.T + row] = L != L ? L : (L > 0.f ? (Mx + log2f(L)) * kLn2 : -INFINITY);
    }
    const float f = L > 0.f ? unit / L : 0.f;                    // a row that sees nothing gives zeros
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = tc::pack_bf16(acc[2 * k] * f, acc[2 * k + 1] * f);
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + (row * p.Hq + h) * 128 + d0);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// The kernel's shared-memory limit, set once per device.
template <bool F8, int NB>
cudaError_t prepare() {
    static std::atomic<unsigned long long> done[2]{};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 128 && (done[dev >> 6].load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(ragged_rows<F8, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<F8>::smem);
    if (e == cudaSuccess && dev < 128) done[dev >> 6].fetch_or(bit, std::memory_order_release);
    return e;
}

template <bool F8, int NB>
cudaError_t go(const Params &p, unsigned blocks, cudaStream_t st) {
    const cudaError_t e = prepare<F8, NB>();
    if (e != cudaSuccess) return e;
    ragged_rows<F8, NB><<<blocks, 32 * kWarps, Cfg<F8>::smem, st>>>(p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace
}  // namespace rows

cudaError_t ragged_rows_launch(const RaggedCall &a, const RaggedPlan &pl, void *ws, cudaStream_t st) {
    using namespace rows;
    Params p{};
    p.c = a.cache;
    p.T = a.T; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.tiles = pl.tiles;
    p.splits = pl.splits; p.chunk = pl.chunk;
    p.scale_log2 = a.scale * kLog2e;
    p.q = (const __nv_bfloat16 *)a.q; p.ld_q = a.ld_q;
    p.out = (__nv_bfloat16 *)a.out; p.lse = a.lse;
    p.status = (unsigned int *)ws;
    if (pl.splits > 1) {
        p.part_ml = reinterpret_cast<float2 *>((char *)ws + pl.ml_off);
        p.part_o = reinterpret_cast<float *>((char *)ws + pl.o_off);
    }
    const long long blocks = (long long)a.B * p.splits * p.tiles * p.Hkv;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    const bool f8 = a.cache.dtype == HS_E4M3;
    if (pl.tile_rows == 8) return f8 ? go<true, 1>(p, (unsigned)blocks, st) : go<false, 1>(p, (unsigned)blocks, st);
    return f8 ? go<true, 2>(p, (unsigned)blocks, st) : go<false, 2>(p, (unsigned)blocks, st);
}

}  // namespace hs
