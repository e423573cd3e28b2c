// Device helpers shared by the kernels over ragged batches (sequences of
// different lengths packed row after row) and paged caches: which sequence a
// packed row belongs to, which pool row a cache position is, and the rotary
// angle of a position.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace hs {

// A packed row bound from the device, kept inside the T rows that exist.
__device__ __forceinline__ int clamp_row(int r, int T) { return r < 0 ? 0 : (r > T ? T : r); }

// The last sequence b with cu[b] <= row (32-way search, every lane of the
// warp calls it with the same row), or -1.  Any contents of cu are safe: only
// cu[0 .. B-1] is read.
__device__ __forceinline__ int seq_of_row(const int32_t *cu, int B, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    while (true) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool le = i < n && __ldg(cu + lo + i) <= row;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        if (cnt == 0) return -1;
        lo += (cnt - 1) * step;
        if (step == 1) return lo;
        n = min(step, B - lo);
    }
}

// Where row r of the packed rows lies in the paged cache: its position, or a
// negative number when it has none (a row before the first or behind the last
// sequence, a position outside the cache).  Warp-wide; *seq receives the
// sequence.
__device__ __forceinline__ long long cache_position(const PagedCache &c, int T, int row, unsigned int *status,
                                                    int *seq) {
    const int b = seq_of_row(c.cu_rows, c.B, row);
    if (b < 0) return -1;
    const int q1 = __ldg(c.cu_rows + b + 1);
    if (row >= q1) return -1;
    *seq = b;
    const long long pos = (long long)__ldg(c.kv_len + b) - ((long long)q1 - row);
    if (q1 > T || pos < 0 || pos >= ((long long)c.max_pages << c.page_shift)) {
        report(status, HS_ERR_INVALID_ARG);
        return -1;
    }
    return pos;
}

// Pool row of position pos of sequence b, or -1 (reported) when its table
// entry is outside the pool.
__device__ __forceinline__ long long pool_row(const PagedCache &c, int b, long long pos, unsigned int *status) {
    const int page = __ldg(c.block_table + (size_t)b * c.max_pages + (size_t)(pos >> c.page_shift));
    if (page < 0 || page >= c.num_pages) {
        report(status, HS_ERR_INVALID_INDEX);
        return -1;
    }
    return ((long long)page << c.page_shift) | (pos & ((1ll << c.page_shift) - 1));
}

// Index of a pool row's scale byte: [page][Hkv][row in page], so that one
// head's scales are contiguous where attention reads them.
__device__ __forceinline__ size_t scale_index(const PagedCache &c, long long row, int Hkv, int h) {
    const long long page = row >> c.page_shift;
    return ((size_t)(page * Hkv + h) << c.page_shift) + (size_t)(row & ((1ll << c.page_shift) - 1));
}

// A scale byte's power of two.  Byte 0 would be 2^-127 (not a normal float)
// and is never written here; it reads as that all the same.
__device__ __forceinline__ float scale_of_byte(int byte) {
    return byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)byte << 23);
}

// cos and sin of pos * freq, times `amp`, each rounded once to fp32.  The
// angle is held in 64 bits: in fp32 a position near a million would be off by
// 0.06 rad.  Quarter turns are taken out of it (pi / 2 as a sum of two
// doubles), and the rest, within pi / 4, goes through the Taylor series of
// sine and cosine up to x^11 and x^12, whose remainders are below 7e-12 and
// 4e-13: fp32's rounding is then the only one that counts, at a tenth of the
// instructions that the library's 64-bit sine and cosine take.
__device__ __forceinline__ float2 rope_cs(int pos, double freq, float amp) {
    const double t = (double)pos * freq;
    const double quarters = rint(t * 0.63661977236758134);
    double x = fma(-quarters, 1.5707963267948966, t);
    x = fma(-quarters, 6.123233995736766e-17, x);
    const double z = x * x;
    double s = fma(z, -1.0 / 39916800.0, 1.0 / 362880.0);
    s = fma(z, s, -1.0 / 5040.0);
    s = fma(z, s, 1.0 / 120.0);
    s = fma(z, s, -1.0 / 6.0);
    s = fma(z * x, s, x);
    double c = fma(z, 1.0 / 479001600.0, -1.0 / 3628800.0);
    c = fma(z, c, 1.0 / 40320.0);
    c = fma(z, c, -1.0 / 720.0);
    c = fma(z, c, 1.0 / 24.0);
    c = fma(z, c, -0.5);
    c = fma(z, c, 1.0);
    const int q = (int)__double2ll_rn(quarters) & 3;
    const float fs = (float)s, fc = (float)c;
    const float co = (q & 1) ? fs : fc, si = (q & 1) ? fc : fs;
    return make_float2(__fmul_rn((q == 1 || q == 2) ? -co : co, amp), __fmul_rn(q >= 2 ? -si : si, amp));
}

// One rotated pair.  Products and sums are rounded one by one (no fused
// multiply-add), so that a rotation is the same in every kernel here and a
// value at the border of two 8-bit codes gets the same code in all of them.
__device__ __forceinline__ float rope_first(float a, float b, float2 cs) {
    return __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
}
__device__ __forceinline__ float rope_second(float a, float b, float2 cs) {
    return __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
}

// N consecutive elements (N * sizeof(T) a power of two up to 32 bytes, aligned
// to min(that, 16)) as floats.
template <int N, typename T>
__device__ __forceinline__ void load_n(const T *p, float (&f)[N]) {
    constexpr int BYTES = N * (int)sizeof(T);
    union {
        uint4 q[(BYTES + 15) / 16];
        uint2 d;
        uint32_t w;
        T e[N];
    } u;
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) u.q[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else if constexpr (BYTES == 8) {
        u.d = *reinterpret_cast<const uint2 *>(p);
    } else if constexpr (BYTES == 4) {
        u.w = *reinterpret_cast<const uint32_t *>(p);
    } else {
        u.e[0] = p[0];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(u.e[i]);
}

template <int N, typename T>
__device__ __forceinline__ void store_n(T *p, const float (&f)[N]) {
    constexpr int BYTES = N * (int)sizeof(T);
    union U {
        uint4 q[(BYTES + 15) / 16];
        uint2 d;
        uint32_t w;
        T e[N];
        __device__ U() {}
    } u;
#pragma unroll
    for (int i = 0; i < N; ++i) u.e[i] = Elem<T>::from_f(f[i]);
    if constexpr (BYTES >= 16) {
#pragma unroll
        for (int i = 0; i < BYTES / 16; ++i) reinterpret_cast<uint4 *>(p)[i] = u.q[i];
    } else if constexpr (BYTES == 8) {
        *reinterpret_cast<uint2 *>(p) = u.d;
    } else if constexpr (BYTES == 4) {
        *reinterpret_cast<uint32_t *>(p) = u.w;
    } else {
        p[0] = u.e[0];
    }
}

}  // namespace hs
