// The memory-bound operators around the attention calls: rotary positions,
// the write of new keys and values into paged caches (copied, or as 8-bit
// floats under a power-of-two scale per row and head) and its counterpart
// that reads rows back.  Each input byte is read once and each output byte
// written once, in 16-byte accesses where the layout has them: 8-bit rows go in
// 8 bytes a lane, rotated parts whose halves are no multiple of 16 bytes in
// fewer, and the write reads a key again where half of its rotated part is no
// multiple of 8 elements.  Rope and the read run at the copy's rate (6.3 and 6.4
// TB/s); the write does copied (16959 tokens of 8 heads 25.7 us, 5.4 TB/s), but
// turning (37 us), 8-bit rows (35 us) or both (47 us) are bound by instructions
// and by the chains of shuffles.
#include <atomic>

#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"
#include "ragged.cuh"

namespace hs {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ rope

struct RopeParams {
    int T, Hq, Hkv, d, half;
    long long ld_q, ld_k, ld_oq, ld_ok;
    const void *q, *k;
    void *oq, *ok;
    const int32_t *positions;
    const double *inv_freq;
    float amp;
    int inverse;
    int units;      // units of one row that need work (pairs, and the part left as it is when it has to be copied)
    int tokens;     // tokens a block takes
    int dt, dh, du; // what a thread's next unit is further: tokens, heads, units
};

// Units a thread has in flight (65536 tokens of 68 heads, bf16: one 365 us, two
// 362, three 378, four 377; the part of 64 of their 128 elements 423, 402, 422,
// 413).  362 us is 6.3 TB/s, 0.96 of the copy's rate; with the units' places by
// division and the angles before the first loads it was 409 and 696.
constexpr int kRopeBatch = 2;

// As many bytes as they lie in memory.
template <int N> struct RawBytes;
template <> struct RawBytes<16> { uint4 q; };
template <> struct RawBytes<8> { uint2 q; };
template <> struct RawBytes<4> { uint32_t q; };
template <> struct RawBytes<2> { uint16_t q; };

// One unit of a row: V pairs (first and second halves: 2 V elements) or V
// neighbouring elements (V / 2 pairs), or V elements that are only copied.
template <typename T, int V, bool INTER>
struct RopeUnit {
    using Raw = RawBytes<V * (int)sizeof(T)>;
    Raw a, b;
    T *dst;         // null: no unit
    int cs;         // its first pair's angles, < 0: copy
    __device__ void load(const RopeParams &p, int t0, int tok, int head, int u) {
        const long long t = t0 + tok;
        const T *src;
        if (head < p.Hq) {
            src = (const T *)p.q + t * p.ld_q + head * p.d;
            dst = (T *)p.oq + t * p.ld_oq + head * p.d;
        } else {
            src = (const T *)p.k + t * p.ld_k + (head - p.Hq) * p.d;
            dst = (T *)p.ok + t * p.ld_ok + (head - p.Hq) * p.d;
        }
        int at = u * V;
        const bool turned = at < (INTER ? 2 * p.half : p.half);
        cs = turned ? tok * p.half + (INTER ? at / 2 : at) : -1;
        if (!INTER && !turned) at += p.half;   // units from half / V on are the rest, elements 2 * half ..
        a = *reinterpret_cast<const Raw *>(src + at);
        if (!INTER && turned) b = *reinterpret_cast<const Raw *>(src + at + p.half);
        dst += at;
    }
    static __device__ void widen(const Raw &r, float (&x)[V]) {
        const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = Elem<T>::to_f(e[i]);
    }
    __device__ void store(const RopeParams &p, const float2 *angles) const {
        if (cs < 0) {
            *reinterpret_cast<Raw *>(dst) = a;
            return;
        }
        float x[V], y[V];
        widen(a, x);
        const float2 *w = angles + cs;
        if (INTER) {
#pragma unroll
            for (int e = 0; e + 1 < V; e += 2) {
                const float f = x[e], g = x[e + 1];
                x[e] = rope_first(f, g, w[e / 2]);
                x[e + 1] = rope_second(f, g, w[e / 2]);
            }
        } else {
            widen(b, y);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float f = x[e], g = y[e];
                x[e] = rope_first(f, g, w[e]);
                y[e] = rope_second(f, g, w[e]);
            }
            store_n<V>(dst + p.half, y);
        }
        store_n<V>(dst, x);
    }
};

// The angles depend on the token and the pair only, so a block computes them
// once for its tokens (in 64 bits, into shared memory) and turns all the
// heads of q and k with them; a thread's first units are asked for before
// that.  A unit is read whole before any of it is written, so out may be the
// input itself.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
    extern __shared__ float2 cs[];
    const int t0 = blockIdx.x * p.tokens;
    const int nt = min(p.tokens, p.T - t0);
    const int heads = p.Hq + p.Hkv;
    // this thread's next unit: one division, then steps
    const int i0 = blockIdx.y * kThreads + threadIdx.x;
    int u = i0 % p.units, head = i0 / p.units, tok = head / heads;
    head -= tok * heads;
    RopeUnit<T, V, INTER> w[kRopeBatch];
    auto ask = [&]() {
#pragma unroll
        for (int e = 0; e < kRopeBatch; ++e) {
            w[e].dst = nullptr;
            if (tok < nt) w[e].load(p, t0, tok, head, u);
            u += p.du;
            head += p.dh;
            tok += p.dt;
            if (u >= p.units) {
                u -= p.units;
                ++head;
            }
            if (head >= heads) {
                head -= heads;
                ++tok;
            }
        }
    };
    ask();
    for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
        float2 v = rope_cs(__ldg(p.positions + t0 + i / p.half), p.inv_freq[i % p.half], p.amp);
        if (p.inverse) v.y = -v.y;
        cs[i] = v;
    }
    __syncthreads();
    while (w[0].dst != nullptr) {
#pragma unroll
        for (int e = 0; e < kRopeBatch; ++e)
            if (w[e].dst != nullptr) w[e].store(p, cs);
        ask();
    }
}

template <typename T, int V, bool INTER>
cudaError_t rope_go(RopeParams p, bool copy_rest, cudaStream_t st) {
    p.units = INTER ? (copy_rest ? p.d : 2 * p.half) / V : (copy_rest ? p.d - p.half : p.half) / V;
    const long long per_token = (long long)(p.Hq + p.Hkv) * p.units;
    // one token a block while that leaves SMs idle, then eight: fewer blocks,
    // and the angles of eight tokens fill the block's threads (65536 tokens of
    // 68 heads: four 374 us, eight 362)
    p.tokens = p.T >= 4096 ? 8 : 1;
    const int blocks = (p.T + p.tokens - 1) / p.tokens;
    const long long n = per_token * p.tokens;
    int y = (int)((n + 2 * kThreads - 1) / (2 * kThreads));
    if (blocks >= 592) y = 1;          // four blocks an SM: the heads need no further split
    y = y < 1 ? 1 : (y > 8 ? 8 : y);
    const int step = kThreads * y;
    p.dt = (int)(step / per_token);
    p.dh = (int)(step % per_token) / p.units;
    p.du = (int)(step % per_token) % p.units;
    rope_kernel<T, V, INTER><<<dim3(blocks, y), kThreads, p.tokens * p.half * sizeof(float2), st>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t rope_typed(const RopeParams &p, bool interleaved, bool copy_rest, cudaStream_t st) {
    constexpr int W = 16 / (int)sizeof(T);
    // the widest access that the pairs' layout allows: 16 bytes where the
    // rotated part (or each half of it) is a multiple of that
    const int unit = interleaved ? 2 * p.half : p.half;
    if (interleaved) {
        if (unit % W == 0) return rope_go<T, W, true>(p, copy_rest, st);
        return rope_go<T, 2, true>(p, copy_rest, st);
    }
    if (unit % W == 0) return rope_go<T, W, false>(p, copy_rest, st);
    if (unit % 4 == 0) return rope_go<T, 4, false>(p, copy_rest, st);
    return rope_go<T, 1, false>(p, copy_rest, st);
}

// ------------------------------------------------------------------ cache write

struct WriteParams {
    PagedCache c;
    int T, Hkv, d, half;          // half: rotated pairs of a key (0: none)
    int cs_ld;                     // floats of cosines and sines for each token
    int group_shift, dq, dr;       // lanes of a row (log2); tokens and heads that a block's rows advance by
    long long ld_k, ld_v;
    const void *k, *v;
    const double *inv_freq;
    float amp;
    int interleaved;
    unsigned int *status;
    int tokens;                    // tokens a block takes
};

// Eight neighbouring elements of a row as they lie in memory.
template <typename T> struct Raw8 {
    uint4 q[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
        const T *e = reinterpret_cast<const T *>(q);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = Elem<T>::to_f(e[i]);
    }
    __device__ __forceinline__ Raw8 shuffle(int src) const {
        Raw8 r;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            r.q[i].x = __shfl_sync(0xffffffffu, q[i].x, src);
            r.q[i].y = __shfl_sync(0xffffffffu, q[i].y, src);
            r.q[i].z = __shfl_sync(0xffffffffu, q[i].z, src);
            r.q[i].w = __shfl_sync(0xffffffffu, q[i].w, src);
        }
        return r;
    }
};

// The rotated part of elements e0 .. e0 + 7 (d and e0 are multiples of 8) of
// a key row, x, turned in place.  cs: cosines, sines and negative sines of
// the token's pairs, half of each.  y: the elements half further or half back, when half is
// a multiple of 8 (they are another lane's); otherwise `row` is read again.
template <typename T>
__device__ __forceinline__ void turn8(float (&x)[8], const float (&y)[8], const T *row, int e0, int half, bool inter,
                                      const float *cs) {
    if (e0 >= 2 * half) return;
    const float *sn = cs + half;
    if (inter) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            if (e0 + i < 2 * half) {
                const float2 w = make_float2(cs[(e0 + i) / 2], sn[(e0 + i) / 2]);
                const float a = x[i], b = x[i + 1];
                x[i] = rope_first(a, b, w);
                x[i + 1] = rope_second(a, b, w);
            }
        }
        return;
    }
    if ((half & 7) == 0) {
        // the first half's x cos - y sin is x cos + y (-sin), and the negative
        // sines lie after the sines: no lane has to choose
        const bool first = e0 < half;
        const int p0 = first ? e0 : e0 - half;
        const float *sg = sn + (first ? half : 0);
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(cs + p0 + i), s = *reinterpret_cast<const float4 *>(sg + p0 + i);
            const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i + k] = rope_second(y[i + k], x[i + k], make_float2(cc[k], ss[k]));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = e0 + i;
        if (e < half) x[i] = rope_first(x[i], Elem<T>::to_f(row[e + half]), make_float2(cs[e], sn[e]));
        else if (e < 2 * half)
            x[i] = rope_second(Elem<T>::to_f(row[e - half]), x[i], make_float2(cs[e - half], sn[e - half]));
    }
}

// The larger of two; NaN when one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The exponent byte (e + 127) of the smallest power of two 2^e with
// amax <= 448 * 2^e, 448 being the largest 8-bit float; 2^0 for a row of
// zeros, 255 when amax is NaN.  448 = 1.75 * 2^8, so e follows from amax's own exponent and from
// whether its mantissa is above 1.75.
__device__ __forceinline__ int scale_byte(float amax) {
    if (!(amax > 0.f)) return amax == amax ? 127 : 255;
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e < 1 ? 1 : e;
}

constexpr int kBatch = 4;          // rows a thread of the write has in flight
constexpr int kWriteTokens = 8;    // most tokens a block of it takes
static_assert(kWriteTokens <= kThreads / 32, "a warp finds each token's place");

// One group of lanes per (token, K or V, head) row, eight elements a lane.
// 8-bit rows: the group's largest magnitude gives the scale, a power of two,
// so that dividing by it is exact and the 8-bit float is the only rounding
// (by at most 2^-4 of the value); every reader can widen such a value to bf16
// exactly.
//
// The rows themselves are asked for first, kBatch of them a thread: the
// places of the tokens (three dependent loads) and the angles (64-bit
// arithmetic) are found while they come.
template <typename TI, typename TO, bool Q8>
__global__ void __launch_bounds__(kThreads, 4) cache_write_kernel(const WriteParams p) {
    extern __shared__ __align__(16) float wcs[];   // per token: cosines, sines, negative sines
    __shared__ size_t data_at[kWriteTokens];       // the token's place in the pools, in elements
    __shared__ size_t scale_at[kWriteTokens];      // and its first head's scale
    __shared__ int at[kWriteTokens];               // its position; < 0: it has no place
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.tokens;
    const int nt = min(p.tokens, p.T - t0);
    const int lanes = p.d / 8;                     // lanes that hold a row, of a group of 2^group_shift
    const int group = 1 << p.group_shift;
    const int sub = threadIdx.x & (group - 1);
    const int per = kThreads >> p.group_shift;     // rows a block handles at a time
    const int heads = 2 * p.Hkv;                   // rows of a token: K heads, then V heads
    const TI *const kb = (const TI *)p.k + (long long)t0 * p.ld_k + sub * 8;
    const TI *const vb = (const TI *)p.v + (long long)t0 * p.ld_v + sub * 8;
    // this thread's next row, as token and head of the block: one division,
    // then steps of `per` rows (dq tokens and dr heads)
    struct Row {
        int tok, kh;
        __device__ __forceinline__ void next(const WriteParams &p, int heads) {
            tok += p.dq;
            kh += p.dr;
            if (kh >= heads) {
                kh -= heads;
                ++tok;
            }
        }
    };
    Row asked;
    asked.tok = (int)(threadIdx.x >> p.group_shift) / heads;
    asked.kh = (int)(threadIdx.x >> p.group_shift) - asked.tok * heads;
    Row row = asked;
    Raw8<TI> raw[kBatch];
    auto ask = [&]() {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (asked.tok < nt && sub < lanes)
                raw[u].load(asked.kh >= p.Hkv ? vb + asked.tok * p.ld_v + (asked.kh - p.Hkv) * p.d
                                              : kb + asked.tok * p.ld_k + asked.kh * p.d);
            else raw[u].zero();
            asked.next(p, heads);
        }
    };
    ask();
    if (warp < nt) {                               // one warp finds each token's place
        int b = 0;
        const long long pos = cache_position(p.c, p.T, t0 + warp, p.status, &b);
        const long long r = pos < 0 ? -1 : pool_row(p.c, b, pos, p.status);
        if (lane == 0) {
            at[warp] = r < 0 ? -1 : (int)pos;
            data_at[warp] = r < 0 ? 0 : (size_t)r * p.Hkv * p.d;
            scale_at[warp] = r < 0 ? 0 : scale_index(p.c, r, p.Hkv, 0);
        }
    }
    __syncthreads();
    if (p.half > 0) {
        for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
            const int tok = i / p.half, pair = i - tok * p.half;
            if (at[tok] >= 0) {
                const float2 w = rope_cs(at[tok], p.inv_freq[pair], p.amp);
                wcs[tok * p.cs_ld + pair] = w.x;
                wcs[tok * p.cs_ld + p.half + pair] = w.y;
                wcs[tok * p.cs_ld + 2 * p.half + pair] = -w.y;
            }
        }
        __syncthreads();
    }
    const int passes = (nt * heads + per - 1) >> (8 - p.group_shift);      // per = 2^(8 - group_shift)
    for (int i0 = 0; i0 < passes; i0 += kBatch) {
        if (i0 > 0) ask();
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (i0 + u >= passes) break;                               // (the same for the whole block)
            const int tok = min(row.tok, nt - 1), kh = row.kh;
            const bool is_v = kh >= p.Hkv;
            const bool live = row.tok < nt && sub < lanes && at[tok] >= 0;
            row.next(p, heads);
            float x[8];
            raw[u].widen(x);
            if (p.half > 0 && __any_sync(0xffffffffu, live && !is_v)) {
                float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (!p.interleaved && (p.half & 7) == 0) {             // the partners are another lane's
                    const int hl = p.half / 8;
                    raw[u].shuffle((lane & ~(group - 1)) + (sub < hl ? sub + hl : max(sub - hl, 0))).widen(y);
                }
                if (live && !is_v)
                    turn8(x, y, kb - sub * 8 + tok * p.ld_k + kh * p.d, sub * 8, p.half, p.interleaved != 0,
                          wcs + tok * p.cs_ld);
            }
            [[maybe_unused]] int byte = 127;
            if constexpr (Q8) {
                float m = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
                for (int o = group >> 1; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                byte = scale_byte(m);
            }
            if (!live) continue;
            const int h = is_v ? kh - p.Hkv : kh;
            const size_t o = data_at[tok] + (h * p.d + sub * 8);
            if constexpr (Q8) {
                // 2^-e, e <= 120; NaN, which makes every code NaN, for a row that holds one
                const float inv = __uint_as_float(byte == 255 ? 0x7fc00000u : (uint32_t)(254 - byte) << 23);
                uint2 w;
                __nv_fp8x2_storage_t c[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE,
                                                    __NV_E4M3);
                w.x = (uint32_t)c[0] | ((uint32_t)c[1] << 16);
                w.y = (uint32_t)c[2] | ((uint32_t)c[3] << 16);
                *reinterpret_cast<uint2 *>((uint8_t *)(is_v ? p.c.v_pages : p.c.k_pages) + o) = w;
                if (sub == 0)
                    (is_v ? p.c.v_scale : p.c.k_scale)[scale_at[tok] + ((size_t)h << p.c.page_shift)] = (uint8_t)byte;
            } else {
                store_n<8>((TO *)(is_v ? p.c.v_pages : p.c.k_pages) + o, x);
            }
        }
    }
}

template <typename TI, typename TO, bool Q8>
cudaError_t write_go(WriteParams p, cudaStream_t st) {
    // eight tokens a block once that still gives every SM several blocks: what a
    // block does besides its rows (places, angles) is then an eighth (16959
    // tokens of 8 heads, copied: four tokens 27.3 us, eight 25.5)
    p.tokens = p.T >= 4096 ? kWriteTokens : 1;
    p.cs_ld = (3 * p.half + 3) & ~3;               // whole 16-byte units for each token
    p.group_shift = 0;                             // lanes of a row, rounded up to a power of two (<= 32)
    while ((8 << p.group_shift) < p.d) ++p.group_shift;
    p.dq = (kThreads >> p.group_shift) / (2 * p.Hkv);
    p.dr = (kThreads >> p.group_shift) % (2 * p.Hkv);
    cache_write_kernel<TI, TO, Q8><<<(p.T + p.tokens - 1) / p.tokens, kThreads,
                                     (size_t)p.tokens * p.cs_ld * sizeof(float), st>>>(p);
    count_launch();
    return cudaGetLastError();
}

// ------------------------------------------------------------------ cache read

struct ReadParams {
    PagedCache c;
    const int32_t *start;
    int total, Hkv, d;
    void *k, *v;
    unsigned int *status;
    int tokens;
    int group_shift, dq, dr;       // as in WriteParams
};

// Most packed rows a block takes, and rows a thread of it has in flight, of K
// and of V (24 caches of 16384, e4m3 to bf16, 8 heads: 8 rows and 1, 2, 4 in
// flight 186, 183, 181 us; 16 rows 188, 186, 183; but 64 elements a head 105,
// 95, 113.  183 us is 6.4 TB/s, the copy's rate; with 16 elements a thread,
// whose two stores each fill half of a 32-byte sector, it was 208).
constexpr int kReadTokens = 8, kReadBatch = 2;

// Eight neighbouring elements of a cache row and its scale.
template <typename TC> struct CacheRaw8 : Raw8<TC> {
    __device__ __forceinline__ void widen_scaled(float (&x)[8], float) const { this->widen(x); }
};
template <> struct CacheRaw8<__nv_fp8_e4m3> {
    uint2 q;
    __device__ __forceinline__ void load(const __nv_fp8_e4m3 *p) { q = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void widen_scaled(float (&x)[8], float scale) const {
        const uint32_t w[2] = {q.x, q.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2_raw h =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i & 1))), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = f.x * scale;
            x[2 * i + 1] = f.y * scale;
        }
    }
};

template <typename TC, typename TO, bool Q8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const ReadParams p) {
    __shared__ long long slot[kReadTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * p.tokens;
    const int nt = min(p.tokens, p.total - t0);
    for (int i = warp; i < nt; i += kThreads / 32) {
        const int row = t0 + i;
        const int b = seq_of_row(p.c.cu_rows, p.c.B, row);
        long long r = -1;
        if (b >= 0 && row < __ldg(p.c.cu_rows + b + 1)) {
            const long long pos = (long long)row - __ldg(p.c.cu_rows + b) + (p.start ? __ldg(p.start + b) : 0);
            if (pos < 0 || pos >= ((long long)p.c.max_pages << p.c.page_shift)) report(p.status, HS_ERR_INVALID_ARG);
            else r = pool_row(p.c, b, pos, p.status);
        }
        if (lane == 0) slot[i] = r;
    }
    __syncthreads();
    // one group of lanes per (token, head) row of K and of V, eight elements a lane
    const int group = 1 << p.group_shift, sub = threadIdx.x & (group - 1);
    int tok = (int)(threadIdx.x >> p.group_shift) / p.Hkv, h = (int)(threadIdx.x >> p.group_shift) - tok * p.Hkv;
    while (tok < nt) {
        CacheRaw8<TC> k[kReadBatch], v[kReadBatch];
        int kb[kReadBatch], vb[kReadBatch];
        size_t dst[kReadBatch];
        bool live[kReadBatch];
#pragma unroll
        for (int u = 0; u < kReadBatch; ++u) {
            const long long r = tok < nt ? slot[tok] : -1;
            live[u] = r >= 0 && sub * 8 < p.d;
            dst[u] = ((size_t)(t0 + tok) * p.Hkv + h) * p.d + sub * 8;
            if (live[u]) {
                const size_t src = ((size_t)r * p.Hkv + h) * p.d + sub * 8;
                k[u].load((const TC *)p.c.k_pages + src);
                v[u].load((const TC *)p.c.v_pages + src);
                if (Q8) {
                    const size_t si = scale_index(p.c, r, p.Hkv, h);
                    kb[u] = p.c.k_scale[si];
                    vb[u] = p.c.v_scale[si];
                }
            }
            tok += p.dq;
            h += p.dr;
            if (h >= p.Hkv) {
                h -= p.Hkv;
                ++tok;
            }
        }
#pragma unroll
        for (int u = 0; u < kReadBatch; ++u) {
            if (!live[u]) continue;
            float x[8];
            k[u].widen_scaled(x, Q8 ? scale_of_byte(kb[u]) : 1.f);
            store_n<8>((TO *)p.k + dst[u], x);
            v[u].widen_scaled(x, Q8 ? scale_of_byte(vb[u]) : 1.f);
            store_n<8>((TO *)p.v + dst[u], x);
        }
    }
}

template <typename TC, typename TO, bool Q8>
cudaError_t read_go(ReadParams p, cudaStream_t st) {
    p.tokens = p.total >= 8192 ? kReadTokens : (p.total >= 1024 ? 4 : 1);
    p.group_shift = 0;
    while ((8 << p.group_shift) < p.d) ++p.group_shift;
    p.dq = (kThreads >> p.group_shift) / p.Hkv;
    p.dr = (kThreads >> p.group_shift) % p.Hkv;
    cache_read_kernel<TC, TO, Q8><<<(p.total + p.tokens - 1) / p.tokens, kThreads, 0, st>>>(p);
    count_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t rope_launch(const RopeCall &a, cudaStream_t st) {
    RopeParams p{};
    p.T = a.T; p.Hq = a.Hq; p.Hkv = a.Hkv; p.d = a.d; p.half = a.rot / 2;
    p.q = a.q; p.k = a.k; p.oq = a.out_q; p.ok = a.out_k;
    p.ld_q = a.ld_q; p.ld_k = a.ld_k; p.ld_oq = a.ld_oq; p.ld_ok = a.ld_ok;
    p.positions = a.positions; p.inv_freq = a.inv_freq; p.amp = a.factor; p.inverse = a.inverse;
    // turned in place, the rest of each head needs no work
    const bool copy_rest = a.rot < a.d && (a.out_q != a.q || (a.Hkv > 0 && a.out_k != a.k));
    if (a.dtype == HS_F32) return rope_typed<float>(p, a.interleaved, copy_rest, st);
    return rope_typed<__nv_bfloat16>(p, a.interleaved, copy_rest, st);
}

cudaError_t cache_write_launch(const PagedCache &c, int T, int Hkv, int d, int dtype, const void *k, long long ld_k,
                               const void *v, long long ld_v, const double *inv_freq, int rot, bool interleaved,
                               float factor, unsigned int *status, cudaStream_t st) {
    WriteParams p{};
    p.c = c; p.T = T; p.Hkv = Hkv; p.d = d; p.half = inv_freq ? rot / 2 : 0;
    p.k = k; p.v = v; p.ld_k = ld_k; p.ld_v = ld_v; p.inv_freq = inv_freq; p.amp = factor;
    p.interleaved = interleaved; p.status = status;
    if (dtype == HS_F32) {
        if (c.dtype == HS_E4M3) return write_go<float, uint8_t, true>(p, st);
        if (c.dtype == HS_BF16) return write_go<float, __nv_bfloat16, false>(p, st);
        return write_go<float, float, false>(p, st);
    }
    if (c.dtype == HS_E4M3) return write_go<__nv_bfloat16, uint8_t, true>(p, st);
    if (c.dtype == HS_BF16) return write_go<__nv_bfloat16, __nv_bfloat16, false>(p, st);
    return write_go<__nv_bfloat16, float, false>(p, st);
}

cudaError_t cache_read_launch(const PagedCache &c, const int32_t *start, int total, int Hkv, int d, int dtype,
                              void *k, void *v, unsigned int *status, cudaStream_t st) {
    ReadParams p{c, start, total, Hkv, d, k, v, status, 1, 0, 0, 0};
    if (dtype == HS_F32) {
        if (c.dtype == HS_E4M3) return read_go<__nv_fp8_e4m3, float, true>(p, st);
        if (c.dtype == HS_BF16) return read_go<__nv_bfloat16, float, false>(p, st);
        return read_go<float, float, false>(p, st);
    }
    if (c.dtype == HS_E4M3) return read_go<__nv_fp8_e4m3, __nv_bfloat16, true>(p, st);
    if (c.dtype == HS_BF16) return read_go<__nv_bfloat16, __nv_bfloat16, false>(p, st);
    return read_go<float, __nv_bfloat16, false>(p, st);
}

}  // namespace hs
