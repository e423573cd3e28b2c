// Causal attention over ragged batches on the tcgen05 tensor cores (bf16
// queries, head dim 128): whole packed prompts, and chunks of new tokens
// (from one a sequence to thousands) over paged caches of bf16 or of 8-bit
// floats with power-of-two scales.
//
//   out[t,h] = sum_j softmax_j(scale * q[t,h].k[j,h/G]) v[j,h/G],  j <= pos(t)
//   lse[h,t] = ln sum_j exp(scale * q[t,h].k[j,h/G])
//
// Work item.  The query heads of a KV group are rows like the tokens are: a
// 128-row tile holds 128 / G tokens x G heads of one KV head (row = token * G
// + head, which is how a {64, G, 128 / G} TMA box lands), so one token fills
// G rows, any G up to 32 works, and a tile's causal edge spans 128 / G
// tokens.  A CTA takes two such tiles of one sequence and KV head, so each
// K/V tile is loaded once for 256 rows.  When only the first tile has tokens
// (decode, short chunks) both softmax warpgroups share it and take the key
// tiles in turn ("solo"); their results are joined at the end.
// A piece of at most `chunk` key tiles is one item; sequences with more keys
// are split over several items, whose partial results a second kernel joins.
//
// One CTA per SM runs through its share of the items (longest first, dealt
// forth and back), so that an item's loads and first products run under the
// softmax and the stores of the one before.  CTA (warps):
//   0-3, 4-7  softmax warpgroups, thread = row
//   8         TMA producer (Q once; K and V tiles, or the pages that make one
//             up, in the order the MMAs consume them)
//   9, 10     MMA issuers of row tile 0 and 1
//   11        finds the items, two ahead
//   12-15     8-bit caches only: widen staged rows to bf16 tiles.  A code
//             times a power of two from 2^-124 to 2^119 is a bf16 number, so
//             nothing is rounded there.  Their instructions are what bounds
//             8-bit chunks (430 to 435 us for 4 of 1000 over 12000, 365 to 377
//             with bf16 pages).
// TMEM (512 columns): two S buffers of 64 keys for each row tile, then O0 and
// O1.  A key tile is taken in two steps of 64 keys, so that S of the next step
// is computed while the softmax of this one runs: with one 128-key S per row
// tile the softmax would wait for P V and the next Q K^T each time (measured
// 4300 clocks a pair of tiles against 2048 of products).  P overwrites its S
// buffer and is the MMA's A operand there: P in shared memory would add its
// writes and reads to an operand traffic that already fills the 128 bytes a
// clock (64-key Q K^T: 48 KB in 256 clocks of products).
// Bound: the softmax's chain of load, maximum, exponentials and store, with two
// warps a scheduler: ~4000 clocks a pair of tiles against 2476 of products at
// this step (8192-token prompt, 64/4 heads: 960 us, 1145 TFLOP/s, while the clock
// is up; 1060 to 1140 us from call to call at the power limit).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "common.cuh"
#include "internal.h"
#include "ragged.cuh"
#include "tc_attn.cuh"
#include "tc_util.cuh"

namespace hs {
namespace tc {
namespace {

constexpr int kStage = TILE / 2;       // one 128-key tile of 8-bit rows: 16 KB
constexpr int kBadBufs = 8;
constexpr int kMaxSplits = 64;         // pieces of a row at most

// Shared memory: Q0, Q1, four K/V tiles (for 8-bit caches three, and two
// staged 8-bit tiles), and 4 KB for each softmax warp's results on their way
// out.
template <bool F8> struct Ring {
    static constexpr int slots = F8 ? 3 : 4;
    static constexpr int stages = F8 ? 2 : 0;
    static_assert(slots <= 4 && stages <= 2, "RaggedBars");
    static constexpr int threads = F8 ? 512 : 384;
    // launch registers and shares after the hand-over (setmaxnreg): the
    // shares add up to at most what the block was launched with
    static constexpr int launch = F8 ? 128 : 168;
    static constexpr int ctl = F8 ? 64 : 104;
    static constexpr int soft = F8 ? 192 : 200;
    static_assert(256 * soft + (threads - 256) * ctl <= threads * launch, "register hand-over over budget");
    static_assert(launch * threads <= 65536, "launch registers");
};

struct Work {
    int q0, ql, kvl;           // the sequence's first packed row, its rows, its keys
    int b, g, piece;           // sequence, KV head, piece
    int t0;                    // first token of the item (within the sequence)
    int off;                   // position of token 0 of the sequence (kvl - ql; may be negative)
    int j0, n, n0, n1;         // first key tile; tiles of the item, of row tile 0 and 1
    int solo, partial;
    int go;                    // 0: no more items
};

struct RaggedBars {
    uint64_t q_full, q_empty;             // q_empty: the MMAs have read Q (commit), and a warpgroup has no use for its place
    uint64_t kv_full[4], kv_empty[4];     // K/V tiles (Ring::slots of them)
    uint64_t st_full[2], st_empty[2];     // staged 8-bit tiles
    uint64_t s_full[2][2], p_full[2][2];  // of each S buffer
    uint64_t pv_done[2];                  // each step's P V
    uint64_t o_full[2], o_empty[2];       // an item's last P V; O read out
    uint64_t work_full[2], work_empty[2];
    uint64_t q_read;                      // solo: issuer 0's last product with the shared Q tile is done
    uint64_t side_full;                   // solo: warpgroup 1's half is in shared memory
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    uint32_t bad_any[kBadBufs];           // K tile i of the CTA has boxes on pages outside the pool: bad[i % 8] says which
    uint32_t bad[kBadBufs][4];            // (a bit for each box)
    uint8_t scale[2][128];                // scale bytes of the staged tiles
    float2 side[128];                     // solo: warpgroup 1's maximum and sum of each row
    Work work[2];
};

constexpr size_t kRaggedSmem = 1024 + 7 * TILE + sizeof(RaggedBars);
static_assert(kRaggedSmem <= 232448, "ragged attention shared memory");

struct RaggedParams {
    PagedCache c;              // cu_rows, B; paged: kv_len, block_table, pages, scales
    int paged;
    int T, Hq, Hkv, G, tpt;    // tpt: tokens per 128-row tile (128 / G)
    uint32_t g_inv;            // ceil(2^16 / G): row / G = row * g_inv >> 16 for rows below 128
    int box_rows;              // keys one TMA box brings
    int works, splits, chunk;  // work items planned for; pieces per item; key tiles per piece
    float scale_log2;
    __nv_bfloat16 *out;
    float *lse;
    float *part_o;             // [splits][T][Hq][128]
    float2 *part_ml;           // [splits][T][Hq]: max (log2 units), sum; sum < 0: written to out already
    unsigned int *status;
    unsigned long long wait_ns;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Sequence b's rows and keys, kept inside what exists whatever the device
// arrays hold.
__device__ __forceinline__ void seq_bounds(const RaggedParams &p, int b, int &q0, int &ql, int &kvl) {
    q0 = clamp_row(__ldg(p.c.cu_rows + b), p.T);
    ql = max(clamp_row(__ldg(p.c.cu_rows + b + 1), p.T) - q0, 0);
    kvl = ql;
    if (p.paged) kvl = min(max(__ldg(p.c.kv_len + b), 0), p.c.max_pages << p.c.page_shift);
}

// What the warp that finds items keeps from one to the next, so that the
// batch is read once.  Up to 32 sequences: lane b holds sequence b.  More:
// lane i holds how many row groups the sequences [i * per, (i + 1) * per)
// have, and all up to them.
struct Batch {
    int q0 = 0, ql = 0, kvl = 0;
    int sum = 0, upto = 0, per = 0;
};

__device__ __forceinline__ Batch read_batch(const RaggedParams &p) {
    const int lane = threadIdx.x & 31, B = p.c.B, qt = 2 * p.tpt;
    Batch t;
    if (B <= 32) {
        if (lane < B) seq_bounds(p, lane, t.q0, t.ql, t.kvl);
        return t;
    }
    t.per = (B + 31) / 32;
    const int first = min(lane * t.per, B), last = min(first + t.per, B);
#pragma unroll 4
    for (int i = first; i < last; ++i) {
        int q0, ql, kvl;
        seq_bounds(p, i, q0, ql, kvl);
        t.sum += (ql + qt - 1) / qt;
    }
    t.upto = t.sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, t.upto, o);
        if (lane >= o) t.upto += y;
    }
    return t;
}

// Which sequence and rows work item `idx` is (one warp).  Up to 32 sequences:
// items in descending order of their keys, so that the longest start first.
// More: in order, each sequence's last rows first; a lane holds one sequence's
// lengths only.  A batch that comes longest first then loses nothing; at random
// 64 prompts of 4 to 2000 tokens take 358 us against 331, 200 744 against 702.
__device__ __forceinline__ bool find_rows(const RaggedParams &p, const Batch &bt, int idx, Work *w) {
    const int lane = threadIdx.x & 31;
    const int qt = 2 * p.tpt;
    const int B = p.c.B;
    int b = -1, t = 0;
    if (B <= 32) {
        const int nt = (bt.ql + qt - 1) / qt;
        const int base = max(bt.kvl - bt.ql, 0) / qt;
        const int total = __reduce_add_sync(0xffffffffu, nt);
        if (idx == 0 && lane == 0 && total > p.works) report(p.status, HS_ERR_INVALID_ARG);
        if (idx >= total) return false;
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, base + nt);   // items at or past lo: > idx; past hi: none
        while (hi - lo > 1) {
            const int x = lo + (hi - lo) / 2;
            const int at = __reduce_add_sync(0xffffffffu, min(max(base + nt - x, 0), nt));
            if (at > idx) lo = x; else hi = x;
        }
        const int past = __reduce_add_sync(0xffffffffu, min(max(base + nt - lo - 1, 0), nt));
        const unsigned there = __ballot_sync(0xffffffffu, lo >= base && lo < base + nt);
        b = __fns(there, 0, idx - past + 1);
        t = lo - __shfl_sync(0xffffffffu, base, b);
        w->q0 = __shfl_sync(0xffffffffu, bt.q0, b);
        w->ql = __shfl_sync(0xffffffffu, bt.ql, b);
        w->kvl = __shfl_sync(0xffffffffu, bt.kvl, b);
    } else {
        const int total = __shfl_sync(0xffffffffu, bt.upto, 31);
        if (idx == 0 && lane == 0 && total > p.works) report(p.status, HS_ERR_INVALID_ARG);
        if (idx >= total) return false;
        // the lane whose sequences the item is among, then those, 32 at a time
        const int owner = __ffs(__ballot_sync(0xffffffffu, bt.upto > idx)) - 1;
        int left = idx - __shfl_sync(0xffffffffu, bt.upto - bt.sum, owner);
        const int first = owner * bt.per, last = min(first + bt.per, B);
        for (int i0 = first; i0 < last; i0 += 32) {
            int q0 = 0, ql = 0, kvl = 0;
            if (i0 + lane < last) seq_bounds(p, i0 + lane, q0, ql, kvl);
            const int nt = (ql + qt - 1) / qt;
            int upto = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, upto > left);
            if (past != 0) {
                const int src = __ffs(past) - 1;
                b = i0 + src;
                t = __shfl_sync(0xffffffffu, upto, src) - 1 - left;      // last rows first
                w->q0 = __shfl_sync(0xffffffffu, q0, src);
                w->ql = __shfl_sync(0xffffffffu, ql, src);
                w->kvl = __shfl_sync(0xffffffffu, kvl, src);
                break;
            }
            left -= __shfl_sync(0xffffffffu, upto, 31);
        }
        if (b < 0) return false;       // (the batch changed under the call)
    }
    w->b = b;
    if (lane == 0 && (__ldg(p.c.cu_rows + b + 1) > p.T || __ldg(p.c.cu_rows + b) < 0 ||
                      (p.paged && __ldg(p.c.kv_len + b) != w->kvl)))
        report(p.status, HS_ERR_INVALID_ARG);
    w->t0 = t * qt;
    w->off = w->kvl - w->ql;
    return true;
}

__device__ __forceinline__ int key_tiles(int last_pos) { return last_pos < 0 ? 0 : last_pos / BN + 1; }

// The i-th item of this CTA (one warp): items are numbered work, piece, KV
// head (fastest) and dealt to the CTAs forth and back.
__device__ __forceinline__ Work find_work(const RaggedParams &p, const Batch &bt, int i) {
    Work w{};
    const long long id = (long long)i * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (id >= (long long)p.works * p.splits * p.Hkv) return w;
    const int item = (int)(id / p.Hkv);
    w.g = (int)(id - (long long)item * p.Hkv);
    w.piece = item % p.splits;
    if (!find_rows(p, bt, item / p.splits, &w)) return w;
    const int nq = min(2 * p.tpt, w.ql - w.t0);
    const int nk = key_tiles(w.off + w.t0 + nq - 1);
    const int nk0 = key_tiles(w.off + w.t0 + min(p.tpt, nq) - 1);
    w.solo = nq <= p.tpt;
    w.j0 = min(w.piece * p.chunk, nk);
    // (the last piece also takes keys past the length the plan was made for)
    w.n = w.piece == p.splits - 1 ? nk - w.j0 : min(nk - w.j0, p.chunk);
    if (w.solo) {
        w.n0 = (w.n + 1) >> 1;
        w.n1 = w.n >> 1;
    } else {
        w.n0 = min(max(nk0 - w.j0, 0), w.n);
        w.n1 = w.n;
    }
    // one piece holds all the keys: no partial results for this item
    w.partial = nk > p.chunk;
    w.go = 1;
    return w;
}

// Item `it` of the K/V sequence, in the order the MMAs consume it: with two
// row tiles K0 V0 K1 V1 ...; solo, where two key tiles are in the air, K0 K1
// V0 K2 V1 ... V(n-1).
__device__ __forceinline__ void kv_item(int it, int n, bool solo, int &j, bool &is_v) {
    if (!solo) {
        j = it >> 1;
        is_v = (it & 1) != 0;
    } else if (it == 0) {
        j = 0;
        is_v = false;
    } else if (it == 2 * n - 1) {
        j = n - 1;
        is_v = true;
    } else {
        is_v = (it & 1) == 0;
        j = is_v ? (it - 2) / 2 : (it + 1) / 2;
    }
}

// Position in a ring of `slots`.
struct RingPos {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// Two of the four 8-bit floats of w to a bf16 pair scaled by 2^-120: the sign
// stays, the code's four exponent bits go to the low end of the bf16 exponent,
// whose bias is larger by 120; subnormal codes become subnormal bf16 numbers.
// The byte permutation puts each code's sign into all bits of the byte above
// it, so that one shift and one mask are left (sel: 0x9180 for the lower two).
template <int sel>
__device__ __forceinline__ uint32_t e4m3_to_bf16_tiny(uint32_t w) {
    uint32_t t;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(t) : "r"(w), "n"(sel));
    return (t << 4) & 0x87f087f0u;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One lane of the warp, the same each time.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r;
}

// Shared-memory descriptors (sdesc_sw128) in two words: the low one holds the
// address / 16 and the leading byte offset / 16, the high one is the same for
// every operand here (stride 1024 bytes, version 1, 128-byte swizzle).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescLboK = 16 >> 4;                    // K-major operands: not used by the 128-byte swizzle
constexpr uint32_t kDescLboV = (HALF >> 4) - kDescLboK;    // what a value tile (N-major) has more: its halves lie 16 KB apart
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr) { return ((addr >> 4) & 0x3fffu) | (kDescLboK << 16); }

// mma_ss / mma_ts / mma_commit by the lane with leader != 0; every lane of
// the warp calls them.
__device__ __forceinline__ void mma_ss_one(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t a_hi, uint32_t b_hi,
                                           uint32_t idesc, uint32_t accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %4};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts_one(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                           uint32_t accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}

// mbar_wait for warps that share their scheduler with others' arithmetic:
// the first poll does not suspend the thread (with a limit of 0 the wait
// gives up whenever the phase is not complete yet), the others suspend it
// for up to kSuspendNs, so that waiting takes no issue slots.
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int *abort) {
    uint32_t there;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(there)
        : "r"(bar), "r"(parity)
        : "memory");
    if (there) return true;
    if (limit_ns == 0) {
        *abort = 1;
        return false;
    }
    const uint64_t t0 = globaltimer();
    while (true) {
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(there)
            : "r"(bar), "r"(parity), "r"(kSuspendNs)
            : "memory");
        if (there) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > limit_ns) {
            *abort = 1;
            return false;
        }
    }
}

// A count of uses whose parity a barrier's waits follow.
struct Phase {
    uint32_t n = 0;
    __device__ __forceinline__ uint32_t take() { return n++ & 1; }          // parity of the phase to wait for
    __device__ __forceinline__ uint32_t take_free() { return (n++ & 1) ^ 1; }   // of the phase before it (free at the start)
};

// Largest of three; NaN when one of them is.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^x for two x up to 8 (0 for x <= -127 and for NaN, less than 2^-126 between
// -127 and -126.5): 2^n by the exponent field, n = rint(x), times a polynomial
// for the rest in [-0.5, 0.5].  Degree 4, 1 at 0, the least largest
// relative error with a mean of 0 (a linear programme over its coefficients):
// 3.1e-6, 1/1270 of a bf16 rounding, and 6e-10 on average, so sums of many keep
// fp32's accuracy.  That it is exactly 1 at 0 makes the result at -127, where
// the exponent field gets to 0, exactly 0: a masked key's (-inf).
// It runs on the FMA pipes beside the special-function unit, which at 16
// results a clock would otherwise bound the softmax (128 x 128 x 2 per 2048
// clocks of products).
__device__ __forceinline__ float2 exp2_fma(float2 x) {
    const float magic = 12582912.f;          // 1.5 * 2^23: adding it rounds to an integer, left in the low bits
    x.x = fmaxf(x.x, -127.f);
    x.y = fmaxf(x.y, -127.f);
    const float2 t = fadd2(x, make_float2(magic, magic));
    const float2 r = fadd2(t, make_float2(-magic, -magic));
    const float2 f = ffma2(r, make_float2(-1.f, -1.f), x);
    float2 y = ffma2(f, make_float2(0.00962985866f, 0.00962985866f), make_float2(0.0559173897f, 0.0559173897f));
    y = ffma2(y, f, make_float2(0.240228951f, 0.240228951f));
    y = ffma2(y, f, make_float2(0.693121016f, 0.693121016f));
    y = ffma2(y, f, make_float2(1.f, 1.f));
    return make_float2(__int_as_float(__float_as_int(y.x) + (__float_as_int(t.x) << 23)),
                       __int_as_float(__float_as_int(y.y) + (__float_as_int(t.y) << 23)));
}

// Of every 8 pairs of probabilities, how many come from exp2_fma (8192-token
// prompt, 64/4 heads: none 1008 us, two 975, four 1020).
constexpr int kFmaPairs = 2;

// The scale bytes of keys key0 + 4 * lane .. + 3 of a tile to `to` (one warp);
// 0 for a row that is not there, whose leftovers in the stage become next to
// nothing then.  page: lane i has the page of the tile's i-th box.  Their
// arrival counts on the tile's barrier: nobody waits for them here.  (Looked
// up by the converters a tile ahead, they cost an eighth of the whole: 512 us
// for 4 chunks of 1000 over 12000 cached, here 441.)
__device__ __forceinline__ void load_scales(const RaggedParams &p, const Work &wk, const int32_t *table, int page,
                                            int rshift, int key0, bool is_v, uint8_t *to, uint32_t bar) {
    const int lane = threadIdx.x & 31;
    const int key = key0 + 4 * lane, mask = (1 << p.c.page_shift) - 1;
    const uint8_t *const scales = is_v ? p.c.v_scale : p.c.k_scale;
    if (p.c.page_shift >= 2) {
        const int pg = __shfl_sync(0xffffffffu, page, (4 * lane) >> rshift);
        int n = min(max(wk.kvl - key, 0), 4);
        if (pg < 0 || pg >= p.c.num_pages) n = 0;
        const size_t at = n > 0 ? (((size_t)pg * p.Hkv + wk.g) << p.c.page_shift) + (key & mask) : 0;
        asm volatile(
            "cp.async.ca.shared.global [%0], [%1], 4, %2;\n\t"
            "cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%3];" ::"r"(smem_u32(to)),
            "l"(scales + at), "r"(n), "r"(bar)
            : "memory");
        return;
    }
    uint32_t bytes = 0;                        // pages of one and two rows
    for (int r = 0; r < 4; ++r) {
        if (key + r >= wk.kvl) break;
        const int pg = __ldg(table + ((key + r) >> p.c.page_shift));
        if (pg >= 0 && pg < p.c.num_pages)
            bytes |= (uint32_t)__ldg(scales + (((size_t)pg * p.Hkv + wk.g) << p.c.page_shift) + ((key + r) & mask)) << (8 * r);
    }
    *reinterpret_cast<uint32_t *>(to) = bytes;
    mbar_arrive(bar);
}

template <bool F8>
__global__ void __launch_bounds__(Ring<F8>::threads, 1)
ragged_attn_tc(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
               const __grid_constant__ CUtensorMap tv, const RaggedParams p) {
    using R = Ring<F8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = align1024(smem_raw);
    uint8_t *sq = smem;
    uint8_t *skv = smem + 2 * TILE;
    uint8_t *sst = skv + R::slots * TILE;
    uint8_t *so = smem + 6 * TILE;
    RaggedBars *bars = reinterpret_cast<RaggedBars *>(smem + 7 * TILE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int readers = F8 ? 15 : 11;      // warps that read each work item (all but the one that finds it)
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        mbar_init(smem_u32(&bars->q_empty), 2 + 128);
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), F8 ? 128 : 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&bars->st_full[s]), 1 + 32);     // the tile; each lane's scales
            mbar_init(smem_u32(&bars->st_empty[s]), 128);
        }
        for (int w = 0; w < 2; ++w) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_u32(&bars->s_full[w][b]), 1);
                mbar_init(smem_u32(&bars->p_full[w][b]), 128);
            }
            mbar_init(smem_u32(&bars->pv_done[w]), 1);
            mbar_init(smem_u32(&bars->o_full[w]), 1);
            mbar_init(smem_u32(&bars->o_empty[w]), 128);
            mbar_init(smem_u32(&bars->work_full[w]), 1);
            mbar_init(smem_u32(&bars->work_empty[w]), readers);
        }
        mbar_init(smem_u32(&bars->q_read), 1);
        mbar_init(smem_u32(&bars->side_full), 128);
        mbar_init(smem_u32(&bars->drain[0]), 1);
        mbar_init(smem_u32(&bars->drain[1]), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch(&tq);
        tma_prefetch(&tk);
        tma_prefetch(&tv);
    }
    Batch batch;
    if (warp == 11) batch = read_batch(p);       // under the set-up
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int *abort = &bars->abort;

    // The next item, for a whole warp; false: none left, or a wait gave up
    // (then *abort is set).
    int work_i = 0;
    Work wk;
    auto next_work = [&]() -> bool {
        const int slot = work_i & 1;
        const bool ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->work_full[slot]), (work_i >> 1) & 1, p.wait_ns,
                                                          abort));
        if (!ok) return false;
        wk = bars->work[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->work_empty[slot]));
        ++work_i;
        return wk.go != 0;
    };
    // Whether no row of row tile w sees a key of the second half of key tile j,
    // as in the last tile of many: that half's products and softmax are left
    // out, its hand-overs are not (148 prompts of 64 tokens, 32/8 heads: 63 to
    // 57 us; 37 of 1024: 412 to 400).
    auto half_unseen = [&](int w, int j) {
        const int last = wk.off + min(wk.t0 + (wk.solo ? 1 : w + 1) * p.tpt, wk.ql) - 1;
        return (wk.j0 + j) * BN + BN / 2 > last;
    };
    // value rows of the item's last tile that exist
    auto tail_rows = [&]() { return (wk.j0 + wk.n) * BN > wk.kvl ? wk.kvl - (wk.j0 + wk.n - 1) * BN : BN; };

    if (warp >= 8) {
        regs_release<R::ctl>();
        if (warp == 11) {
            // ------------------------------------------------ items
            for (int i = 0;; ++i) {
                const Work w = find_work(p, batch, i);
                const bool ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->work_empty[i & 1]), ((i >> 1) & 1) ^ 1,
                                                                  p.wait_ns, abort));
                if (!ok) break;
                if (lane == 0) {
                    bars->work[i & 1] = w;
                    mbar_arrive(smem_u32(&bars->work_full[i & 1]));
                }
                __syncwarp();
                if (!w.go) break;
            }
        } else if (warp == 8) {
            // ------------------------------------------------ TMA producer
            constexpr int slots = F8 ? R::stages : R::slots;
            uint64_t *full = F8 ? bars->st_full : bars->kv_full;
            uint64_t *empty = F8 ? bars->st_empty : bars->kv_empty;
            constexpr int parts = F8 ? 1 : 2;        // boxes per group of rows (64-column halves of bf16 rows)
            constexpr int row_bytes = 128;           // per box row
            const int rshift = 31 - __clz(p.box_rows);
            const uint32_t qb = smem_u32(&bars->q_full);
            RingPos pos;
            Phase q_free;
            uint32_t issued = 0, k_tiles = 0, q_loads = 0;
            bool ok = true;
            while (ok && next_work()) {
                const int n = wk.n;
                if (n == 0) continue;
                ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->q_empty), q_free.take_free(), p.wait_ns, abort));
                if (!ok) break;
                const bool solo = wk.solo != 0;
                if (lane == 0) {
                    const int tiles = solo ? 1 : 2;
                    mbar_expect_tx(qb, tiles * 2 * p.tpt * p.G * 128);
                    for (int s = 0; s < tiles; ++s)
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_3d(smem_u32(sq + s * TILE + hf * HALF), &tq, qb, hf * 64, wk.g * p.G,
                                        wk.q0 + wk.t0 + s * p.tpt);
                }
                ++q_loads;
                const int32_t *table = p.paged ? p.c.block_table + (size_t)wk.b * p.c.max_pages : nullptr;
                for (int it = 0; it < 2 * n; ++it) {
                    int j;
                    bool is_v;
                    kv_item(it, n, solo, j, is_v);
                    const int key0 = (wk.j0 + j) * BN;
                    const int boxes = p.paged ? (min(BN, wk.kvl - key0) + p.box_rows - 1) >> rshift : 1;
                    int page = 0;
                    if (p.paged && lane < boxes) page = __ldg(table + ((key0 + (lane << rshift)) >> p.c.page_shift));
                    if (!is_v && p.paged) {
                        const int bad = (k_tiles + j) % kBadBufs;
                        // Which boxes lie on pages outside the pool, for the softmax to leave
                        // their keys out.  By the lane that arrives on the barrier below, before
                        // it does: the copies' bytes order nothing before the readers.
                        uint32_t any = 0;
#pragma unroll 1
                        for (int w = 0; w < boxes; w += 32) {
                            const int i = w + lane;
                            int pg = page;
                            if (w > 0 && i < boxes) pg = __ldg(table + ((key0 + (i << rshift)) >> p.c.page_shift));
                            const uint32_t out = __ballot_sync(0xffffffffu, i < boxes && (pg < 0 || pg >= p.c.num_pages));
                            if (lane == 0) bars->bad[bad][w >> 5] = out;
                            any |= out;
                        }
                        if (lane == 0) bars->bad_any[bad] = any;
                    }
                    ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&empty[pos.slot]), pos.phase ^ 1, p.wait_ns, abort));
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&full[pos.slot]);
                    const uint32_t dst = smem_u32(F8 ? sst + pos.slot * kStage : skv + pos.slot * TILE);
                    const CUtensorMap *m = is_v ? &tv : &tk;
                    if (lane == 0) mbar_expect_tx(fb, (uint32_t)(boxes * p.box_rows * parts * row_bytes));
                    __syncwarp();
                    for (int i = lane; i < boxes; i += 32) {
                        int c2 = wk.q0 + key0, c3 = 0;
                        if (p.paged) {
                            const int key = key0 + (i << rshift);
                            if (i >= 32) page = __ldg(table + (key >> p.c.page_shift));
                            c2 = key & ((1 << p.c.page_shift) - 1);
                            c3 = page;
                            if (page < 0 || page >= p.c.num_pages) {
                                // outside the pool: a box past the map's end reads zeros
                                report(p.status, HS_ERR_INVALID_INDEX);
                                c3 = p.c.num_pages;
                            }
                        }
                        for (int hf = 0; hf < parts; ++hf)
                            tma_load_4d(dst + hf * HALF + (i << rshift) * row_bytes, m, fb, hf * 64, wk.g, c2, c3);
                    }
                    if constexpr (F8) load_scales(p, wk, table, page, rshift, key0, is_v, &bars->scale[pos.slot][4 * lane], fb);
                    ++issued;
                    pos.next(slots);
                }
                k_tiles += n;
            }
            __syncwarp();
            // Let our own copies land before the CTA goes away.  Always: a wait of
            // another warp may be given up after this one has found nothing to do.
            if (lane == 0) {
                if (q_loads > 0) mbar_drain(qb, (q_loads - 1) & 1);
                for (uint32_t it = issued > (uint32_t)slots ? issued - slots : 0; it < issued; ++it)
                    mbar_drain(smem_u32(&full[it % slots]), (it / slots) & 1);
            }
        } else if (warp == 9 || warp == 10) {
            // ------------------------------------------------ MMA issuers, one for each row tile
            // The whole warp goes through the loop and one elected lane issues, so
            // that descriptors stay in uniform registers.  Two issuers, because one
            // spent as long on its waits and commits between the two row tiles'
            // chains as the products took.
            const int w = warp - 9;
            const uint32_t leader = elect_one();
            const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;
            const uint32_t kv_lo = desc_lo(smem_u32(skv));
            Phase q_phase, o_free;
            uint32_t p_uses = 0;                       // P handed over so far: buffer = the last bit
            RingPos pos;
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, bar_wait(smem_u32(bar), parity, p.wait_ns, abort));
                if (ok) tc_fence_after();
                return ok;
            };
            while (ok && next_work()) {
                const int n = __shfl_sync(0xffffffffu, wk.n, 0);
                if (n == 0) continue;
                const bool solo = __shfl_sync(0xffffffffu, wk.solo, 0) != 0;
                const int nw = __shfl_sync(0xffffffffu, w == 0 ? wk.n0 : wk.n1, 0);
                const int tail = __shfl_sync(0xffffffffu, tail_rows(), 0);
                // this row tile's last key tile and whether its second half is unseen
                const int j_last = solo ? w + 2 * (nw - 1) : nw - 1;
                const int stop = __shfl_sync(0xffffffffu, nw > 0 && half_unseen(w, j_last) ? 1 : 0, 0);
                const uint32_t q_lo = desc_lo(smem_u32(solo ? sq : sq + w * TILE));
                uint32_t begun = 0;                    // O has been written by this item
                int left = 2 * nw, qk_left = 2 * nw;   // halves to go; at `stop` the unseen one
                // S = Q K^T for half h of the key tile in ring slot `slot` (buffer h)
                auto qk = [&](int slot, int h) {
                    const uint32_t b = kv_lo + slot * (TILE >> 4) + h * ((64 * 128) >> 4);
                    constexpr uint32_t I = idesc_bf16(128, 64, false, false);
                    if (qk_left-- != stop)
#pragma unroll
                        for (int kk = 0; kk < HD / 16; ++kk) {
                            const uint32_t o = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                            mma_ss_one(tS + h * 64, q_lo + o, b + o, kDescHi, kDescHi, I, kk > 0 ? 1u : 0u, leader);
                        }
                    commit_one(smem_u32(&bars->s_full[w][h]), leader);
                };
                // O += P V for half h of the value tile in ring slot `slot`
                auto pv = [&](int slot, int h) {
                    constexpr uint32_t I = idesc_bf16(128, 128, false, true);
                    if (!wait(&bars->p_full[w][h], (p_uses >> 1) & 1)) return false;
                    ++p_uses;
                    const uint32_t b = kv_lo + slot * (TILE >> 4) + h * ((64 * 128) >> 4) + (kDescLboV << 16);
                    if (left != stop)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts_one(tO, tS + h * 64 + kk * 8, b + ((kk * 2048) >> 4), kDescHi, I, kk > 0 ? 1u : begun,
                                       leader);
                    begun = 1;
                    commit_one(smem_u32(&bars->pv_done[w]), leader);
                    if (--left == 0) commit_one(smem_u32(&bars->o_full[w]), leader);
                    return true;
                };
                // Zero the value rows behind the sequence's end, in the last tile: whatever
                // lies there, NaN included, would reach the output as 0 * NaN.  (Both
                // issuers may do it to the same tile.)  Whole 128-byte rows, so the
                // swizzle within a row does not matter.
                auto zero_tail = [&](int slot, int j) {
                    if constexpr (!F8) {
                        if (j != n - 1 || tail >= BN) return;
                        for (int i = lane; i < (BN - tail) * 16; i += 32) {
                            const int row = tail + (i >> 4), part = i & 15;
                            *reinterpret_cast<uint4 *>(skv + slot * TILE + (part >> 3) * HALF + row * 128 +
                                                       (part & 7) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                };
                auto kv_wait = [&]() { return wait(&bars->kv_full[pos.slot], pos.phase); };
                auto take_slot = [&]() {
                    const int slot = pos.slot;
                    pos.next(R::slots);
                    return slot;
                };
                // A slot is free once both issuers have let go of it: by a commit after the
                // products that read it, or at once where it is the other's (solo).  That
                // arrival keeps a slot from being filled again before this issuer has seen
                // it full: two fills later the phase's parity would tell it nothing.
                auto release = [&](int slot) { commit_one(smem_u32(&bars->kv_empty[slot]), leader); };
                auto pass = [&](int slot) {
                    if (leader) mbar_arrive(smem_u32(&bars->kv_empty[slot]));
                    __syncwarp();
                };
                if (!wait(&bars->q_full, q_phase.take())) break;
                // First both steps of the row tile's first key tile; then, step by step, P V
                // and the same step of its next key tile's Q K^T, which may overwrite S as
                // soon as that P has been read.
                if (!solo) {
                    if (!kv_wait()) break;
                    const int slot = take_slot();
                    if (nw > 0) {
                        qk(slot, 0);
                        qk(slot, 1);
                    }
                    release(slot);
                } else {
                    // (the first two K tiles are row tile 0's and 1's; each issuer waits for
                    // the other's tiles too, or it would lose count of the slots' phases)
                    for (int j = 0; j < min(n, 2); ++j) {
                        if (!kv_wait()) break;
                        const int slot = take_slot();
                        if (j != w) {
                            pass(slot);
                            continue;
                        }
                        qk(slot, 0);
                        qk(slot, 1);
                        release(slot);
                    }
                }
                // after the last product with Q; warpgroup 1 waits for issuer 0's before it
                // stores its half of a joined item there
                auto release_q = [&]() {
                    commit_one(smem_u32(&bars->q_empty), leader);
                    if (solo && w == 0 && n > 1) commit_one(smem_u32(&bars->q_read), leader);
                };
                if (nw <= 1) release_q();
                // O may be overwritten once the item that had it before has been read out
                if (nw > 0 && !wait(&bars->o_empty[w], o_free.take_free())) break;
                int done = 0;                          // key tiles of this row tile
                for (int j = 0; ok && j < n; ++j) {
                    const bool mine = solo ? (j & 1) == w : j < nw;
                    const bool k_there = j + (solo ? 2 : 1) < n;       // a K tile follows V_j in the ring
                    if (!kv_wait()) break;
                    const int v = take_slot();
                    if (solo && !mine) {
                        pass(v);
                        if (k_there) {
                            if (!kv_wait()) break;
                            pass(take_slot());
                        }
                        continue;
                    }
                    int k = -1;
                    if (mine) {
                        zero_tail(v, j);
                        ++done;
                        for (int h = 0; h < 2; ++h) {
                            if (!pv(v, h)) break;
                            if (done < nw) {
                                if (k < 0) {
                                    if (!kv_wait()) break;
                                    k = take_slot();
                                }
                                qk(k, h);
                            }
                        }
                        if (!ok) break;
                        if (done + 1 == nw) release_q();
                    }
                    release(v);
                    if (k_there) {
                        if (k < 0) {                   // not needed here, but there to be released
                            if (!kv_wait()) break;
                            k = take_slot();
                        }
                        release(k);
                    }
                }
            }
            // all MMAs this warp issued have completed before TMEM is freed
            commit_one(smem_u32(&bars->drain[w]), leader);
            if (leader) mbar_drain(smem_u32(&bars->drain[w]), 0);
            __syncwarp();
        } else if (F8) {
            // ------------------------------------------------ 8-bit rows to bf16 tiles
            const int t = threadIdx.x - 384;
            const int c16 = t & 7, r0 = t >> 3;      // 16 codes of rows r0, r0 + 16, ...
            // read and stored as two halves of 8 codes, in an order that lets the
            // lanes of each access touch all banks
            const int first = (c16 >= 4) ^ (r0 & 1);
            const uint32_t row_at = (c16 >> 2) * HALF + r0 * 128;
            const uint32_t at0 = row_at + ((((2 * c16) & 7) + first) ^ (r0 & 7)) * 16;
            const uint32_t at1 = row_at + ((((2 * c16) & 7) + 1 - first) ^ (r0 & 7)) * 16;
            RingPos st, kv;
            bool ok = true;
            while (ok && next_work()) {
                const int n = wk.n;
                for (int it = 0; it < 2 * n; ++it) {
                    ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->st_full[st.slot]), st.phase, p.wait_ns, abort));
                    ok = ok && __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->kv_empty[kv.slot]), kv.phase ^ 1,
                                                                 p.wait_ns, abort));
                    if (!ok) break;
                    const uint8_t *src = sst + st.slot * kStage + r0 * 128 + c16 * 16;
                    uint8_t *dst = skv + kv.slot * TILE;
                    // rows that are not there keep finite leftovers: their probabilities are exactly 0
                    uint32_t scales[8], top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        scales[i] = bars->scale[st.slot][r0 + 16 * i];
                        top = max(top, scales[i]);
                    }
                    // Four rows' codes are read before the first of them is stored (571 to 508 us
                    // for 4 chunks of 1000 over 12000 cached; two 522, eight 540), and no
                    // branch lies between rows (446 to 435): the compiler moves neither a read
                    // over a store to the same memory nor anything over a branch.
                    auto widen = [&](auto large) {
                        uint2 u[4], v[4];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if ((i & 3) == 0)
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    u[k] = *reinterpret_cast<const uint2 *>(src + (i + k) * 2048 + first * 8);
                                    v[k] = *reinterpret_cast<const uint2 *>(src + (i + k) * 2048 + 8 - first * 8);
                                }
                            const uint32_t w[4] = {u[i & 3].x, u[i & 3].y, v[i & 3].x, v[i & 3].y};
                            const uint32_t sb = scales[i];
                            uint32_t o[8];
                            // 2^(120 + byte - 127) as a bf16 pair, up to 2^127
                            const uint32_t f = (large ? min(sb, 134u) : sb) * 0x00800080u + 0x3c003c00u;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                o[2 * q] = bf16x2_mul(e4m3_to_bf16_tiny<0x9180>(w[q]), f);
                                o[2 * q + 1] = bf16x2_mul(e4m3_to_bf16_tiny<0xb3a2>(w[q]), f);
                            }
                            if (large) {           // the rest of a scale above 2^7, or a row of NaN
                                const uint32_t g =
                                    sb == 255u ? 0x7fff7fffu : (max(sb, 134u) - 134u) * 0x00800080u + 0x3f803f80u;
#pragma unroll
                                for (int q = 0; q < 8; ++q) o[q] = bf16x2_mul(o[q], g);
                            }
                            *reinterpret_cast<uint4 *>(dst + at0 + i * 2048) = make_uint4(o[0], o[1], o[2], o[3]);
                            *reinterpret_cast<uint4 *>(dst + at1 + i * 2048) = make_uint4(o[4], o[5], o[6], o[7]);
                        }
                    };
                    if (__any_sync(0xffffffffu, top > 134u)) widen(std::true_type{});
                    else widen(std::false_type{});
                    fence_proxy_async_smem();
                    mbar_arrive(smem_u32(&bars->kv_full[kv.slot]));
                    mbar_arrive(smem_u32(&bars->st_empty[st.slot]));
                    st.next(R::stages);
                    kv.next(R::slots);
                }
            }
        }
    } else {
        regs_acquire<R::soft>();
        // ------------------------------------------------ softmax warpgroups
        const int w = warp >> 2;
        const int tw = threadIdx.x - 128 * w;
        const uint32_t lane_off = (uint32_t)(tw & ~31) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)(w * 128);
        const uint32_t tO = tmem + lane_off + 256u + (uint32_t)(w * 128);
        const float c2 = p.scale_log2;
        const float nan = __int_as_float(0x7fc00000);
        const int row_tok = (int)((uint32_t)tw * p.g_inv >> 16), row_head = tw - row_tok * p.G;
        Phase side_phase, o_phase;
        uint32_t steps_done = 0;       // steps of 64 keys so far: the buffer and the parities follow
        uint32_t k_tiles = 0;
        bool ok = true;
        while (ok && next_work()) {
            const bool solo = wk.solo != 0;
            const int n = wk.n;
            const int first = wk.t0 + (solo ? 0 : w * p.tpt);      // this row tile's first token
            const int tok = first + row_tok;
            const bool valid = tw < p.tpt * p.G && tok < wk.ql;
            const int pos = wk.off + min(tok, wk.ql - 1);
            const int pos_first = wk.off + first;
            const int nw = w == 0 ? wk.n0 : wk.n1;
            const bool join = solo && n > 1;
            float m = -INFINITY, l = 0.f;
            const int unseen = nw > 0 && half_unseen(w, solo ? w + 2 * (nw - 1) : nw - 1) ? 1 : 0;
            const int u_end = 2 * nw - unseen;
            for (int u = 0; u < u_end; ++u, ++steps_done) {
                const int buf = steps_done & 1;             // = u & 1: half of the key tile
                const int j = solo ? (u & ~1) + w : u >> 1;
                const int key0 = (wk.j0 + j) * BN + buf * 64;
                ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->s_full[w][buf]), (steps_done >> 1) & 1, p.wait_ns,
                                                       abort));
                if (!ok) break;
                tc_fence_after();
                // Q's place is only needed here again when the halves are joined there
                // (then warpgroup 0 says when it is done with it)
                if (u == 0 && !join && w == (solo ? 0 : 1)) mbar_arrive(smem_u32(&bars->q_empty));
                float s[64];
                {
                    uint32_t r[2][32];
                    tmem_ld32(tS + buf * 64, r[0]);
                    tmem_ld32(tS + buf * 64 + 32, r[1]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(r[c >> 5][c & 31]);
                }
                const int bad = (k_tiles + j) % kBadBufs;
                const bool lost = p.paged && bars->bad_any[bad] != 0;
                const bool masked = lost || key0 + 63 > pos_first;
                if (masked) {
                    // keys up to the row's own position, and not on a lost page
                    const int seen = pos - key0;
#pragma unroll
                    for (int c = 0; c < 64; ++c) s[c] = c <= seen ? s[c] : -INFINITY;
                    if (lost) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int c = 64 * buf + 32 * q + lane, box = c >> (31 - __clz(p.box_rows));
                            const uint32_t bits = __ballot_sync(0xffffffffu, (bars->bad[bad][box >> 5] >> (box & 31)) & 1u);
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if ((bits >> c) & 1u) s[32 * q + c] = -INFINITY;
                        }
                    }
                }
                float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < 64; c += 2) m4[(c >> 1) & 3] = fmax3_nan(m4[(c >> 1) & 3], s[c], s[c + 1]);
                const float mx2 = fmax3_nan(fmax3_nan(m4[0], m4[1], m4[2]), m4[3], m4[3]) * c2;
                // the running maximum only moves when it grows by more than 8 (log2
                // units); the final division uses the same reference.  Rows that are
                // nobody's have no say: NaN in them (another sequence's, or what shared
                // memory held) would move it in every step (16 chunks of 33 rows over 8000
                // cached, NaN behind them: 177 us, 149 without).
                if (__any_sync(0xffffffffu, valid && !(mx2 <= m + 8.0f))) {
                    // (a score that is NaN or +inf makes the row NaN, here and for good)
                    const float m_new = mx2 < INFINITY ? fmax3_nan(m, mx2, mx2) : nan;
                    if (u > 0) {
                        // The product of the step before has to be in O first.  (Its phase is
                        // the barrier's last or current one: the step before that is done,
                        // since this step's S was computed after it, and this one's P is not
                        // handed over yet.)
                        ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->pv_done[w]), (steps_done - 1) & 1, p.wait_ns,
                                                               abort));
                        if (!ok) break;
                        tc_fence_after();
                        const float corr = m_new == -INFINITY ? 1.f : ex2(m - m_new);
                        l *= corr;
#pragma unroll 1
                        for (int c = 0; c < 8; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
                            tmem_st16(tO + 16 * c, o);
                        }
                        tmem_wait_st();
                    }
                    m = m_new;
                }
                // masked keys (-inf) give exactly 0
                const float mref = m == -INFINITY ? 0.f : m;
                const float2 c2v = make_float2(c2, c2), mv = make_float2(-mref, -mref);
                float2 ps01 = make_float2(0.f, 0.f), ps23 = make_float2(0.f, 0.f);
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int c = ch * 32 + 2 * e;
                        const float2 t = ffma2(make_float2(s[c], s[c + 1]), c2v, mv);
                        const float2 ab = (e & 7) < kFmaPairs ? exp2_fma(t) : make_float2(ex2(t.x), ex2(t.y));
                        if (e & 1) ps23 = fadd2(ps23, ab); else ps01 = fadd2(ps01, ab);
                        // P is rounded to bf16, the type of V: one MMA takes one type
                        pk[e] = pack_bf16(ab.x, ab.y);
                    }
                    tmem_st16(tS + buf * 64 + 16 * ch, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(smem_u32(&bars->p_full[w][buf]));
                l += (ps01.x + ps01.y) + (ps23.x + ps23.y);
            }
            if (unseen && ok) {
                ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->s_full[w][1]), (steps_done >> 1) & 1, p.wait_ns,
                                                       abort));
                if (ok) mbar_arrive(smem_u32(&bars->p_full[w][1]));
                ++steps_done;
            }
            k_tiles += n;
            if (nw > 0)
                ok = __all_sync(0xffffffffu, ok && bar_wait(smem_u32(&bars->o_full[w]), o_phase.take(), p.wait_ns, abort));
            bool fin = ok;
            tc_fence_after();
            // O of this thread's row: columns [32 c, 32 c + 32), zeros when there were no tiles
            auto load_o = [&](int c, float (&o)[32]) {
                uint32_t r[32];
                if (nw > 0) {
                    tmem_ld32(tO + 32 * c, r);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = nw > 0 ? __uint_as_float(r[e]) : 0.f;
            };
            float *const side = reinterpret_cast<float *>(sq) + tw * 128;   // 64 KB: the Q tiles, no longer read
            float a0 = 1.f, a1 = 0.f;
            if (join) {
                // Warpgroup 1 hands its half of the keys over through shared memory, once
                // issuer 0's products have read Q there: its last key tile may be the
                // item's last, and then nothing else says that they have.
                if (w == 1) {
                    ok = __all_sync(0xffffffffu, ok && bar_wait(smem_u32(&bars->q_read), side_phase.take(), p.wait_ns, abort));
                    fin = ok;
                    bars->side[tw] = make_float2(fin ? m : nan, l);
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        float o[32];
                        load_o(c, o);
                        if (valid && ok) {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                *reinterpret_cast<float4 *>(side + (((8 * c + e) ^ (tw & 31)) << 2)) =
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        }
                    }
                    fence_proxy_async_smem();      // the next Q tiles come here through the async proxy
                    mbar_arrive(smem_u32(&bars->side_full));
                } else {
                    ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&bars->side_full), side_phase.take(), p.wait_ns, abort));
                    if (!ok) fin = false;
                    const float2 other = bars->side[tw];
                    const float top = fmaxf(m, other.x);
                    if (other.x != other.x) fin = false;
                    a0 = m == -INFINITY ? 0.f : ex2(m - top);
                    a1 = other.x == -INFINITY ? 0.f : ex2(other.x - top);
                    l = l * a0 + other.y * a1;
                    m = top;
                }
            }
            const bool partial = wk.partial != 0;
            const size_t row = (size_t)wk.q0 + tok;
            const int h = wk.g * p.G + row_head;
            // the row's result is this item's to write: not warpgroup 1's of a shared
            // tile, and not an empty piece's of a row that one piece holds
            const bool mine = !(solo && w == 1);
            if (valid && mine && (partial || wk.piece == 0)) {
                const size_t pr = ((size_t)wk.piece * p.T + row) * p.Hq + h;
                if (partial) p.part_ml[pr] = make_float2(fin ? m : nan, l);
                else {
                    if (p.splits > 1) p.part_ml[pr] = make_float2(0.f, -1.f);
                    // a bounded wait gave up: NaN in the row's lse, as in the full layer
                    p.lse[(size_t)h * p.T + row] = !fin || l != l ? nan : (l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY);
                }
            }
            if (mine && (partial ? n > 0 : wk.piece == 0)) {
                const float inv_l = partial ? 1.f : (l > 0.f ? 1.0f / l : 0.f);   // a row that sees nothing gives zeros
                a0 *= inv_l;
                a1 *= inv_l;
                // Through shared memory, 32 rows x 128 bytes of a warp at a time, so that
                // a store writes whole 128-byte lines (a thread's own row would be 32 of
                // them a store).  Chunk c of row r lies at c ^ (r & 7).
                uint8_t *stage = so + (warp & 7) * 4096;
                uint8_t *mine_at = stage + lane * 128;
                const int rows32 = tw & ~31;
                // Four rows a store, eight lanes each.
                const int r_mine = lane >> 3, ch = lane & 7;
                const int el = partial ? 4 : 2;                        // bytes of a result
                uint8_t *const base = (partial ? (uint8_t *)(p.part_o + (size_t)wk.piece * p.T * p.Hq * HD) : (uint8_t *)p.out) +
                                      (((size_t)wk.q0 + first) * p.Hq + wk.g * p.G) * (HD * el) + 16 * ch;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {                          // 32 columns
                    float o[32];
                    load_o(c, o);
                    if (join) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 y = *reinterpret_cast<const float4 *>(side + (((8 * c + e) ^ (tw & 31)) << 2));
                            o[4 * e] = o[4 * e] * a0 + y.x * a1;
                            o[4 * e + 1] = o[4 * e + 1] * a0 + y.y * a1;
                            o[4 * e + 2] = o[4 * e + 2] * a0 + y.z * a1;
                            o[4 * e + 3] = o[4 * e + 3] * a0 + y.w * a1;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= a0;
                    }
                    if (partial) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(mine_at + ((e ^ (lane & 7)) << 4)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4 *>(mine_at + (((4 * (c & 1) + e) ^ (lane & 7)) << 4)) =
                                make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]), pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                           pack_bf16(o[8 * e + 4], o[8 * e + 5]), pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    }
                    if (!partial && (c & 1) == 0) continue;            // half of the stage's 128 bytes
                    __syncwarp();
                    uint8_t *const to = base + (partial ? c : c >> 1) * 128;
                    uint4 x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + r_mine;
                        x[i] = *reinterpret_cast<const uint4 *>(stage + r * 128 + ((ch ^ (r & 7)) << 4));
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int tr = rows32 + 4 * i + r_mine;
                        const int t_tok = (int)((uint32_t)tr * p.g_inv >> 16);
                        if (tr < p.tpt * p.G && first + t_tok < wk.ql)
                            *reinterpret_cast<uint4 *>(to + (size_t)(t_tok * p.Hq + (tr - t_tok * p.G)) * (HD * el)) = x[i];
                    }
                    __syncwarp();                                      // read before it is written again
                }
            }
            if (w == 0 && join) {
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(&bars->q_empty));
            }
            if (nw > 0) {
                tc_fence_before();
                mbar_arrive(smem_u32(&bars->o_empty[w]));
            }
        }
        // a wait gave up: the rows of the items that this CTA did not get to
        // are marked like those of the one it was at
        // (one answer for the warp: its lanes look for the items together)
        if (__any_sync(0xffffffffu, *abort != 0) && (warp & 3) == 0) {
            const Batch bt = read_batch(p);
            for (int i = work_i;; ++i) {
                const Work x = find_work(p, bt, i);
                if (!x.go) break;
                if (x.solo && w == 1) continue;
                for (int r = lane; r < p.tpt * p.G; r += 32) {
                    const int tok = x.t0 + (x.solo ? 0 : w * p.tpt) + r / p.G, h = x.g * p.G + r % p.G;
                    if (tok >= x.ql) continue;
                    const size_t row = (size_t)x.q0 + tok;
                    if (x.partial) p.part_ml[((size_t)x.piece * p.T + row) * p.Hq + h] = make_float2(nan, 1.f);
                    else if (x.piece == 0) {
                        if (p.splits > 1) p.part_ml[row * p.Hq + h] = make_float2(0.f, -1.f);
                        p.lse[(size_t)h * p.T + row] = nan;
                    }
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && bars->abort) report(p.status, HS_ERR_TIMEOUT);
}

// Joins the pieces of rows that were split over several CTAs: one warp per
// (row, head), in piece order, so the result does not depend on timing.
__global__ void __launch_bounds__(256) ragged_combine(const RaggedParams p) {
    const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)p.T * p.Hq;
    if (r >= rows) return;
    const int t = (int)(r / p.Hq), h = (int)(r - (long long)t * p.Hq);
    // everything is asked for at once: two pieces' maximum and sum a lane, O of
    // the first eight pieces (what an empty piece left there is not used)
    static_assert(kMaxSplits <= 64, "two pieces a lane");
    float2 ml[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        ml[i] = lane + 32 * i < p.splits ? p.part_ml[(lane + 32 * i) * rows + r] : make_float2(-INFINITY, 0.f);
    const float *const src = p.part_o + r * HD + lane * 4;
    float4 o[8];
    auto ask = [&](int s0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (s0 + j < p.splits) o[j] = __ldcg(reinterpret_cast<const float4 *>(src + (s0 + j) * rows * HD));
    };
    ask(0);
    if (t < clamp_row(__ldg(p.c.cu_rows), p.T) || t >= clamp_row(__ldg(p.c.cu_rows + p.c.B), p.T)) return;
    if (__shfl_sync(0xffffffffu, ml[0].y, 0) < 0.f) return;   // written by its only piece
    const float m = warp_max(fmaxf(ml[0].x, ml[1].x));
    // each piece's weight, 0 when it saw nothing (its O was not written then);
    // NaN of a piece that gave up carries through
    float a[2], l = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        a[i] = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - m);
        l += ml[i].x == -INFINITY ? 0.f : a[i] * ml[i].y;
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0;;) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = __shfl_sync(0xffffffffu, s0 < 32 ? a[0] : a[1], (s0 + j) & 31);
            if (s0 + j < p.splits && f != 0.f) {
                acc.x += f * o[j].x;
                acc.y += f * o[j].y;
                acc.z += f * o[j].z;
                acc.w += f * o[j].w;
            }
        }
        s0 += 8;
        if (s0 >= p.splits) break;
        ask(s0);
    }
    l = warp_sum(l);
    const float inv = l > 0.f ? 1.f / l : (l != l ? l : 0.f);
    uint2 w;
    w.x = pack_bf16(acc.x * inv, acc.y * inv);
    w.y = pack_bf16(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2 *>(p.out + r * HD + lane * 4) = w;
    if (lane == 0) p.lse[(long long)h * p.T + t] = l != l ? l : (l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY);
}

// ------------------------------------------------------------------ host

// 3-D map of packed rows [T][H][128] (row stride ld elements): (d, H, T)
bool map_rows(CUtensorMap *m, const void *base, int H, int T, long long ld, int box_h, int box_t) {
    auto enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)HD, (cuuint64_t)H, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)HD * 2, (cuuint64_t)ld * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_h, (cuuint32_t)box_t};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 4-D map of keys or values: (d, Hkv, row, page), boxes of box_rows rows of
// one head; bf16 rows in swizzled 64-column halves, 8-bit rows whole.
bool map_keys(CUtensorMap *m, const void *base, int Hkv, long long rows, long long ld, int pages, int box_rows,
              bool f8) {
    auto enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t es_b = f8 ? 1 : 2;
    cuuint64_t dims[4] = {(cuuint64_t)HD, (cuuint64_t)Hkv, (cuuint64_t)rows, (cuuint64_t)pages};
    cuuint64_t strides[3] = {HD * es_b, (cuuint64_t)ld * es_b, (cuuint64_t)ld * es_b * (cuuint64_t)rows};
    cuuint32_t box[4] = {f8 ? 128u : 64u, 1, (cuuint32_t)box_rows, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return enc(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               f8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A kernel's shared-memory limit, set once per device (threads that meet here
// set it twice, to the same value).
template <bool F8>
cudaError_t prepare() {
    static std::atomic<unsigned long long> done[2]{};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 128 && (done[dev >> 6].load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(ragged_attn_tc<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRaggedSmem);
    if (e == cudaSuccess && dev < 128) done[dev >> 6].fetch_or(bit, std::memory_order_release);
    return e;
}

constexpr int kSms = 148;
// Rows (new tokens x group) a sequence up to which the warp-MMA kernel runs.
// Measured with 32 / 8 heads, 16 caches of 8192, 64 of 2048 (us; 8, 16, 32, 64
// rows): bf16 82, 84, 110, 215 against 111 of the tcgen05 kernel, and 83, 87,
// 138, 210 against 127; 8-bit 53, 70, 130, 255 against 152, and 70, 99, 147,
// 232 against 174.
constexpr int kFewRows16 = 16, kFewRows8 = 32;
constexpr int kFewRowsCtas16 = 2, kFewRowsCtas8 = 3;   // CTAs of that kernel an SM holds (bf16, 8-bit caches)
constexpr int kFewRowsFixed = 16;          // what a piece costs besides its keys, in 16-key blocks
constexpr int kFewRowsMinChunk = 4;        // fewest 16-key blocks in a piece (one for each warp)
constexpr size_t kMaxPartRows = 180000;    // rows of partial results: 520 bytes each

// SMs of the current device (one CTA of the tcgen05 kernel runs on each).
int sm_count() {
    static std::atomic<int> cached[64]{};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kSms;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = kSms;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Work items of a batch (an upper bound from what the host knows).
long long work_bound(const RaggedCall &a) {
    const long long qt = 2 * (128 / (a.Hq / a.Hkv));
    const long long by_rows = a.T / qt + a.B;
    const long long by_len = (long long)a.B * ((std::min<long long>(a.max_q, a.T) + qt - 1) / qt);
    return std::max<long long>(1, std::min(by_rows, by_len));
}

cudaError_t combine_launch(const RaggedParams &p, cudaStream_t st) {
    if (p.splits == 1) return cudaSuccess;
    const long long rows = (long long)p.T * p.Hq;
    if ((rows + 7) / 8 > 0x7fffffffLL) return cudaErrorInvalidValue;
    ragged_combine<<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(p);
    count_launch();
    return cudaGetLastError();
}

// Workspace layout: status word, (max, sum) and O of every piece of every row.
void plan_bytes(size_t rows, RaggedPlan *pl) {
    pl->ml_off = kStatusBytes;
    pl->o_off = align_up(pl->ml_off + (pl->splits > 1 ? pl->splits * rows * sizeof(float2) : 0), 256);
    pl->bytes = align_up(pl->o_off + (pl->splits > 1 ? pl->splits * rows * 128 * sizeof(float) : 0), 256);
}

}  // namespace
}  // namespace tc

// How many pieces each item's keys are cut into (1: none).  A piece costs
// about three key tiles to start and end; pieces are added while they shorten
// the longest SM's share by more than that, up to what the workspace bound
// allows.
RaggedPlan ragged_plan(const RaggedCall &a) {
    using namespace tc;
    RaggedPlan pl;
    const size_t rows = (size_t)a.T * a.Hq;
    const int G = a.Hq / a.Hkv;
    const long long row_most = (long long)std::max(1, std::min(a.max_q, a.T)) * G;   // rows of a sequence, at most
    if (a.paged && row_most <= (a.cache.dtype == HS_E4M3 ? kFewRows8 : kFewRows16)) {
        // few rows a sequence: 8- or 16-row tiles on the warp MMAs, pieces of 16-key blocks
        pl.few_rows = true;
        pl.tile_rows = row_most <= 8 ? 8 : 16;
        pl.tiles = (int)((row_most + pl.tile_rows - 1) / pl.tile_rows);
        const long long items = (long long)a.B * pl.tiles * a.Hkv;
        const long long blocks = std::max<long long>(1, (a.max_len + 15) / 16);
        // a piece costs about kFewRowsFixed blocks to start and end, the join of pieces
        // as much; of the splits within 3 % of the cheapest the finest, because
        // the caches' real lengths differ and small pieces even them out
        const long long slots = (long long)kSms * (a.cache.dtype == HS_E4M3 ? kFewRowsCtas8 : kFewRowsCtas16);
        auto cost = [&](long long s) {
            const long long chunk = (blocks + s - 1) / s;
            return (items * s + slots - 1) / slots * (chunk + kFewRowsFixed) + (s > 1 ? kFewRowsFixed : 0);
        };
        long long most = std::min<long long>(std::max<long long>(blocks / kFewRowsMinChunk, 1), kMaxSplits);
        if (rows > 0) most = std::max<long long>(1, std::min<long long>(most, (long long)(kMaxPartRows / rows)));
        // the finest split of each number of waves (a cheaper one there is none)
        long long best = cost(1), s = 1;
        for (int pass = 0; pass < 2; ++pass)
            for (long long w = 1, t = 0; w <= 32 && t < most; ++w) {
                t = std::min(most, w * slots / items);
                if (t < 1) continue;
                const long long ct = cost(t);
                if (pass == 0) best = std::min(best, ct);
                else if (ct * 100 <= best * 103) s = t;
            }
        pl.chunk = (int)((blocks + s - 1) / s);
        pl.splits = (int)((blocks + pl.chunk - 1) / pl.chunk);
        if (pl.splits == 1) pl.chunk = 0x7fffffff / 16;
        plan_bytes(rows, &pl);
        return pl;
    }
    const long long works = work_bound(a) * a.Hkv;
    const long long tiles = std::max<long long>(1, (a.max_len + BN - 1) / BN);
    pl.works = (int)std::min<long long>(work_bound(a), 0x7fffffff);
    long long best = -1;
    for (long long s = 1; s <= std::min<long long>(tiles, kMaxSplits); ++s) {
        if (s > 1 && (works * s > 8 * kSms || rows * s > kMaxPartRows)) break;
        const long long chunk = (tiles + s - 1) / s;
        const long long waves = (works * s + kSms - 1) / kSms;
        const long long cost = waves * (chunk + 3) + (s > 1 ? 2 : 0);
        if (best < 0 || cost < best) {
            best = cost;
            pl.splits = (int)((tiles + chunk - 1) / chunk);
            pl.chunk = (int)chunk;
        }
    }
    if (pl.splits == 1) pl.chunk = 0x7fffffff / BN;      // lengths past max_len still run, in one piece
    plan_bytes(rows, &pl);
    return pl;
}

// No plan for these rows takes more, whatever the keys' lengths.
size_t ragged_most_bytes(const RaggedCall &a) {
    using namespace tc;
    const size_t rows = (size_t)a.T * a.Hq;
    RaggedPlan pl;
    if (rows > 0) pl.splits = (int)std::max<size_t>(1, std::min<size_t>(kMaxSplits, kMaxPartRows / rows));
    plan_bytes(rows, &pl);
    return pl.bytes;
}

cudaError_t ragged_attn_launch(const RaggedCall &a, const RaggedPlan &pl, void *ws, unsigned long long wait_ns,
                               cudaStream_t st) {
    using namespace tc;
    cudaError_t e = cudaSuccess;
    RaggedParams p{};
    p.c = a.cache;
    p.paged = a.paged;
    p.T = a.T; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.tpt = 128 / p.G;
    p.g_inv = (65536u + p.G - 1) / p.G;
    const bool f8 = a.paged && a.cache.dtype == HS_E4M3;
    const int page = a.paged ? 1 << a.cache.page_shift : 0;
    p.box_rows = a.paged ? std::min(page, BN) : BN;
    p.works = pl.works; p.splits = pl.splits; p.chunk = pl.chunk;
    p.scale_log2 = a.scale * kLog2e;
    p.out = (__nv_bfloat16 *)a.out; p.lse = a.lse;
    p.status = (unsigned int *)ws;
    p.wait_ns = wait_ns;
    if (pl.splits > 1) {
        p.part_ml = reinterpret_cast<float2 *>((char *)ws + pl.ml_off);
        p.part_o = reinterpret_cast<float *>((char *)ws + pl.o_off);
    }
    if (pl.few_rows) {
        e = ragged_rows_launch(a, pl, ws, st);
        return e == cudaSuccess ? combine_launch(p, st) : e;
    }
    CUtensorMap mq, mk, mv;
    if (!map_rows(&mq, a.q, a.Hq, a.T, a.ld_q, p.G, p.tpt)) return cudaErrorInvalidValue;
    if (a.paged) {
        const long long ld = (long long)a.Hkv * HD;
        if (!map_keys(&mk, a.cache.k_pages, a.Hkv, page, ld, a.cache.num_pages, p.box_rows, f8) ||
            !map_keys(&mv, a.cache.v_pages, a.Hkv, page, ld, a.cache.num_pages, p.box_rows, f8))
            return cudaErrorInvalidValue;
    } else if (!map_keys(&mk, a.k, a.Hkv, a.T, a.ld_k, 1, p.box_rows, false) ||
               !map_keys(&mv, a.v, a.Hkv, a.T, a.ld_v, 1, p.box_rows, false)) {
        return cudaErrorInvalidValue;
    }
    const long long items = (long long)p.works * p.splits * p.Hkv;
    if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)std::min<long long>(items, sm_count());
    e = f8 ? prepare<true>() : prepare<false>();
    if (e != cudaSuccess) return e;
    if (f8) ragged_attn_tc<true><<<blocks, Ring<true>::threads, kRaggedSmem, st>>>(mq, mk, mv, p);
    else ragged_attn_tc<false><<<blocks, Ring<false>::threads, kRaggedSmem, st>>>(mq, mk, mv, p);
    count_launch();
    e = cudaGetLastError();
    return e == cudaSuccess ? combine_launch(p, st) : e;
}

}  // namespace hs
