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
// A piece of at most `chunk` key tiles is one CTA's; sequences with more keys
// are split over several CTAs, whose partial results a second kernel joins.
//
// CTA (warps):
//   0-3, 4-7  softmax warpgroups, thread = row
//   8         TMA producer (Q once; K and V tiles, or the pages that make one
//             up, in the order the MMAs consume them)
//   9         MMA issuer (one thread)
//   10        zeroes the value rows behind a sequence's end (whatever lies
//             there, NaN included, would reach the output as 0 * NaN)
//   12-15     8-bit caches only: widen staged rows to bf16 tiles.  A code
//             times a power of two is a bf16 number, so nothing is rounded.
// TMEM (512 columns): S0 | S1 | O0 | O1.  P overwrites its S tile (64 of 128
// columns) and is the MMA's A operand there: with both operands in shared
// memory, Q K^T and P V of 128 keys read 128 bytes a clock, all that shared
// memory has, and writing P there too would add a quarter; from TMEM the P V
// products read V only.  The two tiles alternate on the tensor cores: one's
// softmax runs under the other's products.
#include <algorithm>
#include <atomic>

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

// Shared memory: Q0, Q1, then five K/V tiles; for 8-bit caches three tiles
// and four staged 8-bit tiles.
template <bool F8> struct Ring {
    static constexpr int slots = F8 ? 3 : 5;
    static constexpr int stages = F8 ? 4 : 0;
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
    int b, q0, ql, kvl;        // sequence, its first packed row, its rows, its keys
    int t0, nq;                // first token of this CTA (within the sequence), tokens
    int off;                   // position of token 0 of the sequence (kvl - ql; may be negative)
    int j0, n, n0, n1;         // first key tile; tiles for the CTA, of row tile 0 and 1
    int solo, go, partial;
};

struct RaggedBars {
    uint64_t q_full;
    uint64_t kv_full[5], kv_empty[5];
    uint64_t st_full[4], st_empty[4];     // staged 8-bit tiles
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t vgo, vfix;                   // last value tile: there / its rows behind the end zeroed
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
    uint32_t bad_any[kBadBufs];           // key tile j has keys on pages outside the pool: bad[j % 8] says which
    uint32_t bad[kBadBufs][4];
    uint8_t scale[2][128];                // 8-bit caches: scale bytes of the tile being widened
    float2 side[128];                     // solo: warpgroup 1's maximum and sum of each row
    Work work;
};

constexpr size_t kRaggedSmem = 1024 + 7 * TILE + sizeof(RaggedBars);
static_assert(kRaggedSmem <= 232448, "ragged attention shared memory");

struct RaggedParams {
    PagedCache c;              // cu_rows, B; paged: kv_len, block_table, pages, scales
    int paged;
    int T, Hq, Hkv, G, tpt;    // tpt: tokens per 128-row tile (128 / G)
    int box_rows;              // keys one TMA box brings
    int works, splits, chunk;  // launched work items; pieces per item; key tiles per piece
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

// Which sequence and rows work item `idx` is (one warp).  Up to 32 sequences:
// items in descending order of their keys, so that the longest start first.
// More: in order, each sequence's last rows first.
__device__ __forceinline__ bool find_work(const RaggedParams &p, int idx, Work *w) {
    const int lane = threadIdx.x & 31;
    const int qt = 2 * p.tpt;
    const int B = p.c.B;
    int b = -1, t = 0;
    if (B <= 32) {
        int q0, ql = 0, kvl = 0;
        if (lane < B) seq_bounds(p, lane, q0, ql, kvl);
        const int nt = (ql + qt - 1) / qt;
        const int base = max(kvl - ql, 0) / qt;
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
    } else {
        const int per = (B + 31) / 32, first = lane * per, last = min(first + per, B);
        int sum = 0;
        for (int i = first; i < last; ++i) {
            int q0, ql, kvl;
            seq_bounds(p, i, q0, ql, kvl);
            sum += (ql + qt - 1) / qt;
        }
        int upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const int total = __shfl_sync(0xffffffffu, upto, 31);
        if (idx == 0 && lane == 0 && total > p.works) report(p.status, HS_ERR_INVALID_ARG);
        if (idx >= total) return false;
        const int owner = __ffs(__ballot_sync(0xffffffffu, upto > idx)) - 1;
        if (lane == owner) {
            int left = idx - (upto - sum);
            for (int i = first; i < last; ++i) {
                int q0, ql, kvl;
                seq_bounds(p, i, q0, ql, kvl);
                const int nt = (ql + qt - 1) / qt;
                if (left < nt) {
                    b = i;
                    t = nt - 1 - left;
                    break;
                }
                left -= nt;
            }
        }
        b = __shfl_sync(0xffffffffu, b, owner);
        t = __shfl_sync(0xffffffffu, t, owner);
    }
    w->b = b;
    seq_bounds(p, b, w->q0, w->ql, w->kvl);
    if (lane == 0 && (__ldg(p.c.cu_rows + b + 1) > p.T || __ldg(p.c.cu_rows + b) < 0 ||
                      (p.paged && __ldg(p.c.kv_len + b) != w->kvl)))
        report(p.status, HS_ERR_INVALID_ARG);
    w->t0 = t * qt;
    w->nq = min(qt, w->ql - w->t0);
    w->off = w->kvl - w->ql;
    return true;
}

__device__ __forceinline__ int key_tiles(int last_pos) { return last_pos < 0 ? 0 : last_pos / BN + 1; }

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

// Two 8-bit floats (low halves of both 16-bit lanes of `x`, i.e. x = code0 |
// code1 << 16) to a bf16 pair scaled by 2^-120: the code's four exponent bits
// go to the low end of the bf16 exponent, whose bias is larger by 120;
// subnormal codes become subnormal bf16 numbers.
__device__ __forceinline__ uint32_t e4m3_to_bf16_tiny(uint32_t x) {
    return ((x & 0x00800080u) << 8) | ((x & 0x007f007fu) << 4);
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Named barrier 2 over 128 threads; whether all of them said yes.
__device__ __forceinline__ bool all_128(bool yes) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)yes)
        : "memory");
    return r != 0;
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
    RaggedBars *bars = reinterpret_cast<RaggedBars *>(smem + 7 * TILE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = blockIdx.x % p.Hkv;
    const int item = blockIdx.x / p.Hkv;
    const int piece = item % p.splits;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bars->q_full), 1);
        for (int s = 0; s < 5; ++s) {
            mbar_init(smem_u32(&bars->kv_full[s]), F8 ? 128 : 1);
            mbar_init(smem_u32(&bars->kv_empty[s]), 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(smem_u32(&bars->st_full[s]), 1);
            mbar_init(smem_u32(&bars->st_empty[s]), 128);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_u32(&bars->s_full[w]), 1);
            mbar_init(smem_u32(&bars->p_full[w]), 128);
            mbar_init(smem_u32(&bars->o_full[w]), 1);
        }
        mbar_init(smem_u32(&bars->vgo), 1);
        mbar_init(smem_u32(&bars->vfix), 32);
        mbar_init(smem_u32(&bars->drain), 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(&bars->tmem_base), 512);
        tmem_relinquish();
    }
    if (warp == 8) {
        if (lane == 0) {
            tma_prefetch(&tq);
            tma_prefetch(&tk);
            tma_prefetch(&tv);
        }
        Work w{};
        const bool go = find_work(p, item / p.splits, &w);
        if (go) {
            const int nk = key_tiles(w.off + w.t0 + w.nq - 1);
            const int nk0 = key_tiles(w.off + w.t0 + min(p.tpt, w.nq) - 1);
            w.solo = w.nq <= p.tpt;
            w.j0 = min(piece * p.chunk, nk);
            // (the last piece also takes keys past the length the plan was made for)
            w.n = piece == p.splits - 1 ? nk - w.j0 : min(nk - w.j0, p.chunk);
            if (w.solo) {
                w.n0 = (w.n + 1) >> 1;
                w.n1 = w.n >> 1;
            } else {
                w.n0 = min(max(nk0 - w.j0, 0), w.n);
                w.n1 = w.n;
            }
            // one piece holds all the keys: no partial results for this item
            w.partial = nk > p.chunk;
        }
        w.go = go;
        if (lane == 0) bars->work = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int *abort = &bars->abort;
    const bool go = bars->work.go != 0;
    const bool solo = bars->work.solo != 0;
    const int n = bars->work.n;          // key tiles of this CTA (0: rows that see nothing, or an empty piece)
    const int jb = bars->work.j0;
    const int kvl = bars->work.kvl;
    // value rows behind the sequence's end in the last tile
    const int tail = go && n > 0 && (jb + n) * BN > kvl ? kvl - (jb + n - 1) * BN : BN;

    if (warp >= 8) {
        regs_release<R::ctl>();
        if (warp == 8 && go && n > 0) {
            // ------------------------------------------------ TMA producer
            const int q_row = bars->work.q0;
            const int32_t *table = p.paged ? p.c.block_table + (size_t)bars->work.b * p.c.max_pages : nullptr;
            const uint32_t qb = smem_u32(&bars->q_full);
            if (lane == 0) {
                const int tiles = solo ? 1 : 2;
                mbar_expect_tx(qb, tiles * 2 * p.tpt * p.G * 128);
                for (int s = 0; s < tiles; ++s)
                    for (int hf = 0; hf < 2; ++hf)
                        tma_load_3d(smem_u32(sq + s * TILE + hf * HALF), &tq, qb, hf * 64, g * p.G,
                                    q_row + bars->work.t0 + s * p.tpt);
            }
            constexpr int slots = F8 ? R::stages : R::slots;
            uint64_t *full = F8 ? bars->st_full : bars->kv_full;
            uint64_t *empty = F8 ? bars->st_empty : bars->kv_empty;
            constexpr int parts = F8 ? 1 : 2;        // boxes per group of rows (64-column halves of bf16 rows)
            constexpr int row_bytes = 128;           // per box row
            const int rshift = 31 - __clz(p.box_rows);
            RingPos pos;
            int issued = 0;
            bool ok = true;
            for (int it = 0; it < 2 * n; ++it) {
                int j;
                bool is_v;
                kv_item(it, n, solo, j, is_v);
                const int key0 = (jb + j) * BN;
                const int boxes = p.paged ? (min(BN, kvl - key0) + p.box_rows - 1) >> rshift : 1;
                int page = 0;
                if (p.paged && lane < boxes) page = __ldg(table + ((key0 + (lane << rshift)) >> p.c.page_shift));
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[pos.slot]), pos.phase ^ 1, p.wait_ns, abort));
                if (!ok) break;
                const uint32_t fb = smem_u32(&full[pos.slot]);
                const uint32_t dst = smem_u32(F8 ? sst + pos.slot * kStage : skv + pos.slot * TILE);
                const CUtensorMap *m = is_v ? &tv : &tk;
                if (!is_v) {
                    if (lane == 0) bars->bad_any[j % kBadBufs] = 0;
                    if (lane < 4) bars->bad[j % kBadBufs][lane] = 0;
                }
                if (lane == 0) mbar_expect_tx(fb, (uint32_t)(boxes * p.box_rows * parts * row_bytes));
                __syncwarp();
                for (int i = lane; i < boxes; i += 32) {
                    int c2 = 0, c3 = 0;
                    if (p.paged) {
                        const int key = key0 + (i << rshift);
                        if (i >= 32) page = __ldg(table + (key >> p.c.page_shift));
                        c2 = key & ((1 << p.c.page_shift) - 1);
                        c3 = page;
                        if (page < 0 || page >= p.c.num_pages) {
                            // outside the pool: a box past the map's end reads zeros,
                            // and the softmax leaves its keys out
                            report(p.status, HS_ERR_INVALID_INDEX);
                            c3 = p.c.num_pages;
                            if (!is_v) {
                                bars->bad_any[j % kBadBufs] = 1;
                                for (int r = 0; r < p.box_rows; ++r)
                                    atomicOr(&bars->bad[j % kBadBufs][((i << rshift) + r) >> 5],
                                             1u << (((i << rshift) + r) & 31));
                            }
                        }
                    } else {
                        c2 = q_row + key0;
                    }
                    for (int hf = 0; hf < parts; ++hf)
                        tma_load_4d(dst + hf * HALF + (i << rshift) * row_bytes, m, fb, hf * 64, g, c2, c3);
                }
                issued = it + 1;
                pos.next(slots);
            }
            __syncwarp();
            if (lane == 0 && *abort) {   // let our own copies land before the CTA goes away
                mbar_drain(qb, 0);
                for (int it = issued > slots ? issued - slots : 0; it < issued; ++it)
                    mbar_drain(smem_u32(&full[it % slots]), (it / slots) & 1);
            }
        } else if (warp == 9 && go && n > 0) {
            // ------------------------------------------------ MMA issuer
            if (lane == 0) {
                const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 384};
                const uint32_t qa[2] = {smem_u32(sq), smem_u32(sq + (solo ? 0 : TILE))};
                const int nw[2] = {bars->work.n0, bars->work.n1};
                int done_qk[2] = {0, 0}, done_pv[2] = {0, 0};
                RingPos pos;
                bool ok = mbar_wait(smem_u32(&bars->q_full), 0, p.wait_ns, abort);
                auto kv_wait = [&]() {
                    ok = ok && mbar_wait(smem_u32(&bars->kv_full[pos.slot]), pos.phase, p.wait_ns, abort);
                    if (ok) tc_fence_after();
                    return ok;
                };
                auto qk = [&](int w) {
                    issue_qk(tS[w], qa[w], smem_u32(skv + pos.slot * TILE));
                    mma_commit(smem_u32(&bars->s_full[w]));
                    ++done_qk[w];
                };
                auto pv = [&](int w, uint32_t v_addr) {
                    ok = mbar_wait(smem_u32(&bars->p_full[w]), done_pv[w] & 1, p.wait_ns, abort);
                    if (!ok) return;
                    tc_fence_after();
                    issue_pv(tO[w], tS[w], v_addr, done_pv[w] > 0);
                    if (++done_pv[w] == nw[w]) mma_commit(smem_u32(&bars->o_full[w]));
                };
                // the last value tile may have rows to be zeroed first
                auto tail_wait = [&](int j) {
                    if (!F8 && j == n - 1 && tail < BN) {
                        mbar_arrive(smem_u32(&bars->vgo));
                        ok = ok && mbar_wait(smem_u32(&bars->vfix), 0, p.wait_ns, abort);
                        if (ok) tc_fence_after();
                    }
                };
                auto release = [&]() {
                    mma_commit(smem_u32(&bars->kv_empty[pos.slot]));
                    pos.next(R::slots);
                };
                if (!solo) {
                    if (kv_wait()) {
                        for (int w = 0; w < 2; ++w)
                            if (nw[w] > 0) qk(w);
                        release();
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        if (!kv_wait()) break;
                        tail_wait(j);
                        if (!ok) break;
                        const RingPos vpos = pos;
                        const uint32_t v_addr = smem_u32(skv + vpos.slot * TILE);
                        pos.next(R::slots);
                        bool have_k = false;
                        for (int w = 0; ok && w < 2; ++w) {
                            if (j < nw[w]) pv(w, v_addr);
                            if (ok && w == 1) mma_commit(smem_u32(&bars->kv_empty[vpos.slot]));
                            if (ok && j + 1 < nw[w]) {
                                if (!have_k && !kv_wait()) break;
                                have_k = true;
                                qk(w);
                            }
                        }
                        if (ok && have_k) release();
                    }
                } else {
                    for (int j = 0; ok && j < min(n, 2); ++j) {
                        if (!kv_wait()) break;
                        qk(j);
                        release();
                    }
                    for (int j = 0; ok && j < n; ++j) {
                        if (!kv_wait()) break;
                        tail_wait(j);
                        if (!ok) break;
                        pv(j & 1, smem_u32(skv + pos.slot * TILE));
                        if (!ok) break;
                        release();
                        if (j + 2 < n) {
                            if (!kv_wait()) break;
                            qk(j & 1);
                            release();
                        }
                    }
                }
                // all MMAs this thread issued have completed before TMEM is freed
                mma_commit(smem_u32(&bars->drain));
                mbar_drain(smem_u32(&bars->drain), 0);
            }
        } else if (!F8 && warp == 10 && go && tail < BN) {
            // ------------------------------------------------ value rows behind the end
            // (the MMA thread, which has waited for the tile, says when)
            const int slot = (2 * n - 1) % R::slots;
            const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->vgo), 0, p.wait_ns, abort));
            if (ok) {
                // whole 128-byte rows, so the swizzle within a row does not matter
                for (int i = lane; i < (BN - tail) * 16; i += 32) {
                    const int row = tail + (i >> 4), part = i & 15;
                    *reinterpret_cast<uint4 *>(skv + slot * TILE + (part >> 3) * HALF + row * 128 + (part & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(&bars->vfix));
            }
        } else if (F8 && warp >= 12 && go && n > 0) {
            // ------------------------------------------------ 8-bit rows to bf16 tiles
            const int t = threadIdx.x - 384;
            const int32_t *table = p.c.block_table + (size_t)bars->work.b * p.c.max_pages;
            const int c16 = t & 7, r0 = t >> 3;      // 16 codes of rows r0, r0 + 16, ...
            auto scale_load = [&](int it) -> int {   // scale byte of this thread's row (t) of item `it`
                if (it >= 2 * n) return 0;
                int j;
                bool is_v;
                kv_item(it, n, solo, j, is_v);
                const int key = (jb + j) * BN + t;
                if (key >= kvl) return 0;
                const int page = __ldg(table + (key >> p.c.page_shift));
                if (page < 0 || page >= p.c.num_pages) return 0;
                const uint8_t *s = is_v ? p.c.v_scale : p.c.k_scale;
                return __ldg(s + (((size_t)page * p.Hkv + g) << p.c.page_shift) + (key & ((1 << p.c.page_shift) - 1)));
            };
            RingPos st, kv;
            int byte = scale_load(0);
            bool ok = true;
            for (int it = 0; it < 2 * n; ++it) {
                bars->scale[it & 1][t] = (uint8_t)byte;
                byte = scale_load(it + 1);
                ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->st_full[st.slot]), st.phase, p.wait_ns, abort));
                ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->kv_empty[kv.slot]), kv.phase ^ 1, p.wait_ns,
                                                             abort));
                // the four warps meet here for the scale bytes, and leave together when
                // one of them gave up waiting
                if (!all_128(ok)) break;
                const uint8_t *src = sst + st.slot * kStage;
                uint8_t *dst = skv + kv.slot * TILE;
                const int live = it == 2 * n - 1 ? tail : BN;   // value rows behind the end are zeroed
#pragma unroll 4
                for (int i = 0; i < 8; ++i) {
                    const int row = r0 + 16 * i;
                    const uint4 u = *reinterpret_cast<const uint4 *>(src + row * 128 + c16 * 16);
                    const int e = (int)bars->scale[it & 1][row] - 7;          // 120 + (byte - 127)
                    const int e1 = max(min(e, 127), -126), e2 = min(e - e1, 127);
                    const uint32_t f1 = (uint32_t)(e1 + 127) * 0x00800080u;
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
                    uint32_t o[8];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        o[2 * q] = bf16x2_mul(e4m3_to_bf16_tiny(__byte_perm(w[q], 0, 0x4140)), f1);
                        o[2 * q + 1] = bf16x2_mul(e4m3_to_bf16_tiny(__byte_perm(w[q], 0, 0x4342)), f1);
                    }
                    if (e2 != 0) {       // scales above 2^7 take a second power of two
                        const uint32_t f2 = (uint32_t)(e2 + 127) * 0x00800080u;
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = bf16x2_mul(o[q], f2);
                    }
                    if (row >= live) {
#pragma unroll
                        for (int q = 0; q < 8; ++q) o[q] = 0;
                    }
                    // chunks 2 c16 and 2 c16 + 1 of the row's 16 (8 a half); lanes of
                    // the second half store them in the other order, so that the
                    // eight lanes of a store phase touch all banks
                    uint8_t *row_dst = dst + (c16 >> 2) * HALF + row * 128;
                    const int c0 = (2 * c16) & 7;
                    const uint4 a = make_uint4(o[0], o[1], o[2], o[3]), b = make_uint4(o[4], o[5], o[6], o[7]);
                    const bool second = c16 >= 4;
                    *reinterpret_cast<uint4 *>(row_dst + (((c0 + (second ? 1 : 0)) ^ (row & 7)) << 4)) = second ? b : a;
                    *reinterpret_cast<uint4 *>(row_dst + (((c0 + (second ? 0 : 1)) ^ (row & 7)) << 4)) = second ? a : b;
                }
                fence_proxy_async_smem();
                mbar_arrive(smem_u32(&bars->kv_full[kv.slot]));
                mbar_arrive(smem_u32(&bars->st_empty[st.slot]));
                st.next(R::stages);
                kv.next(R::slots);
            }
        }
    } else {
        regs_acquire<R::soft>();
        // ------------------------------------------------ softmax warpgroups
        const int w = warp >> 2;
        const int tw = threadIdx.x - 128 * w;
        const int tok = bars->work.t0 + (solo ? 0 : w * p.tpt) + tw / p.G;
        const int h = g * p.G + tw % p.G;
        const bool valid = go && tw < p.tpt * p.G && tok < bars->work.ql;
        const int pos = bars->work.off + min(tok, bars->work.ql - 1);
        // a key tile with any key past this position needs the causal mask
        const int pos_first = bars->work.off + bars->work.t0 + (solo ? 0 : w * p.tpt);
        const uint32_t lane_off = (uint32_t)(tw & ~31) << 16;
        const uint32_t tS = tmem + lane_off + (uint32_t)(w * 128);
        const uint32_t tO = tmem + lane_off + 256u + (uint32_t)(w * 128);
        const float c2 = p.scale_log2;
        const int nw = go ? (w == 0 ? bars->work.n0 : bars->work.n1) : 0;
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int i = 0; i < nw; ++i) {
            const int j = solo ? 2 * i + w : i;
            const int key0 = (jb + j) * BN;
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->s_full[w]), i & 1, p.wait_ns, abort));
            if (!ok) break;
            tc_fence_after();
            // S_i is there, and P V of the previous tile (issued before it) is done
            float s[128];
            {
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, r[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 128; ++c) s[c] = __uint_as_float(r[c >> 5][c & 31]);
            }
            if (key0 + BN - 1 > pos_first) {
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if (key0 + c > pos) s[c] = -INFINITY;
            }
            if (p.paged && bars->bad_any[j % kBadBufs]) {
#pragma unroll
                for (int c = 0; c < 128; ++c)
                    if ((bars->bad[j % kBadBufs][c >> 5] >> (c & 31)) & 1u) s[c] = -INFINITY;
            }
            float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 128; c += 2) m4[(c >> 1) & 3] = fmax3(m4[(c >> 1) & 3], s[c], s[c + 1]);
            const float mx2 = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
            // the running maximum only moves when it grows by more than 8 (log2
            // units); the final division uses the same reference
            if (__any_sync(0xffffffffu, mx2 > m + 8.0f)) {
                const float m_new = fmaxf(m, mx2);
                if (i > 0) {
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
            const float mref = m == -INFINITY ? 0.f : m;   // masked keys (-inf) give 2^-inf = 0
            const float2 c2v = make_float2(c2, c2), mv = make_float2(-mref, -mref);
            float2 ps01 = make_float2(0.f, 0.f), ps23 = make_float2(0.f, 0.f);
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {            // 32 keys, 16 TMEM columns of bf16 pairs
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int c = ch * 32 + 2 * e;
                    const float2 t = ffma2(make_float2(s[c], s[c + 1]), c2v, mv);
                    const float2 ab = make_float2(ex2(t.x), ex2(t.y));
                    if (e & 1) ps23 = fadd2(ps23, ab); else ps01 = fadd2(ps01, ab);
                    // P is rounded to bf16, the type of V: one MMA takes one type
                    pk[e] = pack_bf16(ab.x, ab.y);
                }
                tmem_st16(tS + 16 * ch, pk);
            }
            l += (ps01.x + ps01.y) + (ps23.x + ps23.y);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&bars->p_full[w]));
        }
        bool fin = ok;
        if (nw > 0)
            fin = __all_sync(0xffffffffu, ok && mbar_wait(smem_u32(&bars->o_full[w]), 0, p.wait_ns, abort));
        tc_fence_after();
        // O of this thread's row: columns [16 c, 16 c + 16), zeros when there were no tiles
        auto load_o = [&](int c, float (&o)[16]) {
            uint32_t r[16];
            if (nw > 0) {
                tmem_ld16(tO + 16 * c, r);
                tmem_wait_ld();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = nw > 0 ? __uint_as_float(r[e]) : 0.f;
        };
        const bool join = go && solo && n > 1;
        float *const side = reinterpret_cast<float *>(sq) + tw * 128;   // 64 KB: the Q tiles, no longer read
        float a0 = 1.f, a1 = 0.f;
        if (join) {
            // warpgroup 1 hands its half of the keys over through shared memory
            if (w == 1) {
                bars->side[tw] = make_float2(fin ? m : __int_as_float(0x7fc00000), l);
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                    float o[16];
                    load_o(c, o);
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4 *>(side + (((4 * c + e) ^ (tw & 31)) << 2)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            if (w == 0) {
                const float2 other = bars->side[tw];
                const float top = fmaxf(m, other.x);
                if (other.x != other.x) fin = false;
                a0 = m == -INFINITY ? 0.f : ex2(m - top);
                a1 = other.x == -INFINITY ? 0.f : ex2(other.x - top);
                l = l * a0 + other.y * a1;
                m = top;
            }
        }
        const bool partial = bars->work.partial != 0;
        // the row's result is this CTA's to write: not warpgroup 1 of a shared
        // tile, and not an empty piece of an item that one piece holds
        if (valid && !(solo && w == 1) && (partial || piece == 0)) {
            const size_t row = (size_t)bars->work.q0 + tok;
            const size_t pr = ((size_t)piece * p.T + row) * p.Hq + h;
            const float bad = __int_as_float(0x7fc00000);
            if (partial) p.part_ml[pr] = make_float2(fin ? m : bad, l);
            else {
                if (p.splits > 1) p.part_ml[pr] = make_float2(0.f, -1.f);
                // a bounded wait gave up: NaN in the row's lse, as in the full layer
                p.lse[(size_t)h * p.T + row] = !fin ? bad : (l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY);
            }
        }
        if (go && !(solo && w == 1) && (partial ? n > 0 : piece == 0)) {
            const size_t row = (size_t)bars->work.q0 + tok;
            const float inv_l = partial ? 1.f : (l > 0.f ? 1.0f / l : 0.f);   // a row that sees nothing gives zeros
            a0 *= inv_l;
            a1 *= inv_l;
            __nv_bfloat16 *orow = p.out + (row * p.Hq + h) * HD;
            float *prow = p.part_o + (((size_t)piece * p.T + row) * p.Hq + h) * HD;
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
                float o[16];
                load_o(c, o);
                if (!valid) continue;
                if (join) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 y = *reinterpret_cast<const float4 *>(side + (((4 * c + e) ^ (tw & 31)) << 2));
                        o[4 * e] = o[4 * e] * a0 + y.x * a1;
                        o[4 * e + 1] = o[4 * e + 1] * a0 + y.y * a1;
                        o[4 * e + 2] = o[4 * e + 2] * a0 + y.z * a1;
                        o[4 * e + 3] = o[4 * e + 3] * a0 + y.w * a1;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] *= a0;
                }
                if (partial) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<float4 *>(prow + 16 * c + 4 * e) =
                            make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                } else {
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) pk[e] = pack_bf16(o[2 * e], o[2 * e + 1]);
                    uint4 *dst = reinterpret_cast<uint4 *>(orow + 16 * c);
                    dst[0] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    dst[1] = make_uint4(pk[4], pk[5], pk[6], pk[7]);
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
    if (t < clamp_row(__ldg(p.c.cu_rows), p.T) || t >= clamp_row(__ldg(p.c.cu_rows + p.c.B), p.T)) return;
    if (p.part_ml[r].y < 0.f) return;                       // written by its only piece
    float m = -INFINITY;
    for (int s = lane; s < p.splits; s += 32) m = fmaxf(m, p.part_ml[s * rows + r].x);
    m = warp_max(m);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < p.splits; ++s) {
        const float2 ml = p.part_ml[s * rows + r];
        if (ml.x == -INFINITY) continue;                    // nothing seen in this piece
        const float a = exp2f(ml.x - m);                    // NaN (a piece that gave up) carries through
        l += a * ml.y;
        const float4 o = *reinterpret_cast<const float4 *>(p.part_o + (s * rows + r) * HD + lane * 4);
        acc.x += a * o.x;
        acc.y += a * o.y;
        acc.z += a * o.z;
        acc.w += a * o.w;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
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
constexpr int kMaxSplits = 64;
constexpr int kFewRows = 16;               // rows (new tokens x group) a sequence up to which the warp-MMA kernel runs
constexpr int kFewRowsCtas16 = 2, kFewRowsCtas8 = 3;   // CTAs of that kernel an SM holds (bf16, 8-bit caches)
constexpr int kFewRowsFixed = 8;           // what a piece costs besides its keys, in 16-key blocks
constexpr int kFewRowsMinChunk = 4;        // fewest 16-key blocks in a piece (one for each warp)
constexpr size_t kMaxPartRows = 180000;    // rows of partial results: 520 bytes each

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
    if (a.paged && row_most <= kFewRows) {
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

cudaError_t ragged_attn_launch(const RaggedCall &a, const RaggedPlan &pl, void *ws, unsigned long long wait_ns,
                               cudaStream_t st) {
    using namespace tc;
    cudaError_t e = cudaSuccess;
    RaggedParams p{};
    p.c = a.cache;
    p.paged = a.paged;
    p.T = a.T; p.Hq = a.Hq; p.Hkv = a.Hkv; p.G = a.Hq / a.Hkv; p.tpt = 128 / p.G;
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
    const long long blocks = (long long)p.works * p.splits * p.Hkv;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    e = f8 ? prepare<true>() : prepare<false>();
    if (e != cudaSuccess) return e;
    if (f8) ragged_attn_tc<true><<<(unsigned)blocks, Ring<true>::threads, kRaggedSmem, st>>>(mq, mk, mv, p);
    else ragged_attn_tc<false><<<(unsigned)blocks, Ring<false>::threads, kRaggedSmem, st>>>(mq, mk, mv, p);
    count_launch();
    e = cudaGetLastError();
    return e == cudaSuccess ? combine_launch(p, st) : e;
}

}  // namespace hs
