// The experts' kernel of the mixture-of-experts layer for weights that TMA can
// address: fp16 in either orientation, and MXFP4.
//
// The layer is bound by reading the chosen experts' weights, once for every piece
// of 11 to 16 tokens (StreamShape) that chose one, so the kernel is built around that
// stream: one thread a CTA keeps a ring of 32 KB pairs of
// weight tiles in flight by TMA, the tensor cores take them from shared memory
// as the 128-row side (tcgen05.mma), and a few token columns are the narrow
// side.  No instruction is spent per weight: MXFP4 codes are multiplied as they
// lie, their scales applied by the block-scaled MMA.  A pair is the gate and
// the up rows of the same 128 hidden values, whose sums meet in one lane, or 256
// rows of the down projection.
//
// Both operands of an MMA have one type, so the narrow side is held in the
// weights' format.  fp16: a hidden value is two columns, its fp16 rounding and
// that of 2^11 times the rest (split_hidden).  MXFP4: a value is 8 columns, each the e2m1
// rounding of what the columns before it leave, which is under 2^-22.5 of the
// block's largest magnitude in the end (split_blocks).  The epilogue adds the
// columns in fp32.
//
// Work is cut into gridDim parts of equal bytes in each of the two phases
// (gate/up, down), wherever that falls: a part's first and last output tile may
// be shared with its neighbours, whose sums go through the workspace; the part
// that finishes such a tile last adds them in order.
//
// A CTA takes parts by ticket.  All gate/up parts have been taken, by CTAs that
// run, before any CTA goes on to the down phase and waits for the hidden values,
// so the wait ends however few CTAs the device holds at once; with one CTA an SM
// each takes one part of either phase.  The weights of a down part are on their
// way before the wait.
//
// Measured, both kernels: 64 tokens, 8 of 64 experts of 7168 x 2048 in MXFP4, 1.5 GB:
// 288 to 295 us (5.2 TB/s); 16 tokens, 8 of 64 of 2048 x 1024 in fp16, 0.7 GB: 128 us; 4
// tokens in MXFP4, 88 MB: 42 us, latency for the most part (routing 7 us, first
// weights 5, exchange between the phases 8, last sums 4).  Experts with several
// pieces: 64 tokens, 4 of 8 of 4096 x 2048 (37 tokens the most) 149 us in fp16 and 93 in
// MXFP4, all 8 (64 each) 260 and 122, where one reading takes 59 and 16.
#pragma once

#include <cuda.h>

#include "moe_kernel.cuh"
#include "mxf4_ptx.cuh"

namespace moe_dev {

constexpr int kLoadWarps = 10;  // warps 6 .. 15 bring the narrow side
constexpr uint32_t kTileBytes = 128 * 128;
constexpr int kMaxParts = 160;
constexpr uint32_t kTmemCols = 512;

// A call's shares of tensor memory, in columns: two accumulators a row tile,
// the scales (MXFP4), and y's sums, a column a token (rounded up to 8) and row tile.
struct StreamShape {
    int cap;                                  // tokens of a piece: of one reading of an expert's weights
    uint32_t acc_cols, y_col, need, alloc;    // an accumulator, where y's sums begin, all, as allocated
    // Pieces of 16 tokens, with MXFP4 as many as there are columns for next to the scales
    // and y's sums: 14 for 16 tokens, 13 for 32, 11 for 64.
    __host__ __device__ constexpr StreamShape(bool mx, int tokens)
        : cap(mx ? static_cast<int>((kTmemCols - 24 - 2 * ((tokens + 7) & ~7)) / (4 * kPieces)) : 16),
          acc_cols(mx ? cap * kPieces : 32),
          y_col(4 * acc_cols + (mx ? 24 : 0)), need(y_col + 2 * ((tokens + 7) & ~7)),
          alloc(need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : kTmemCols)
    {
    }
};

// Columns past the allocation would be an illegal access, so no number of tokens may need more.
constexpr bool every_call_fits()
{
    for (int t = 1; t <= kMaxTokens; ++t)
        if (StreamShape(false, t).need > kTmemCols || StreamShape(true, t).need > kTmemCols) return false;
    return true;
}
static_assert(every_call_fits(), "the expert stream's columns fit tensor memory");

// Counters of one call, zeroed by the routing kernel.
struct StreamControl {
    int done;                 // finished gate/up parts
    int ticket[2];            // parts taken
    int up[kMaxParts];        // by the first part of a shared tile: parts that have stored their sums
    int down[kMaxParts];
};

struct StreamParams {
    CUtensorMap gate, up, down;
    Params p;
    StreamControl* ctl;
    const uint8_t* x;         // narrow side of gate/up: rows (token, column) of xpitch bytes
    const uint8_t* xs;        // MXFP4: their scales, xwords 32-bit words a row
    uint8_t* h;               // narrow side of down: rows (choice by expert, column) of hpitch bytes
    uint8_t* hs;
    float* sums;              // [parts][2][max(cap, T)][256]
    int32_t xpitch, xwords, hpitch, hwords;
    int32_t cap;              // tokens of a piece of an expert's work
    int32_t stages, stage_bytes, b_bytes;   // 3 stages at least
    uint32_t tmem_cols, acc_cols, y_col;    // y_col: y's sums, a column a token (of T, rounded up to 8) and row tile
};

// Ranges of a phase, walked alike by every role of a CTA.
struct Segment {
    int tile, item, s0, s1;   // steps s0 .. s1 - 1 of `steps` for (tile, item)
};

enum { kStreamRows = 0, kStreamCols = 1, kStreamMxf4 = 2 };

__device__ __forceinline__ void tmem_ld_x1(uint32_t taddr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(*r) : "r"(taddr) : "memory");
}

__device__ __forceinline__ void tmem_st_x1(uint32_t taddr, uint32_t r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t* r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}

// Four tokens' sums of this thread's row: `width` adjacent columns each, the
// later, smaller ones added first; two are the halves of hidden values.
template <int kWidth>
__device__ __forceinline__ void take4(uint32_t taddr, float* v)
{
    uint32_t r[4 * kWidth];
    if constexpr (kWidth == 1) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(taddr)
                     : "memory");
    } else {
#pragma unroll
        for (int i = 0; i < 4 * kWidth; i += 8) tmem_ld_x8(taddr + i, r + i);
    }
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (kWidth == 2) {
            v[j] = join_hidden(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        } else {
            v[j] = __uint_as_float(r[j * kWidth + kWidth - 1]);
#pragma unroll
            for (int q = kWidth - 2; q >= 0; --q) v[j] += __uint_as_float(r[j * kWidth + q]);
        }
    }
}

// Whether an output tile, `steps` steps from `first` on, lies in more than one
// part, and in which.
struct Parts {
    int64_t total;
    int count;
    __device__ int64_t start(int part) const { return total * min(part, count) / count; }
    __device__ int of(int64_t step) const
    {
        int v = static_cast<int>((step * count) / total);
        while (start(v + 1) <= step) ++v;
        while (start(v) > step) --v;
        return v;
    }
};

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1) moe_stream(const __grid_constant__ StreamParams sp)
{
    constexpr bool kMx = kFmt == kStreamMxf4;
    const Params& p = sp.p;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* smem = smem_raw + (base - smem_u32(smem_raw));
    __shared__ Choices ch;
    __shared__ __align__(8) uint64_t bars[3 * 16 + 5];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;
    __shared__ int last_flag, fixes;
    __shared__ uint32_t fix[kMaxParts];   // shared tiles of y that this CTA adds up: tile, first and last part
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int parts = gridDim.x;
    // parts of each phase in the order this CTA takes them: the weights' warp
    // draws them, `parts` or more ends the list
    __shared__ volatile int16_t list[2][kMaxParts + 1];

    const uint32_t bar0 = smem_u32(bars);
    auto full_a = [&](int s) { return bar0 + 24u * s; };
    auto full_b = [&](int s) { return bar0 + 24u * s + 8u; };
    auto empty = [&](int s) { return bar0 + 24u * s + 16u; };
    auto tfull = [&](int b) { return bar0 + 24u * 16u + 8u * b; };
    auto tempty = [&](int b) { return bar0 + 24u * 16u + 16u + 8u * b; };
    const uint32_t drain = bar0 + 24u * 16u + 32u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < sp.stages; ++s) {
            mbar_init(full_a(s), 1);
            mbar_init(full_b(s), kLoadWarps);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(tfull(b), 1);
            mbar_init(tempty(b), 4);
        }
        mbar_init(drain, 1);
        abort_flag = 0;
        fixes = 0;

        fence_mbarrier_init();
        tma_prefetch_desc(&sp.gate);
        tma_prefetch_desc(&sp.up);
        tma_prefetch_desc(&sp.down);
    }
    for (int i = threadIdx.x; i <= kMaxParts; i += kThreads) list[0][i] = list[1][i] = -1;
    if (warp == 5) {
        tmem_alloc(smem_u32(&tmem_slot), sp.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    griddep_wait();
    int ticket = 0;   // of the weights' warp
    if (threadIdx.x == 4 * 32) ticket = atomicAdd(&sp.ctl->ticket[0], 1);
    order_choices(p, ch, reinterpret_cast<uint16_t*>(smem), sp.cap);
    fence_proxy_async_smem();   // the counts lay where the copies will write
    __syncthreads();
    tc_fence_after();
    // Only now that this CTA has its tensor memory: a kernel that started in between
    // could take it and then wait for this one.
    griddep_launch_dependents();
    const uint32_t tmem = tmem_slot;
    const int items = ch.items;

    // Phase 0: (piece, 128 hidden values) tiles of d_steps steps; phase 1: 256
    // columns of y, for each all pieces of f_steps steps.
    constexpr int kVals = kMx ? 256 : 64;
    const int d_steps = (p.D + kVals - 1) / kVals, f_steps = (p.F + kVals - 1) / kVals;
    const int f_tiles = (p.F + 127) >> 7, y_tiles = (p.D + 255) >> 8;
    const int64_t up_steps = static_cast<int64_t>(items) * f_tiles * d_steps,
                  down_steps = static_cast<int64_t>(y_tiles) * items * f_steps;
    // (no part is empty but those past the number of steps)
    const Parts phase[2] = {{up_steps, static_cast<int>(min(up_steps, static_cast<int64_t>(parts)))},
                            {down_steps, static_cast<int>(min(down_steps, static_cast<int64_t>(parts)))}};
    auto segment = [&](int ph, int64_t at, int64_t hi) {
        Segment g;
        const int steps = ph ? f_steps : d_steps;
        const int64_t q = at / steps;
        g.s0 = static_cast<int>(at - q * steps);
        g.s1 = static_cast<int>(min(static_cast<int64_t>(steps), g.s0 + hi - at));
        if (ph) {
            g.tile = static_cast<int>(q / items);
            g.item = static_cast<int>(q - static_cast<int64_t>(g.tile) * items);
        } else {
            g.item = static_cast<int>(q / f_tiles);
            g.tile = static_cast<int>(q - static_cast<int64_t>(g.item) * f_tiles);
        }
        return g;
    };
    const volatile int* abort = &abort_flag;
    auto fail = [&]() {
        abort_flag = 1;
        atomicExch(p.status, GEMM_F16_ERR_TIMEOUT);
    };
    // The lanes of a warp wait for themselves and may see a wait's limit pass, or the
    // CTA give up, at different times: before they next meet in a warp-wide
    // instruction they agree, and all go on only if each does.
    // The i-th part of a phase; -1 once the CTA has given up, or when the weights' warp,
    // which names a part as soon as the one before is on its way, has not by the limit.
    auto part_at = [&](int ph, int i) {
        int v = list[ph][i];
        if (v >= 0) return v;
        const uint64_t t0 = globaltimer_ns();
        while ((v = list[ph][i]) < 0)
            if (*abort || globaltimer_ns() - t0 > p.timeout_ns) break;
        return v;
    };
    auto columns = [&](int ph, int count) { return kMx ? count * kPieces : ph ? 2 * count : count; };

    if (warp == 4) {
        // ---------------------------------------------------------- weights
        const bool issue = elect_one();
        int n = 0, st = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int ph = 0; ph < 2 && ok; ++ph) {
            for (int i = 0; (ok = __all_sync(~0u, ok)); ++i) {
                int part = ticket;
                if (ph || i) part = lane == 0 ? atomicAdd(&sp.ctl->ticket[ph], 1) : 0;
                part = __shfl_sync(~0u, part, 0);
                if (lane == 0) list[ph][i] = static_cast<int16_t>(min(part, parts));
                if (part >= parts) break;
                const int64_t hi = phase[ph].start(part + 1);
                for (int64_t at = phase[ph].start(part); at < hi && ok;) {
                    const Segment g = segment(ph, at, hi);
                    at += g.s1 - g.s0;
                    const int e = ch.item[g.item].expert;
                    const CUtensorMap* m0 = ph ? &sp.down : &sp.gate;
                    const CUtensorMap* m1 = ph ? &sp.down : &sp.up;
                    const int o0 = ph ? g.tile * 256 : g.tile * 128, o1 = ph ? o0 + 128 : o0;
                    const Weight& w0 = ph ? p.down : p.gate;
                    const Weight& w1 = ph ? p.down : p.up;
                    // scales of 128 rows and, but at an odd end, two tiles of K; rows
                    // 128 on may be past y's last scale tile (and then past its columns)
                    const bool both = o1 < (ph ? p.D : p.F);
                    const uint8_t* f0 = kMx ? w0.scales + e * w0.scale_se + static_cast<int64_t>(o0 >> 7) * w0.kt * mxf4_dev::kScaleTile : nullptr;
                    const uint8_t* f1 = kMx ? w1.scales + e * w1.scale_se + static_cast<int64_t>(o1 >> 7) * w1.kt * mxf4_dev::kScaleTile : nullptr;
                    for (int s = g.s0; s < g.s1; ++s, ++n) {
                        ok = mbar_wait(empty(st), par ^ 1u, abort, p.timeout_ns);
                        if (!ok) break;
                        const uint32_t a = base + st * sp.stage_bytes;
                        if (issue) {
                            if (kMx) {
                                const uint32_t sf = min(2, w0.kt - 2 * s) * mxf4_dev::kScaleTile;
                                const uint32_t fa = a + 2 * kTileBytes + sp.b_bytes;
                                const int64_t off = static_cast<int64_t>(2 * s) * mxf4_dev::kScaleTile;
                                mbar_arrive_expect_tx(full_a(st), 2 * kTileBytes + (both ? 2 : 1) * sf);
                                bulk_load(fa, f0 + off, sf, full_a(st));
                                if (both) bulk_load(fa + 2 * mxf4_dev::kScaleTile, f1 + off, sf, full_a(st));
                            } else {
                                mbar_arrive_expect_tx(full_a(st), 2 * kTileBytes);
                            }
                            if (kFmt == kStreamCols) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    tma_load_3d(a + h * (kTileBytes / 2), m0, o0 + 64 * h, s * 64, e, full_a(st));
                                    tma_load_3d(a + kTileBytes + h * (kTileBytes / 2), m1, o1 + 64 * h, s * 64, e, full_a(st));
                                }
                            } else {
                                tma_load_3d(a, m0, s * (kMx ? 128 : 64), o0, e, full_a(st));
                                tma_load_3d(a + kTileBytes, m1, s * (kMx ? 128 : 64), o1, e, full_a(st));
                            }
                        }
                        if (++st == sp.stages) st = 0, par ^= 1u;
                    }
                }
            }
        }
        if (!ok) {   // copies in flight land before the CTA leaves
            if (issue) fail();
            for (int q = 0; q < sp.stages && q < n; ++q)
                mbar_wait(full_a(q), ((n - q + sp.stages - 1) / sp.stages - 1) & 1u, nullptr, mxf4_dev::kDrainNs);
        }
    } else if (warp == 5) {
        // -------------------------------------------------------------- MMA
        const bool issue = elect_one();
        int st = 0, buf = 0;
        uint32_t par = 0, bpar = 0;
        bool ok = true;
        const uint32_t tsa = tmem + 4 * sp.acc_cols, tsb = tsa + 16;
        for (int ph = 0; ph < 2 && ok; ++ph) {
            const int k64 = ((ph ? p.F : p.D) + 63) >> 6;
            for (int i = 0; (ok = __all_sync(~0u, ok)); ++i) {
                const int part = __shfl_sync(~0u, part_at(ph, i), 0);
                if (part < 0) ok = false;
                if (part < 0 || part >= parts) break;
                const int64_t hi = phase[ph].start(part + 1);
                for (int64_t at = phase[ph].start(part); at < hi && ok;) {
                    const Segment g = segment(ph, at, hi);
                    at += g.s1 - g.s0;
                    const int cols = columns(ph, ch.item[g.item].count);
                    const uint32_t d = tmem + 2 * buf * sp.acc_cols;
                    ok = mbar_wait(tempty(buf), bpar ^ 1u, abort, p.timeout_ns);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t id0 = kMx ? mxf4_dev::idesc_mxf4(128, (cols + 7) & ~7, 0)
                                             : (1u << 4) | ((kFmt == kStreamCols ? 1u : 0u) << 15) |
                                                   ((static_cast<uint32_t>(cols + 15) >> 4) << 18) | (8u << 24);
                    const uint32_t id1 = kMx ? mxf4_dev::idesc_mxf4(128, (cols + 7) & ~7, 1) : 0u;
                    for (int s = g.s0; s < g.s1; ++s) {
                        ok = mbar_wait(full_a(st), par, abort, p.timeout_ns) && mbar_wait(full_b(st), par, abort, p.timeout_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t a = base + st * sp.stage_bytes, b = a + 2 * kTileBytes;
                        // (descriptors count 16 bytes: 32 of K, or 16 rows of K, a step; 32 a scale tile)
                        const uint64_t da = kFmt == kStreamCols ? umma_desc_sw128(a, 8192, 1024) : umma_desc_sw128(a, 16, 1024);
                        const uint64_t db = umma_desc_sw128(b, 16, 1024);
                        const uint64_t fa = mxf4_dev::scale_desc(b + sp.b_bytes), fb = fa + 4 * 32;
                        if (issue) {
                            const int nk = kMx ? min(4, k64 - 4 * s) : 4;
                            if (kMx) {
#pragma unroll
                                for (int q = 0; q < 2; ++q) {
                                    if (2 * q >= nk) break;
                                    mxf4_dev::tmem_copy_scales(tsa + 4 * q, fa + 32 * q);
                                    mxf4_dev::tmem_copy_scales(tsa + 8 + 4 * q, fa + 64 + 32 * q);
                                    mxf4_dev::tmem_copy_scales(tsb + 4 * q, fb + 32 * q);
                                }
                            }
#pragma unroll
                            for (int t = 0; t < 2; ++t)
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    if (q >= nk) break;
                                    const uint64_t at = da + t * (kTileBytes / 16) + q * (kFmt == kStreamCols ? 128 : 2);
                                    const uint32_t acc = s > g.s0 || q > 0;
                                    if (kMx)
                                        mxf4_dev::umma_mxf4(d + t * sp.acc_cols, at, db + 2 * q, q & 1 ? id1 : id0,
                                                            tsa + 8 * t + 4 * (q >> 1), tsb + 4 * (q >> 1), acc);
                                    else
                                        umma_f16(d + t * sp.acc_cols, at, db + 2 * q, id0, acc);
                                }
                            umma_commit(empty(st));
                        }
                        if (++st == sp.stages) st = 0, par ^= 1u;
                    }
                    if (!ok) break;
                    if (issue) umma_commit(tfull(buf));
                    if (++buf == 2) buf = 0, bpar ^= 1u;
                }
            }
        }
        if (!ok) {   // MMAs in flight end before the CTA's memory goes
            if (issue) {
                fail();
                umma_commit(drain);
            }
            mbar_wait(drain, 0, nullptr, mxf4_dev::kDrainNs);
        }
    } else if (warp >= 6) {
        // ---------------------------------------------------- narrow side
        // Every warp brings some rows of every step and is up to two steps ahead
        // of the one whose copies it has waited for: a stage's next use needs only
        // steps that this warp has handed over (3 stages at least).
        int st = 0, pend = 0, pst = 0;   // steps under way, the stage of the oldest
        uint32_t par = 0;
        bool ok = true;
        const int w = warp - 6, c = lane & 7;
        auto hand_over = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full_b(pst));
            if (++pst == sp.stages) pst = 0;
            --pend;
        };
        auto flush = [&]() {
            cp_async_wait<0>();
            while (pend) hand_over();
        };
        for (int ph = 0; ph < 2 && ok; ++ph) {
            bool waited = ph == 0;
            for (int i = 0; ok; ++i) {
            const int part = part_at(ph, i);
            ok = __all_sync(~0u, part >= 0);
            if (!ok || part >= parts) break;
            const int64_t lo = phase[ph].start(part), hi = phase[ph].start(part + 1);
            const int width = kMx ? kPieces : ph ? 2 : 1;   // rows of a token
            const uint8_t* rows = ph ? sp.h : sp.x;
            const uint8_t* scales = ph ? sp.hs : sp.xs;
            const int64_t pitch = ph ? sp.hpitch : sp.xpitch, words = ph ? sp.hwords : sp.xwords;
            const int kt = (ph ? p.down : p.gate).kt;
            if (!waited && lo < hi) {   // every hidden value is there
                waited = true;
                flush();
                if (lane == 0) {
                    const uint64_t t0 = globaltimer_ns();
                    while (ok && ld_acquire_gpu(&sp.ctl->done) < parts)
                        ok = !*abort && globaltimer_ns() - t0 <= p.timeout_ns;
                }
                __syncwarp();   // the other lanes' reads come after lane 0's acquire (a shuffle orders no memory)
                ok = __shfl_sync(~0u, ok, 0);
                if (!ok) break;
            }
            for (int64_t at = lo; at < hi && ok;) {
                const Segment g = segment(ph, at, hi);
                at += g.s1 - g.s0;
                const Item im = ch.item[g.item];
                const int nrows = im.count * width;
                auto row_of = [&](int r) {
                    const int j = r / width;
                    return static_cast<int64_t>(ph ? im.first + j : ch.slot[im.first + j] / p.top) * width + r - j * width;
                };
                // a lane's rows (no call has larger pieces than one for a token)
                constexpr int kRows = (StreamShape(kMx, 1).cap * (kMx ? kPieces : 2) + 4 * kLoadWarps - 1) / (4 * kLoadWarps);
                const uint8_t* src[kRows];
                uint32_t dst[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int r = (i * kLoadWarps + w) * 4 + (lane >> 3);
                    src[i] = r < nrows ? rows + row_of(r) * pitch + c * 16 : nullptr;
                    dst[i] = r * 128 + ((c ^ (r & 7)) << 4);
                }
                const int sr = w * 32 + lane;   // the row whose scales this lane brings
                const uint8_t* ssrc = kMx && sr < nrows ? scales + row_of(sr) * words * 4 : nullptr;
                for (int s = g.s0; s < g.s1; ++s) {
                    ok = __all_sync(~0u, mbar_wait(empty(st), par ^ 1u, abort, p.timeout_ns));
                    if (!ok) break;
                    const uint32_t b = base + st * sp.stage_bytes + 2 * kTileBytes;
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        if (src[i]) cp_async16(b + dst[i], src[i] + static_cast<int64_t>(s) * 128, 16u);
                    if (kMx && ssrc) {
                        const uint32_t fb = b + sp.b_bytes + 4 * mxf4_dev::kScaleTile + (sr & 31) * 16 + (sr >> 5) * 4;
                        cp_async4(fb, ssrc + s * 8, 4u);
                        if (2 * s + 1 < kt) cp_async4(fb + mxf4_dev::kScaleTile, ssrc + s * 8 + 4, 4u);
                    }
                    cp_async_commit();
                    if (++st == sp.stages) st = 0, par ^= 1u;
                    if (++pend == 3) {
                        cp_async_wait<2>();
                        hand_over();
                    }
                }
            }
            }
        }
        flush();
        if (!ok && lane == 0) fail();
    } else {
        // --------------------------------------------------------- epilogue
        int buf = 0;
        uint32_t bpar = 0;
        bool ok = true;
        const int row = threadIdx.x;   // of the tile
        const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const int64_t slot_floats = static_cast<int64_t>(max(sp.cap, p.T)) * 256;
        // the four warps go on or leave together
        auto all_of = [&](bool mine) {
            uint32_t r;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.u32 p, %1, 0;\n\t"
                "barrier.cta.red.and.pred q, 1, 128, p;\n\t"
                "selp.u32 %0, 1, 0, q;\n\t}"
                : "=r"(r)
                : "r"(static_cast<uint32_t>(mine))
                : "memory");
            return r != 0;
        };
        // the sums of a tile shared by several parts: whether this part is the
        // last to store its own (`first`: the tile's first part)
        auto last_of = [&](int* counter, int sharers) {
            named_bar_sync(1, 128);
            if (threadIdx.x == 0) last_flag = atom_add_acq_rel_gpu(counter, 1) == sharers - 1;
            named_bar_sync(1, 128);
            return last_flag != 0;
        };
        // where part v keeps its sums of a shared tile whose first part is v0: a
        // part has two at most, the tile it begins in and the one it ends in
        auto slot_of = [&](int v, int v0) { return sp.sums + (static_cast<int64_t>(v) * 2 + (v == v0)) * slot_floats; };
        // hidden values (tile's row, tokens j0 .. j0 + 3 of the piece) from their two sums
        auto hidden = [&](const Segment& g, const Item& im, int j0, const float* gate, const float* up) {
            const int f = g.tile * 128 + row;
            float hv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)   // (past F: zeros, whatever the tokens hold)
                hv[j] = f < p.F ? act_f32(p.act, gate[j]) * up[j] : 0.f;
            if (kMx) {
                // lane 8j + i takes values 4i .. 4i + 3 of token j0 + j's block (the warp's 32 rows)
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float o = __shfl_sync(~0u, hv[j], 4 * (lane & 7) + i);
                        v[i] = j == 0 || lane >> 3 == j ? o : v[i];
                    }
                const int j = j0 + (lane >> 3);
                const int64_t r = static_cast<int64_t>(im.first + min(j, im.count - 1)) * kPieces;
                split_blocks(v, j < im.count, lane, sp.h + r * sp.hpitch + ((f - lane) >> 1) + (lane & 7) * 2, sp.hpitch,
                             sp.hs + r * sp.hwords * 4 + ((f - lane) >> 5), sp.hwords * 4);
            } else if (f < p.fp) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j0 + j >= im.count) break;
                    __half* dst = reinterpret_cast<__half*>(sp.h + static_cast<int64_t>(im.first + j0 + j) * 2 * sp.hpitch) + f;
                    split_hidden(hv[j], dst, dst + (sp.hpitch >> 1));
                }
            }
        };
        constexpr int kUpWidth = kMx ? kPieces : 1, kDownWidth = kMx ? kPieces : 2;
        for (int ph = 0; ph < 2 && ok; ++ph) for (int i = 0; ok; ++i) {
            const int part = part_at(ph, i);
            ok = all_of(part >= 0);
            if (!ok || part >= parts) break;
            const Parts& w = phase[ph];
            const int64_t lo = w.start(part), hi = w.start(part + 1);
            bool begun = false;   // (down) ysum holds sums of the current tile
            for (int64_t at = lo; at < hi && ok;) {
                const Segment g = segment(ph, at, hi);
                const Item im = ch.item[g.item];
                ok = all_of(mbar_wait(tfull(buf), bpar, abort, p.timeout_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = trow + 2 * buf * sp.acc_cols;
                auto release = [&]() {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tempty(buf));
                    if (++buf == 2) buf = 0, bpar ^= 1u;
                };
                if (ph == 0) {
                    const int64_t first = at - g.s0;
                    const bool whole = g.s0 == 0 && g.s1 == d_steps;
                    at += g.s1 - g.s0;
                    const int v0 = whole ? part : w.of(first), v1 = whole ? part : w.of(first + d_steps - 1);
                    float* to = slot_of(part, v0) + row;
                    for (int j0 = 0; j0 < im.count; j0 += 4) {
                        float gate[4], up[4];
                        take4<kUpWidth>(d + j0 * kUpWidth, gate);
                        take4<kUpWidth>(d + sp.acc_cols + j0 * kUpWidth, up);
                        if (j0 + 4 >= im.count) release();
                        if (whole) {
                            hidden(g, im, j0, gate, up);
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (j0 + j < im.count) to[(j0 + j) * 256] = gate[j], to[(j0 + j) * 256 + 128] = up[j];
                        }
                    }
                    if (whole) continue;
                    if (!last_of(&sp.ctl->up[v0], v1 - v0 + 1)) continue;
                    for (int j0 = 0; j0 < im.count; j0 += 4) {
                        float gate[4] = {}, up[4] = {};
                        for (int q = v0; q <= v1; ++q) {
                            const float* from = slot_of(q, v0) + row;
                            float a[4], b[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                a[j] = j0 + j < im.count ? ld_cg_f32(from + (j0 + j) * 256) : 0.f;
                                b[j] = j0 + j < im.count ? ld_cg_f32(from + (j0 + j) * 256 + 128) : 0.f;
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) gate[j] += a[j], up[j] += b[j];
                        }
                        hidden(g, im, j0, gate, up);
                    }
                } else {
                    const int64_t per = static_cast<int64_t>(items) * f_steps, first = g.tile * per;
                    at += g.s1 - g.s0;
                    const uint32_t y0 = trow + sp.y_col, y1 = y0 + ((p.T + 7) & ~7);   // this row's, of either row tile
                    if (!begun) {
                        const uint32_t zero[8] = {};
                        for (uint32_t c = y0; c < 2 * y1 - y0; c += 8) mxf4_dev::tmem_st_x8(c, zero);
                        mxf4_dev::tmem_wait_st();
                    }
                    begun = true;
                    for (int j0 = 0; j0 < im.count; j0 += 4) {
                        float a[4], b[4];
                        take4<kDownWidth>(d + j0 * kDownWidth, a);
                        take4<kDownWidth>(d + sp.acc_cols + j0 * kDownWidth, b);
                        if (j0 + 4 >= im.count) release();
                        uint32_t ya[4], yb[4];
                        int t[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            t[j] = ch.slot[im.first + min(j0 + j, im.count - 1)] / p.top;
                            tmem_ld_x1(y0 + t[j], &ya[j]);
                            tmem_ld_x1(y1 + t[j], &yb[j]);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if (j0 + j >= im.count) break;
                            const float wt = ch.weight[im.first + j0 + j];
                            tmem_st_x1(y0 + t[j], __float_as_uint(fmaf(wt, a[j], __uint_as_float(ya[j]))));
                            tmem_st_x1(y1 + t[j], __float_as_uint(fmaf(wt, b[j], __uint_as_float(yb[j]))));
                        }
                        mxf4_dev::tmem_wait_st();
                    }
                    if (at < hi && at < first + per) continue;   // more of this tile
                    begun = false;
                    const int col = g.tile * 256 + row;
                    const bool whole = lo <= first && at == first + per;
                    const int v0 = whole ? part : w.of(first), v1 = whole ? part : w.of(first + per - 1);
                    float* to = slot_of(part, v0) + row;
                    for (int t0 = 0; t0 < p.T; t0 += 8) {
                        uint32_t a[8], b[8];
                        tmem_ld_x8(y0 + t0, a);
                        tmem_ld_x8(y1 + t0, b);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int t = t0 + j;
                            if (t >= p.T) break;
                            if (whole) {
                                if (col < p.D) p.y[t * p.ldy + col] = __float2half_rn(__uint_as_float(a[j]));
                                if (col + 128 < p.D) p.y[t * p.ldy + col + 128] = __float2half_rn(__uint_as_float(b[j]));
                            } else {
                                to[t * 256] = __uint_as_float(a[j]);
                                to[t * 256 + 128] = __uint_as_float(b[j]);
                            }
                        }
                    }
                    if (!whole && last_of(&sp.ctl->down[v0], v1 - v0 + 1) && threadIdx.x == 0)
                        fix[fixes++] = static_cast<uint32_t>(g.tile) << 16 | static_cast<uint32_t>(v0) << 8 | static_cast<uint32_t>(v1);
                }
            }
            if (ph == 0 && ok) {
                named_bar_sync(1, 128);
                if (threadIdx.x == 0 && !p.test_stall) atom_add_acq_rel_gpu(&sp.ctl->done, 1);
            }
        }
        if (!ok) abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, sp.tmem_cols);
    // Shared tiles of y whose last sums this CTA stored: 4 columns a thread, 4
    // parts' and 2 tokens' loads under way at once.
    for (int i = 0; i < fixes; ++i) {
        const int tile = fix[i] >> 16, v0 = fix[i] >> 8 & 255, v1 = fix[i] & 255, c4 = threadIdx.x & 63;
        const int64_t slot_floats = static_cast<int64_t>(max(sp.cap, p.T)) * 256;
        for (int t0 = threadIdx.x >> 6; t0 < p.T; t0 += 16) {
            float4 v[2] = {};
            for (int q0 = v0; q0 <= v1; q0 += 4) {
                float4 a[4][2];
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int u = min(q0 + q, v1);
                        a[q][h] = __ldcg(reinterpret_cast<const float4*>(sp.sums + (static_cast<int64_t>(u) * 2 + (u == v0)) * slot_floats +
                                                                         min(t0 + 8 * h, p.T - 1) * 256) + c4);
                    }
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (q0 + q <= v1) v[h].x += a[q][h].x, v[h].y += a[q][h].y, v[h].z += a[q][h].z, v[h].w += a[q][h].w;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int t = t0 + 8 * h, col = tile * 256 + c4 * 4;
                if (t >= p.T) break;
                const float f[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (col + e < p.D) p.y[t * p.ldy + col + e] = __float2half_rn(f[e]);
            }
        }
    }
}

}  // namespace moe_dev
