// C[m, n] = act(sum_k A[m, k] B[n, k] + bias[n]) for two matrices held in 8 bits
// (e4m3 with a power-of-two scale for 128 values of k), and its grouped form.
//
// The tensor cores take the codes from shared memory and the scales from tensor
// memory (tcgen05.mma kind::mxf8f6f4, block_scale, 32 values of K an instruction, one
// scale byte for each row): every product is exact, sums are fp32 in tensor memory,
// and no sum is taken out to be scaled.  A row of a pipeline slot is 128 bytes = one
// block of 128 values, so that the four instructions of a slot share their scales: a
// word of a scale tile holds four blocks, and the slot's place in it goes into the
// instruction descriptor.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "activation.cuh"
#include "fp8_format.cuh"
#include "fp8_tiles.h"
#include "gemm_f16.h"
#include "mxf4_ptx.cuh"
#include "ptx.cuh"

namespace fp8_dev {

using mxf4_dev::act_all;
using mxf4_dev::act_f32;
using mxf4_dev::kDrainNs;
using mxf4_dev::mbar_arrive_cluster_relaxed;
using mxf4_dev::scale_desc;
using mxf4_dev::tmem_copy_scales;

// D[tmem] (+)= A * B with block scales, 32 values of K.
__device__ __forceinline__ void umma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: e4m3 A and B (0), E8M0 scales (bit 23), N / 8 (17-22),
// M / 128 (27-28), the scales' byte of B (4-5) and of A (29-30).
__host__ __device__ constexpr uint32_t idesc_mxf8(uint32_t m, uint32_t n, uint32_t byte)
{
    return (1u << 23) | ((n >> 3) << 17) | ((m >> 7) << 27) | (byte << 4) | (byte << 29);
}

// An fp32 value as fp16 or bf16, in the low half.
__device__ __forceinline__ uint16_t narrow(float v, int bf16)
{
    return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ uint32_t narrow2(float lo, float hi, int bf16)
{
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    return pack_half2(lo, hi);
}

__device__ __forceinline__ float widen(uint16_t v, int bf16)
{
    return bf16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
}

// ------------------------------------------------------------------ few rows
struct TileParams {
    CUtensorMap tmA, tmB;        // codes: {pitch bytes, rows}, box {128, 128 or bn}
    const uint8_t* sfa;          // scale tiles of the kernel's A and B
    const uint8_t* sfb;
    int64_t kt;                  // scale tiles along k
    const uint16_t* bias;
    uint16_t* C;
    int64_t ldc;
    int64_t M, N;                // of the kernel's A and B rows
    int32_t k32;                 // 32-value MMA steps in all: ceil(k / 32)
    int32_t steps;               // 128-value slots in all
    int32_t stages, act, bf16;
    int32_t swapped;             // the kernel's A is the caller's B: C[n][m], bias along m
    int32_t bn;                  // rows of the kernel's B a tile takes
    int32_t early;               // the kernel before this one is the quantisation of the kernel's B
    uint32_t tmem_cols;
    int32_t test_stall;          // failure test: the MMA thread first waits on a barrier nothing arrives on
    uint64_t timeout_ns;
    int* status;
};

constexpr int kTileThreads = 192;   // warps 0-3 epilogue, 4 loads, 5 MMA
constexpr uint32_t kABytes = 128 * 128;

__host__ __device__ inline uint32_t tile_stage_bytes(int bn) { return kABytes + bn * 128 + 2 * kScaleTile; }

// The first `count` of 16 finished sums of row m, columns n on, to C.
__device__ __forceinline__ void store16(const TileParams& p, int64_t m, int64_t n, int count, float* v)
{
    if (m >= p.M) return;
    if (p.swapped) {   // lanes hold neighbouring columns of C
        const float b = p.bias ? widen(p.bias[m], p.bf16) : 0.f;
        uint16_t* c = p.C + m;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < count && n + i < p.N) c[(n + i) * p.ldc] = narrow(act_f32(p.act, v[i] + b), p.bf16);
        return;
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (n + i < p.N) v[i] += widen(p.bias[n + i], p.bf16);
    }
    if (p.act) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = act_f32(p.act, v[i]);
    }
    uint16_t* c = p.C + m * p.ldc + n;
    if (count == 16 && n + 16 <= p.N && reinterpret_cast<uintptr_t>(c) % 16 == 0) {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = narrow2(v[2 * i], v[2 * i + 1], p.bf16);
        reinterpret_cast<uint4*>(c)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4*>(c)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < count && n + i < p.N) c[i] = narrow(v[i], p.bf16);
    }
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// One 128 x bn tile a cluster, its K slots dealt to the cluster's CTAs in
// contiguous parts; with more than one CTA the parts are summed by rank over
// distributed shared memory (a fixed order, no workspace and no atomics).
// Few rows stream the weights once: 16 x 16384 x 8192, 134 MB in 256 CTAs, takes 25.4 us
// with cold caches (5.3 TB/s), of which some 5 are the start, the first bytes' way from
// DRAM, the sum over two CTAs and the end; 16 x 8192 x 8192 15.1 us.
__global__ void __launch_bounds__(kTileThreads) gemm_fp8_tile(const __grid_constant__ TileParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * 16 + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t bn = p.bn, sbytes = tile_stage_bytes(p.bn);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 16u * s; };
    auto empty = [&](int s) { return bar0 + 16u * s + 8u; };
    const uint32_t done = bar0 + 16u * 16u, never = done + 8u;

    uint32_t crank = 0, csize = 1;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(crank));
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const int64_t tile = blockIdx.x / csize;
    const int64_t tiles_m = (p.M + 127) >> 7;
    const int64_t m0 = (tile % tiles_m) * 128, n0 = (tile / tiles_m) * bn;
    const int s_lo = static_cast<int>(static_cast<int64_t>(p.steps) * crank / csize);
    const int s_hi = static_cast<int>(static_cast<int64_t>(p.steps) * (crank + 1) / csize);
    // a slot brings its scale tile where its block is the tile's first, or the part's
    auto brings = [&](int s) { return (s & 3) == 0 || s == s_lo; };

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full(s), 2);   // A's bytes and B's
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        mbar_init(never, 1);
        abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(&tmem_slot), p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    // After a quantisation of this call, which lets this kernel start only when
    // every kernel before it is done, A is there already: its first slots are
    // loaded while that kernel runs.  Everything else waits.
    if (warp != 4 || !p.early) griddep_wait();
    griddep_launch_dependents();

    const volatile int* abort = &abort_flag;
    auto fail = [&]() {
        abort_flag = 1;
        atomicExch(p.status, GEMM_F16_ERR_TIMEOUT);
    };
    if (warp == 4) {
        const bool issue = elect_one();
        int st = 0;
        uint32_t ph = 0;
        const uint8_t* sa = p.sfa + (m0 >> 7) * p.kt * kScaleTile;
        const uint8_t* sb = p.sfb + (n0 >> 7) * p.kt * kScaleTile;
        bool ok = true;
        int issued = 0;
        auto load_a = [&](int s, int at) {
            const uint32_t a = base + at * sbytes;
            mbar_arrive_expect_tx(full(at), kABytes + (brings(s) ? kScaleTile : 0));
            tma_load_2d(a, &p.tmA, s * 128, static_cast<int32_t>(m0), full(at));
            if (brings(s)) bulk_load(a + kABytes + bn * 128, sa + static_cast<int64_t>(s >> 2) * kScaleTile, kScaleTile, full(at));
        };
        auto load_b = [&](int s, int at) {
            const uint32_t b = base + at * sbytes + kABytes;
            mbar_arrive_expect_tx(full(at), bn * 128 + (brings(s) ? kScaleTile : 0));
            tma_load_2d(b, &p.tmB, s * 128, static_cast<int32_t>(n0), full(at));
            if (brings(s)) bulk_load(b + bn * 128 + kScaleTile, sb + static_cast<int64_t>(s >> 2) * kScaleTile, kScaleTile, full(at));
        };
        const int ahead = p.early ? min(p.stages, s_hi - s_lo) : 0;
        if (issue)
            for (int q = 0; q < ahead; ++q) load_a(s_lo + q, q);
        __syncwarp();
        if (p.early) griddep_wait();
        for (int s = s_lo; s < s_hi; ++s, ++issued) {
            ok = mbar_wait(empty(st), ph ^ 1u, abort, p.timeout_ns);
            if (!ok) break;
            if (issue) {
                if (issued >= ahead) load_a(s, st);
                load_b(s, st);
            }
            if (++st == p.stages) st = 0, ph ^= 1u;
        }
        if (!ok) {   // copies in flight land before the CTA leaves
            if (issue) fail();
            for (int q = 0; q < p.stages && q < issued; ++q)
                mbar_wait(full(q), ((issued - q + p.stages - 1) / p.stages - 1) & 1u, nullptr, kDrainNs);
        }
    } else if (warp == 5) {
        const bool issue = elect_one();
        int st = 0;
        uint32_t ph = 0;
        const uint32_t tsa = tmem + bn, tsb = tsa + 4;
        bool ok = !p.test_stall || mbar_wait(never, 0, abort, p.timeout_ns);
        for (int s = s_lo; s < s_hi && ok; ++s) {
            ok = mbar_wait(full(st), ph, abort, p.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = base + st * sbytes, b = a + kABytes, fa = b + bn * 128;
            const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(b, 16, 1024);
            const uint64_t dfa = scale_desc(fa);   // (16-byte units: 32 a tile)
            const uint32_t id = idesc_mxf8(128, bn, s & 3);
            if (issue) {
                const int n32 = min(4, p.k32 - 4 * s);
                if (brings(s)) {
                    tmem_copy_scales(tsa, dfa);
                    tmem_copy_scales(tsb, dfa + 32);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < n32) umma_mxf8(tmem, da + 2 * q, db + 2 * q, id, tsa, tsb, s > s_lo || q > 0);
                umma_commit(empty(st));
            }
            if (++st == p.stages) st = 0, ph ^= 1u;
        }
        if (issue) {
            umma_commit(done);
            if (!ok) fail();
        }
        if (!ok) mbar_wait(done, 0, nullptr, kDrainNs);
    } else {
        // (a warp's lanes read tensor memory together or not at all)
        const bool ok = __all_sync(~0u, mbar_wait(done, 0, abort, p.timeout_ns));
        if (!ok) fail();
        tc_fence_after();
        const int64_t m = m0 + warp * 32 + lane;
        const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        for (uint32_t c = 0; ok && c < bn; c += 16) {
            uint32_t r[16];
            tmem_ld_x16(trow + c, r);
            tmem_wait_ld();
            if (csize == 1) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
                store16(p, m, n0 + c, 16, v);
            } else {
                // this CTA's part, column by column (lanes hold rows: consecutive words),
                // where the drained pipeline slots were
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + ((c + i) * 128 + warp * 32 + lane) * 4), "r"(r[i])
                                 : "memory");
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (csize > 1) {
        __syncwarp();
        cluster_sync_all();
        // each CTA finishes a share of the tile's columns, 16 at a time at most
        const bool bad = abort_flag != 0;
        if (warp < 4 && !bad) {
            const uint32_t c_lo = bn * crank / csize, c_hi = bn * (crank + 1) / csize;
            for (uint32_t c = c_lo; c < c_hi; c += 16) {
                const uint32_t count = min(16u, c_hi - c);
                float v[16] = {};
#pragma unroll 2
                for (uint32_t q = 0; q < csize; ++q) {
                    const uint32_t at = mapa_shared(base + (c * 128 + warp * 32 + lane) * 4, q);
                    float t[16];
#pragma unroll
                    for (uint32_t i = 0; i < 16; ++i) t[i] = i < count ? ld_cluster_f32(at + i * 512) : 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] += t[i];
                }
                store16(p, m0 + warp * 32 + lane, n0 + c, count, v);
            }
        }
        __syncwarp();
        cluster_sync_all();   // no CTA leaves while its part is being read
    }
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem, p.tmem_cols);
}

// ------------------------------------------------------------------ pairs
// Persistent clusters of two CTAs, one tile at a time, its MMAs over both
// (cta_group::2).  The weights' rows take the 256 lanes and A's rows the columns, in
// every product: a tile's columns are then as many as its rows need (32 to 256, a
// number in the instruction descriptor), so that one kernel serves groups of any
// number of rows, which the host does not know.
//
// Tiles: each group's rows are cut into equal parts of at most W, a multiple of 32;
// every CTA finds the W of least cost for itself from the row counts (choose_tiles).
// A tile ends with its group; it may read rows of the next one, whose columns it
// then leaves out.  A's scales begin at any row, so warps put their words in the
// order of the scale tiles as they load them, one set for 512 values of k.
//
// Up to 224 columns two accumulators and the scales fit tensor memory (512 columns), and a
// tile's MMAs follow the last one's without a pause.  Tiles of 256 columns have one, which
// the epilogue reads before the next tile's MMAs begin.
//
// Large products are bound by the SM's 64 bytes a cycle of operands, close before the MMAs
// (tensor pipe 85 % active), and in long runs by the power limit (1390 MHz at 1.38 kW): 131072 x
// 2048 x 7168 takes 1050 to 1060 us in short runs (3.6 PFLOP/s), 1190 to 1250 in long ones (3.1
// to 3.2), by the device; 131072 x 7168 x 2048 in 8 groups 1170 and 1325 to 1375; 8192^3 308 and
// 350; gate/up of 65536 rows, 8 groups of 2048 x 7168, 1050.  Few rows a group stream the
// weights: 512 rows, 64 groups of twice 2048 x 7168, 280 us (6.6 TB/s).  Small K is the
// epilogue's: 131072 x 7168 x 512 410 to 416 us.  A in 16 bits is quantised before the product
// begins: 131072 x 2048 x 7168 1515 and 1580 us, 131072 x 7168 x 2048 in 8 groups 1305 and 1460.
//
// Gate/up (kGated): the 256 lanes hold 128 rows of either weight, 16 of one and 16 of
// the other by turns, so that a thread of the epilogue holds both values of an output.
constexpr int kMaxStages = 10, kSets = 4, kMaxGroups = 512;
constexpr int kPairThreads = 320 + 32 * kSets;   // warps 0-7 epilogue, 8 loads, 9 MMA, the others scales
constexpr uint32_t kSlotBytes = 6 * (kABytes + 64 * 224), kSetBytes = 3 * kScaleTile, kBoxBytes = 32 * 64;   // kSlotBytes: all stages
constexpr uint32_t kPairSmem = kSlotBytes + 16 * kBoxBytes + kSets * kSetBytes + 1024;
constexpr int kMaxWidth = 256, kTwoWidth = 224; // columns of a tile; of one that has two accumulators
constexpr uint32_t kSfCol = 496, kAcc1 = 256;   // scales of the weights (4), of A (8); the second accumulator

struct PairParams {
    CUtensorMap tmW, tmU;        // weight codes {pitch, n, groups}, boxes of 128 bytes x 128 rows (kGated: 16)
    CUtensorMap tmX[8];          // A's codes {pitch, rows}, boxes of 128 bytes x 16, 32, .. 128 rows (one group: of its width's)
    CUtensorMap tmC;             // boxes of a warp's columns x 32 rows (c_unit 16)
    const uint8_t* sw;           // scale tiles of the weights, of the second ones, and of A
    const uint8_t* su;
    const uint8_t* sx;
    int64_t kt, w_tiles, x_tiles;   // scale tiles along k, along a weight's rows, along A's rows
    const int32_t* group_rows;   // on the device; null: one group of all rows
    const uint16_t* bias;
    uint16_t* C;
    int64_t ldc, rows, n;
    int32_t groups, tiles_w, panel;   // panel: weight tiles walked together
    int32_t width;               // W; 0: of the groups' choice
    int32_t k32, steps, act, bf16, c_unit;   // c_unit: bytes that C's rows, their pitch and C are multiples of, at most 16
    int32_t test_stall;
    uint64_t timeout_ns;
    int* status;
};

// Row ranges of the groups and their tiles, in shared memory.
struct Groups {
    int row0[kMaxGroups + 1];    // rows past the last group's end belong to none
    int tile0[kMaxGroups + 1];   // tiles before the group: its parts x tiles_w
    int parts[kMaxGroups];       // of its rows
    uint16_t width[kMaxGroups];  // columns of each part, at most
    int widest;                  // of all groups
};

// By one warp.  Counts below zero are taken as zero, rows past the matrix as absent.
__device__ __forceinline__ void choose_tiles(const PairParams& p, Groups& g, int clusters, int lane)
{
    if (!p.group_rows) {
        if (lane == 0) {
            const int rows = static_cast<int>(p.rows);
            g.row0[0] = g.tile0[0] = 0, g.row0[1] = rows;
            g.parts[0] = parts_of(rows, p.width), g.tile0[1] = g.parts[0] * p.tiles_w;
            g.width[0] = static_cast<uint16_t>(g.widest = p.width);
        }
        return;
    }
    int64_t before = 0;
    for (int i = lane; i - lane < p.groups; i += 32) {
        int64_t n = i >= p.groups ? 0 : max(0, p.group_rows[i]), sum = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int64_t up = __shfl_up_sync(~0u, sum, d);
            if (lane >= d) sum += up;
        }
        if (i < p.groups) g.row0[i] = static_cast<int>(min(before + sum - n, p.rows));
        before += __shfl_sync(~0u, sum, 31);
    }
    if (lane == 0) g.row0[p.groups] = static_cast<int>(min(before, p.rows));
    __syncwarp();
    // a lane in four takes a width and a quarter of the groups
    const int w = 32 * ((lane & 7) + 1);
    int tiles = 0, widest = 0;
    for (int i = lane >> 3; i < p.groups; i += 4) {
        const int r = g.row0[i + 1] - g.row0[i], parts = parts_of(r, w);
        tiles += parts;
        widest = max(widest, width_of(r, parts));
    }
#pragma unroll
    for (int d = 8; d < 32; d *= 2) {
        tiles += __shfl_xor_sync(~0u, tiles, d);
        widest = max(widest, __shfl_xor_sync(~0u, widest, d));
    }
    int64_t cost = cost_of(tiles * p.tiles_w, widest, clusters, p.steps) * 16 + (7 - (lane & 7));
#pragma unroll
    for (int d = 1; d < 8; d *= 2) cost = min(cost, __shfl_xor_sync(~0u, cost, d));
    const int width = p.width ? p.width : 32 * (8 - static_cast<int>(cost & 15));
    int at = 0;
    widest = 0;
    for (int i = lane; i - lane < p.groups; i += 32) {
        int n = 0;
        if (i < p.groups) {
            const int rows = g.row0[i + 1] - g.row0[i], parts = parts_of(rows, width), w = width_of(rows, parts);
            g.parts[i] = parts;
            g.width[i] = static_cast<uint16_t>(w);
            widest = max(widest, w);
            n = parts * p.tiles_w;
        }
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(~0u, sum, d);
            if (lane >= d) sum += up;
        }
        if (i < p.groups) g.tile0[i] = at + sum - n;
        at += __shfl_sync(~0u, sum, 31);
    }
    widest = __reduce_max_sync(~0u, widest);
    if (lane == 0) g.tile0[p.groups] = at, g.widest = max(widest, 32);
}

// Loads that are issued where they stand (the plain ones may be moved down to the use of
// their values, past the waits between).
__device__ __forceinline__ uint4 ld_now_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_now_u32(const void* p)
{
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// The pair's instructions for the lane that `on` is set in.  A predicate instead of a
// branch: in a branch that not all lanes take every operand is moved to a uniform register
// for each instruction, 60 cycles and more, and a step's six instructions and waits took
// 660 cycles whatever the tile's width.
__device__ __forceinline__ void umma_mxf8_pair_if(uint32_t on, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                                  uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(on)
        : "memory");
}

__device__ __forceinline__ void tmem_copy_scales_pair_if(uint32_t on, uint32_t taddr, uint64_t desc)
{
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
                 "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc), "r"(on)
                 : "memory");
}

__device__ __forceinline__ void umma_commit_pair_mc_if(uint32_t on, uint32_t bar, uint16_t cta_mask)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            bar),
        "h"(cta_mask), "r"(on)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d_if(uint32_t on, const void* tmap, uint32_t src, int32_t x, int32_t y, uint64_t policy)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], %4;\n\t"
        "@q cp.async.bulk.commit_group;\n\t}" ::"l"(reinterpret_cast<uint64_t>(tmap)),
        "r"(x), "r"(y), "r"(src), "l"(policy), "r"(on)
        : "memory");
}

// Whether the phase with the given parity is over, without waiting.
__device__ __forceinline__ uint32_t mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok;
}

struct Tile {
    int group, row, width, rows, w;   // A's first row, the columns, those that are the group's; weight tile
};

// The last group that begins at tile t or before (an empty one has no tile).
__device__ __forceinline__ int group_of(const PairParams& p, const Groups& g, int t)
{
    int lo = 0, hi = p.groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.tile0[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Inside a group: bands of `panel` weight tiles, in a band one part of the rows
// after the other, so that the clusters at work share both operands in L2.
__device__ __forceinline__ Tile place(const PairParams& p, const Groups& g, int t)
{
    Tile o;
    o.group = group_of(p, g, t);
    const int r0 = g.row0[o.group], rows = g.row0[o.group + 1] - r0, all = p.panel * g.parts[o.group];
    const int i = t - g.tile0[o.group], band = i < all ? 0 : i / all, j = i - band * all;
    const int in_band = min(p.panel, p.tiles_w - band * p.panel), part = j / in_band;
    o.w = band * p.panel + (j - part * in_band);
    o.width = g.width[o.group];
    o.row = r0 + part * o.width;
    o.rows = min(o.width, rows - part * o.width);
    return o;
}

// 16 lanes x 32 columns: of 8 columns each, registers 0 and 1 hold row lane / 4, columns
// 2 (lane % 4) and the next, registers 2 and 3 the row 8 further.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, float* r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
          "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
        : "r"(taddr)
        : "memory");
}

// Four 8 x 8 matrices of 16-bit values, each stored transposed: lane 8 i + j gives the
// address of row j of matrix i.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

__device__ __forceinline__ void ld_smem(uint32_t addr, uint4* v)
{
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v->x), "=r"(v->y), "=r"(v->z), "=r"(v->w) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld_smem(uint32_t addr, uint2* v)
{
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v->x), "=r"(v->y) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ld_smem(uint32_t addr, uint32_t* v) { asm volatile("ld.shared.u32 %0, [%1];" : "=r"(*v) : "r"(addr) : "memory"); }
__device__ __forceinline__ void ld_smem(uint32_t addr, uint16_t* v) { asm volatile("ld.shared.u16 %0, [%1];" : "=h"(*v) : "r"(addr) : "memory"); }

template <bool kGated>
__global__ void __launch_bounds__(kPairThreads, 1) gemm_fp8_pair(const __grid_constant__ PairParams p)
{
    constexpr int kRows = kGated ? 64 : 128;        // of a weight, a CTA and a tile
    constexpr int kN = kGated ? 16 : 32;            // columns of C a warp holds
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2 * kSets + 6];
    __shared__ Groups groups;
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 16u * s; };
    auto empty = [&](int s) { return bar0 + 16u * s + 8u; };
    auto sfull = [&](int s) { return bar0 + 16u * (kMaxStages + s); };
    auto sempty = [&](int s) { return bar0 + 16u * (kMaxStages + s) + 8u; };
    const uint32_t tfull = bar0 + 16u * (kMaxStages + kSets), tempty = tfull + 16u, never = tempty + 16u, drain = never + 8u;
    const uint32_t boxes = base + kSlotBytes, sets = boxes + 16 * kBoxBytes;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int s = 0; s < kSets; ++s) {
            mbar_init(sfull(s), 2);   // the scale warps of both CTAs
            mbar_init(sempty(s), 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull + 8 * a, 1);
            mbar_init(tempty + 8 * a, 16);   // every epilogue warp of both CTAs
        }
        mbar_init(never, 1);
        mbar_init(drain, 1);
        abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&p.tmW);
        if (kGated) tma_prefetch_desc(&p.tmU);
        if (p.c_unit == 16) tma_prefetch_desc(&p.tmC);
    }
    if (warp == 9) {
        tmem_alloc_pair(smem_u32(&tmem_slot), 512);
        tmem_relinquish_pair();
    }
    griddep_wait();
    const int clusters = gridDim.x >> 1;
    if (warp == 0) choose_tiles(p, groups, clusters, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    griddep_launch_dependents();   // (this CTA has its tensor memory)
    const uint32_t tmem = tmem_slot;
    const int tiles = __shfl_sync(~0u, groups.tile0[p.groups], 0);
    // as many stages as fit: a tile of few columns brings little for its 16 KB of weights
    const uint32_t stage_bytes = kABytes + __shfl_sync(~0u, groups.widest, 0) * 64u;
    const int stages = static_cast<int>(min(kSlotBytes / stage_bytes, static_cast<uint32_t>(kMaxStages)));
    const bool two = stage_bytes <= kABytes + kTwoWidth * 64u;   // accumulators

    const volatile int* abort = &abort_flag;
    auto fail = [&]() {
        abort_flag = 1;
        atomicExch(p.status, GEMM_F16_ERR_TIMEOUT);
    };

    if (warp == 8) {
        const bool issue = elect_one();
        int st = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int t = blockIdx.x >> 1; t < tiles && ok; t += clusters) {
            const Tile o = place(p, groups, t);
            const int half = o.width >> 1, box = (o.width >> 5) - 1;
            const uint32_t xbytes = 128u * half;
            const int32_t wn = (o.w * 2 + static_cast<int>(rank)) * kRows, xr = o.row + static_cast<int>(rank) * half;
            for (int s = 0; s < p.steps; ++s) {
                ok = mbar_wait_cluster(empty(st), par ^ 1u, abort, p.timeout_ns);
                if (!ok) break;
                const uint32_t a = base + st * stage_bytes;
                const uint32_t bar = mapa_shared(full(st), 0);
                if (issue) {
                    if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * (kABytes + xbytes));
                    if (kGated) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            tma_load_3d_pair(a + j * 4096, &p.tmW, s * 128, wn + 16 * j, o.group, bar);
                            tma_load_3d_pair(a + j * 4096 + 2048, &p.tmU, s * 128, wn + 16 * j, o.group, bar);
                        }
                    } else {
                        tma_load_3d_pair(a, &p.tmW, s * 128, wn, o.group, bar);
                    }
                    tma_load_2d_pair(a + kABytes, &p.tmX[box], s * 128, xr, bar);
                }
                if (++st == stages) st = 0, par ^= 1u;
            }
        }
        if (!ok && issue) {   // copies in flight land before the pair leaves: far longer than any takes
            fail();
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 5000000ull) __nanosleep(100000);
        }
    } else if (warp >= 10) {
        // A warp for each of the kSets sets in shared memory: the fence that hands a set over
        // waits for the loads under way, some 2500 cycles from DRAM, while a 256 x 256 tile
        // uses a set up in 2048.
        // 16 bytes a lane of each tile: the words of rows lane, lane + 32, + 64, + 96.
        const int st = warp - 10;
        uint32_t par = 0;
        bool ok = true;
        int q = st;
        for (int t = blockIdx.x >> 1; t < tiles && ok; t += clusters, q -= static_cast<int>(p.kt)) {
            if (q >= p.kt) continue;
            const Tile o = place(p, groups, t);
            const int wn = (o.w * 2 + static_cast<int>(rank)) * kRows, first = (o.row + lane) & 31;
            const int turn = ((o.row & 127) + lane) >> 5;   // words that the first tile's line lacks: 0 .. 4
            const int64_t matrix = static_cast<int64_t>(o.group) * p.w_tiles * p.kt * kScaleTile;
            for (; q < p.kt && ok; q += kSets) {
                const uint4 none = make_uint4(0u, 0u, 0u, 0u);
                auto line = [&](const uint8_t* scales, int64_t tile, int64_t count, int r) {
                    return tile < count ? ld_now_v4(scales + (tile * p.kt + q) * kScaleTile + r * 16) : none;
                };
                uint4 w, x[3];
                if (kGated) {
                    const uint8_t* from = (lane & 16 ? p.su : p.sw) + matrix;
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = wn + 16 * j + (lane & 15);
                        v[j] = r < p.n ? ld_now_u32(from + scale_at(r, 4 * q, p.kt)) : 0u;
                    }
                    w = make_uint4(v[0], v[1], v[2], v[3]);
                } else {
                    w = line(p.sw + matrix, wn >> 7, p.w_tiles, lane);
                }
#pragma unroll
                for (int h = 0; h < 3; ++h)   // (a tile further is the next one's same line)
                    x[h] = h == 0 || o.width > 128 * (h - 1) ? line(p.sx, (o.row >> 7) + h, p.x_tiles, first) : none;
                ok = __all_sync(~0u, mbar_wait_cluster(sempty(st), par ^ 1u, abort, p.timeout_ns));
                if (!ok) break;
                par ^= 1u;
                const uint32_t at = sets + st * kSetBytes + lane * 16;
                st_smem_v4(at, w);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint4 a = x[h], b = x[h + 1];
                    const uint32_t c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                    uint32_t v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = turn == 0 ? c[j] : turn == 1 ? c[j + 1] : turn == 2 ? c[j + 2] : turn == 3 ? c[j + 3] : c[j + 4];
                    st_smem_v4(at + (h + 1) * kScaleTile, make_uint4(v[0], v[1], v[2], v[3]));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(mapa_shared(sfull(st), 0));
            }
        }
        if (!ok && lane == 0) fail();
    } else if (warp == 9) {
        if (rank == 0) {
            const uint32_t issue = elect_one();
            int st = 0, acc = 0, set = 0, t = blockIdx.x >> 1;
            uint32_t par = 0, spar = 0, tpar = 0;
            bool ok = !p.test_stall || mbar_wait(never, 0, abort, p.timeout_ns);
            const uint32_t tsw = tmem + kSfCol, tsx = tsw + 4, step16 = stage_bytes >> 4;
            const uint64_t desc0 = umma_desc_sw128(base, 16, 1024), sets0 = scale_desc(sets);   // (in 16-byte units)
            auto width_at = [&](int u) {
                return u < tiles ? __shfl_sync(~0u, static_cast<int>(groups.width[group_of(p, groups, u)]), 0) : 0;
            };
            int width = width_at(t);
            // waits for the operands at hand, for their scales and for an accumulator that has been read
            auto ready = [&](bool scales, bool room) {
                return __all_sync(~0u, (!room || mbar_wait_cluster(tempty + 8 * acc, tpar ^ 1u, abort, p.timeout_ns)) &&
                                           (!scales || mbar_wait_cluster(sfull(set), spar, abort, p.timeout_ns)) &&
                                           mbar_wait_cluster(full(st), par, abort, p.timeout_ns)) != 0;
            };
            if (ok && t < tiles) ok = ready(true, true);
            while (ok && t < tiles) {
                const uint32_t d = tmem + (acc ? kAcc1 : 0u), id0 = idesc_mxf8(256, width, 0), over = tfull + 8 * acc;
                const int next_width = width_at(t + clusters);
                // one slot, the `byte`-th of its set; n32 instructions
                auto step = [&](int s, int byte, int n32) {
                    tc_fence_after();
                    const uint64_t da = desc0 + st * step16, db = da + (kABytes >> 4);
                    const uint32_t id = id0 | idesc_mxf8(0, 0, byte), done = empty(st);
                    const bool last = s + 1 == p.steps, fresh = last || byte == 3;
                    if (byte == 0) {
                        const uint64_t df = sets0 + set * (kSetBytes >> 4);
                        tmem_copy_scales_pair_if(issue, tsw, df);
                        tmem_copy_scales_pair_if(issue, tsx, df + 32);
                        if (width > 128) tmem_copy_scales_pair_if(issue, tsx + 4, df + 64);
                        umma_commit_pair_mc_if(issue, sempty(set), 0x3);
                        if (++set == kSets) set = 0, spar ^= 1u;
                    }
                    if (++st == stages) st = 0, par ^= 1u;
                    // the next slot's barriers, asked here and looked at when this one's first
                    // instructions are out: an answer takes some 100 cycles
                    uint32_t there = mbar_test(full(st), par);
                    if (fresh) there &= mbar_test(sfull(set), spar);
                    if (last && two) there &= mbar_test(tempty + 8 * (acc ^ 1), tpar ^ 1u ^ acc);
                    auto mma = [&](int q) {
                        umma_mxf8_pair_if(n32 > q ? issue : 0u, d, da + 2 * q, db + 2 * q, id, tsw, tsx, s > 0 || q > 0);
                    };
                    mma(0), mma(1), mma(2);
                    // (what the next slot waits for hangs on earlier ones than this, and on the tile before)
                    if (last) {
                        t += clusters, width = next_width;
                        if (acc || !two) tpar ^= 1u;
                        if (two) acc ^= 1;
                    }
                    const bool one = last && !two;   // the accumulator's own tile has to end first
                    if (!one && !__all_sync(~0u, there) && t < tiles) ok = ready(fresh, last);
                    mma(3);
                    umma_commit_pair_mc_if(issue, done, 0x3);
                    if (last) umma_commit_pair_mc_if(issue, over, 0x3);
                    if (one && t < tiles) ok = ready(true, true);
                };
                int s = 0;
                for (; s + 4 <= p.steps - 1 && ok; s += 4) {   // whole sets
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        if (ok) step(s + b, b, 4);
                }
                for (; s < p.steps && ok; ++s) step(s, s & 3, min(4, p.k32 - 4 * s));
            }
            if (!ok) {
                if (issue) {
                    fail();
                    umma_commit_pair_mc(drain, 0x1);
                }
                mbar_wait_cluster(drain, 0, nullptr, kDrainNs);
            }
        }
    } else {
        // epilogue: 32 columns of the accumulator (rows of C) at a time, warps 0-3 the even
        // ones, 4-7 the odd ones; a warp's lanes are the weight rows 32 (warp % 4) on
        const int half = warp >> 2;
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t box0 = boxes + warp * 2 * kBoxBytes, leader_empty = mapa_shared(tempty, 0);
        const uint64_t policy = l2_policy(1);   // C first out of L2: the operands stay
        uint32_t turn = 0;
        int acc = 0;
        uint32_t tpar = 0;
        for (int t = blockIdx.x >> 1; t < tiles; t += clusters) {
            const Tile o = place(p, groups, t);
            const int64_t n0 = static_cast<int64_t>(o.w * 2 + static_cast<int>(rank)) * kRows + (warp & 3) * kN;
            uint16_t bias[4] = {};   // (as they are, so that nothing waits for them here)
            if (!kGated && p.bias) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t n = n0 + 8 * i + (lane >> 2);
                    if (n < p.n) bias[i] = ld_nc_u16(p.bias + n);
                }
            }
            const bool ok = __all_sync(~0u, mbar_wait_cluster(tfull + 8 * acc, tpar, abort, p.timeout_ns));
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            const uint32_t d = trow + (acc ? kAcc1 : 0u);
            const int chunks = o.width >> 5;
            auto load = [&](int b, float* v) {
                tmem_ld_16x256b_x4(d + b * 32, v);
                tmem_ld_16x256b_x4(d + b * 32 + (16u << 16), v + 16);
            };
            auto finish = [&](int b, float* v) {
                const int left = o.rows - b * 32;   // rows of C among the 32
                if (left <= 0 || n0 >= p.n) return;
                const uint32_t box = box0 + turn;
                if (kGated) {
                    act_all<16>(p.act, v);
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] *= v[16 + c];
                } else {
                    if (p.bias) {
                        float f[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = widen(bias[i], p.bf16);
#pragma unroll
                        for (int c = 0; c < 32; ++c) v[c] += f[2 * (c >> 4) + ((c >> 1) & 1)];
                    }
                    act_all(p.act, v);
                }
                // to the box as rows of C: row tok at tok * 2 kN, its 16-byte parts shifted as TMA's
                // swizzles have it, so that eight rows fall on different banks
                // (the last copy out of a box took the other one: this one's is the copy before)
                if (lane == 0) bulk_wait_group_read<1>();
                __syncwarp();
                auto part = [&](int tok, int c) {
                    return box + tok * (2 * kN) + ((c ^ (kGated ? (tok >> 2) & 1 : (tok >> 1) & 3)) << 4);
                };
#pragma unroll
                for (int c = 0; c < 4; c += kGated ? 2 : 1) {
                    auto two = [&](int k) { return narrow2(v[k], v[k + 1], p.bf16); };
                    if (kGated)   // two matrices of 8 rows, two of the next 8
                        stmatrix_x4_trans(part(8 * (c + (lane >> 4)) + (lane & 7), (lane >> 3) & 1), two(4 * c), two(4 * c + 2),
                                          two(4 * c + 4), two(4 * c + 6));
                    else
                        stmatrix_x4_trans(part(8 * c + (lane & 7), lane >> 3), two(4 * c), two(4 * c + 2), two(16 + 4 * c),
                                          two(16 + 4 * c + 2));
                }
                if (p.c_unit == 16 && left >= 32) {   // (TMA leaves out columns past C's, not rows past the group's)
                    fence_proxy_async_smem();
                    __syncwarp();
                    tma_store_2d_if(lane == 0, &p.tmC, box, static_cast<int32_t>(n0), o.row + b * 32, policy);
                    turn ^= kBoxBytes;
                    return;
                }
                __syncwarp();
                uint16_t* to = p.C + (static_cast<int64_t>(o.row) + b * 32) * p.ldc + n0;
                // by units of as many bytes as C's rows are multiples of, a row's after one another
                auto store = [&](auto unit) {
                    using U = decltype(unit);
                    constexpr int kParts = 2 * kN / sizeof(U), kPass = 32 / kParts, kRowsAtOnce = 8;
                    const int c = lane % kParts, byte = c * static_cast<int>(sizeof(U)), first = lane / kParts;
                    uint8_t* row = reinterpret_cast<uint8_t*>(to + first * p.ldc) + byte;
                    const int64_t step = 2 * kPass * p.ldc;
                    if (byte >= 2 * (p.n - n0)) return;
#pragma unroll
                    for (int r0 = 0; r0 < 32 / kPass; r0 += kRowsAtOnce) {
                        U x[kRowsAtOnce];
#pragma unroll
                        for (int r = r0; r < r0 + kRowsAtOnce && r < 32 / kPass; ++r) {
                            const int tok = r * kPass + first;
                            ld_smem(part(tok, byte >> 4) + (byte & 15), &x[r - r0]);
                        }
#pragma unroll
                        for (int r = r0; r < r0 + kRowsAtOnce && r < 32 / kPass; ++r, row += step)
                            if (r * kPass + first < left) *reinterpret_cast<U*>(row) = x[r - r0];
                    }
                };
                switch (p.c_unit) {
                case 16: store(uint4()); break;
                case 8: store(uint2()); break;
                case 4: store(uint32_t()); break;
                default: store(uint16_t()); break;
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int b = half; b < chunks; b += 4) {   // twice 32 columns for one wait
                float v[32], w[32];
                load(b, v);
                if (b + 2 < chunks) load(b + 2, w);
                tmem_wait_ld();
                if (b + 4 >= chunks) {   // the accumulator's columns are read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(leader_empty + 8 * acc);
                }
                finish(b, v);
                if (b + 2 < chunks) finish(b + 2, w);
            }
            if (half >= chunks && lane == 0) mbar_arrive_cluster_relaxed(leader_empty + 8 * acc);
            if (acc || !two) tpar ^= 1u;
            if (two) acc ^= 1;
        }
        if (lane == 0) bulk_wait_group_all();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 9) tmem_dealloc_pair(tmem, 512);
}

}  // namespace fp8_dev
