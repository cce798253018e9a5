// C[m, n] = act(sum_k A[m, k] B[n, k] + bias[n]) for two MXFP4 matrices.
//
// The tensor cores take e2m1 codes from shared memory and the blocks' scales
// from tensor memory (tcgen05.mma kind::mxf4, block_scale, 64 values of K an
// instruction): every product is exact, sums are fp32 in tensor memory, and
// nothing is dequantised on the way.  A row of a pipeline slot is 128 bytes =
// 256 values; its scales are two 512-byte tiles for each 128 rows, which
// tcgen05.cp copies to 4 columns of tensor memory each, repeated for the four
// lane quarters as the instruction wants them.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "gemm_f16.h"
#include "mxf4_ptx.cuh"
#include "ptx.cuh"

namespace mxf4_dev {

struct GemmParams {
    CUtensorMap tmA, tmB;        // codes: {16 * blocks bytes, rows}, box {128, 128 or bn}
    const uint8_t* sfa;          // scale tiles of the kernel's A and B
    const uint8_t* sfb;
    int64_t kt;                  // scale tiles along k
    const __half* bias;
    __half* C;
    int64_t ldc;
    int64_t M, N;                // of the kernel's A and B rows
    int32_t k64;                 // 64-value MMA steps in all: ceil(k / 64)
    int32_t steps;               // 256-value slots in all
    int32_t stages, act;
    int32_t swapped;             // the kernel's A is the caller's B: C[n][m], bias along m
    int32_t bn;                  // rows of the kernel's B a tile takes
    int32_t early;               // the kernel before this one is the quantisation of the kernel's B
    uint32_t tmem_cols;
    int32_t test_stall;          // failure test: the MMA thread first waits on a barrier nothing arrives on
    uint64_t timeout_ns;
    int* status;
};

constexpr int kGemmThreads = 192;   // warps 0-3 epilogue, 4 loads, 5 MMA
constexpr uint32_t kABytes = 128 * 128, kSfBytes = 2 * kScaleTile;

__host__ __device__ inline uint32_t gemm_stage_bytes(int bn) { return kABytes + bn * 128 + 2 * kSfBytes; }

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The activations without a branch, so that a thread's 32 values overlap, and of
// few instructions: with erfcf and the full division, whose rare cases branch, a
// SiLU took 220 cycles of a warp and the epilogue 9/10 of a product with K = 1000.
//
// Phi(x) for x < 0 is erfc(z) / 2 with z = -x / sqrt 2, and erfc(z) exp(z^2) is
// smooth and falls like 1 / z: t P(t) with t = 1 / (1 + z / 3) and P of degree 7,
// least relative error over 0 <= z <= 9 (fitted to the function's values in 64
// bits; gelu_factor gives half of P's), is within 1.3e-7 of it.  With the
// rounding of z^2 and the approximate exponential the whole is within 2^-18 of x
// Phi(x) wherever that is not zero in fp16.
__device__ constexpr float gelu_factor(int i)
{
    constexpr float f[8] = {0.0940747783f, 0.0931263119f, 0.0966875404f, 0.0410582423f,
                            0.168501928f,  -0.131988719f, 0.200961143f,  -0.0624212809f};
    return f[i];
}

__device__ __forceinline__ float act_f32(int act, float x)
{
    switch (act) {
    case 1: return x < 0.f ? 0.f : x;
    case 2: return x * rcp(1.f + ex2(-1.44269504f * x));
    case 3: {
        const float t = rcp(fmaf(fabsf(x), 0.70710678f / 3.f, 1.f));
        float q = gelu_factor(7);
#pragma unroll
        for (int i = 6; i >= 0; --i) q = fmaf(q, t, gelu_factor(i));
        const float h = q * t * ex2(x * x * (-0.5f * 1.44269504f));
        return x * (x < 0.f ? h : 1.f - h);
    }
    default: return x;
    }
}

// Sum over the cluster's parts of one output's K range, by distributed shared
// memory: `at` is the same offset in every CTA.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The first `count` of 16 finished sums of row m, columns n on, to C.
__device__ __forceinline__ void store16(const GemmParams& p, int64_t m, int64_t n, int count, float* v)
{
    if (m >= p.M) return;
    if (p.swapped) {   // lanes hold neighbouring columns of C
        const float b = p.bias ? __half2float(p.bias[m]) : 0.f;
        __half* c = p.C + m;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < count && n + i < p.N) c[(n + i) * p.ldc] = __float2half_rn(act_f32(p.act, v[i] + b));
        return;
    }
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (n + i < p.N) v[i] += __half2float(p.bias[n + i]);
    }
    if (p.act) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = act_f32(p.act, v[i]);
    }
    __half* c = p.C + m * p.ldc + n;
    if (count == 16 && n + 16 <= p.N && reinterpret_cast<uintptr_t>(c) % 16 == 0) {
        uint4 o[2];
        o[0] = make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
        o[1] = make_uint4(pack_half2(v[8], v[9]), pack_half2(v[10], v[11]), pack_half2(v[12], v[13]),
                          pack_half2(v[14], v[15]));
        reinterpret_cast<uint4*>(c)[0] = o[0];
        reinterpret_cast<uint4*>(c)[1] = o[1];
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < count && n + i < p.N) c[i] = __float2half_rn(v[i]);
    }
}

// One 128 x bn tile a cluster, its K slots dealt to the cluster's CTAs in
// contiguous parts; with more than one CTA the parts are summed by rank over
// distributed shared memory (a fixed order, no workspace and no atomics).
// Bound by the length of one cold chain: 16 x 16384 x 8192, 71 MB of weights
// in 256 CTAs of 16 steps, takes 15.8 us with cold caches (4.5 TB/s), 9.9 us with
// the weights in L2.
__global__ void __launch_bounds__(kGemmThreads) gemm_mxf4_tile(const __grid_constant__ GemmParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * 16 + 2];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t bn = p.bn, sbytes = gemm_stage_bytes(p.bn);
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
        // (an odd last scale tile: the second one is not this row tile's)
        auto sf_bytes = [&](int s) { return static_cast<uint32_t>(min(static_cast<int64_t>(2), p.kt - 2 * s)) * kScaleTile; };
        auto load_a = [&](int s, int at) {
            const uint32_t a = base + at * sbytes, sf = sf_bytes(s);
            mbar_arrive_expect_tx(full(at), kABytes + sf);
            tma_load_2d(a, &p.tmA, s * 128, static_cast<int32_t>(m0), full(at));
            bulk_load(a + kABytes + bn * 128, sa + static_cast<int64_t>(s) * kSfBytes, sf, full(at));
        };
        auto load_b = [&](int s, int at) {
            const uint32_t b = base + at * sbytes + kABytes, sf = sf_bytes(s);
            mbar_arrive_expect_tx(full(at), bn * 128 + sf);
            tma_load_2d(b, &p.tmB, s * 128, static_cast<int32_t>(n0), full(at));
            bulk_load(b + bn * 128 + kSfBytes, sb + static_cast<int64_t>(s) * kSfBytes, sf, full(at));
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
        const uint32_t tsa = tmem + bn, tsb = tsa + 8;
        const uint32_t id0 = idesc_mxf4(128, bn, 0), id1 = idesc_mxf4(128, bn, 1);
        bool ok = !p.test_stall || mbar_wait(never, 0, abort, p.timeout_ns);
        for (int s = s_lo; s < s_hi && ok; ++s) {
            ok = mbar_wait(full(st), ph, abort, p.timeout_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = base + st * sbytes, b = a + kABytes, fa = b + bn * 128, fb = fa + kSfBytes;
            const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(b, 16, 1024);
            const uint64_t dfa = scale_desc(fa), dfb = scale_desc(fb);   // (16-byte units: 32 a tile)
            if (issue) {
                const int n64 = min(4, p.k64 - 4 * s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (2 * h >= n64) break;
                    tmem_copy_scales(tsa + 4 * h, dfa + 32 * h);
                    tmem_copy_scales(tsb + 4 * h, dfb + 32 * h);
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < n64)
                        umma_mxf4(tmem, da + 2 * q, db + 2 * q, q & 1 ? id1 : id0, tsa + 4 * (q >> 1), tsb + 4 * (q >> 1),
                                  s > s_lo || q > 0);
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
        if (csize == 1) {
            for (uint32_t c = 0; ok && c < bn; c += 16) {
                uint32_t r[16];
                tmem_ld_x16(trow + c, r);
                tmem_wait_ld();
                float v[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
                store16(p, m, n0 + c, 16, v);
            }
        } else if (ok) {
            // this CTA's part, column by column (lanes hold rows: consecutive words),
            // where the drained pipeline slots were
            for (uint32_t c = 0; c < bn; c += 16) {
                uint32_t r[16];
                tmem_ld_x16(trow + c, r);
                tmem_wait_ld();
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
// The form for products of many tiles: persistent clusters of two CTAs, a 256 x
// kBN tile each, its MMAs over both (cta_group::2), so that each CTA brings half
// of B's rows.  L2 is what bounds it otherwise: an MMA step of 256 values takes
// 512 cycles and a CTA then reads 35 KB for it, 70 bytes a cycle, where a CTA
// alone with a 128 x 256 tile would read 100.
//
// Two accumulators of 256 columns and the scales do not fit tensor memory (512
// columns), so the second begins 24 columns inside the first: a tile's MMAs
// begin when the epilogue of the one before has those columns in registers,
// which it reads first: 1 200 cycles from a tile's last MMA to the next one's first.
//
// 131072 x 2048 x 7168: 496 us in short runs (7.8 PFLOP/s), 557 to 576 us in long ones;
// 8192^3 152 us, 7.2; 4096^3 27 us, the last of its 4 turns a third full.  8192 x 8192 x
// 1024 with bias and GELU: 70 us, the epilogue's (33 us without).
struct PairParams {
    CUtensorMap tmA, tmB;        // codes, boxes of 128 bytes x 128 rows and x kBN / 2 rows
    CUtensorMap tmSA, tmSB;      // scale tiles: {128 words, tiles}, boxes of two tiles
    CUtensorMap tmC;             // boxes of 64 columns x 32 rows (c_tma)
    const __half* bias;
    __half* C;
    int64_t ldc, M, N;
    int32_t kt, k64, steps, act, c_tma;
    int32_t tiles_m, tiles_n, panel;   // panel: rows of tiles walked column by column
    int32_t test_stall;
    uint64_t timeout_ns;
    int* status;
};

constexpr int kPairThreads = 320;   // warps 0-7 epilogue, 8 loads, 9 MMA
constexpr int kEpiBox = 32 * 128;   // bytes of a warp's staged 32 rows x 64 columns

template <int kBN>
struct PairShape {
    static constexpr uint32_t kB = kBN / 2 * 128, kSfB = kBN / 128 * kSfBytes;
    static constexpr uint32_t kStage = kABytes + kB + kSfBytes + kSfB;
    static constexpr int kStages = kBN == 256 ? 5 : 7;
    static constexpr uint32_t kSmem = kStages * kStage + 8 * kEpiBox + 1024;
    static constexpr uint32_t kSfCol = 512 - 8 - 2 * kBN / 32;    // scales of A, then of B
    static constexpr uint32_t kAcc1 = kBN == 256 ? kSfCol - 256 : 256;
};

// Two fp32 values an instruction.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}

__device__ __forceinline__ void unpack2(uint64_t v, float* a, float* b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}

// act_f32's GELU of two values.
__device__ __forceinline__ void gelu2(float* x0, float* x1)
{
    const uint64_t x = pack2(*x0, *x1), one = pack2(1.f, 1.f);
    auto both = [](float c) { return pack2(c, c); };
    float a, b;
    unpack2(fma2(pack2(fabsf(*x0), fabsf(*x1)), both(0.70710678f / 3.f), one), &a, &b);
    const uint64_t t = pack2(rcp(a), rcp(b));
    uint64_t q = both(gelu_factor(7));
#pragma unroll
    for (int i = 6; i >= 0; --i) q = fma2(q, t, both(gelu_factor(i)));
    unpack2(mul2(mul2(x, x), both(-0.5f * 1.44269504f)), &a, &b);
    const uint64_t h = mul2(mul2(q, t), pack2(ex2(a), ex2(b))), r = fma2(h, both(-1.f), one);
    float h0, h1, r0, r1;
    unpack2(h, &h0, &h1);
    unpack2(r, &r0, &r1);
    unpack2(mul2(x, pack2(*x0 < 0.f ? h0 : r0, *x1 < 0.f ? h1 : r1)), x0, x1);
}

// act of 32 values; one choice for all of them.
__device__ __forceinline__ void act_all(int act, float* v)
{
    if (act == 1) {
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = act_f32(1, v[c]);
    } else if (act == 2) {
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = act_f32(2, v[c]);
    } else if (act == 3) {
#pragma unroll
        for (int c = 0; c < 32; c += 2) gelu2(&v[c], &v[c + 1]);
    }
}

// 64 finished columns of a warp's 32 rows from its staging box to C, where its
// rows do not begin on 16 bytes: eight lanes a row, 16 aligned bytes of C each,
// shifted into place from two chunks of the box.  Of a row that begins off values
// past a boundary the last lane has the last off values and the first 8 - off.
__device__ __forceinline__ void store_rows(const PairParams& p, uint32_t box, int64_t m0, int64_t n0, int lane)
{
    if (n0 >= p.N || m0 >= p.M) return;
    const int cols = static_cast<int>(min(static_cast<int64_t>(64), p.N - n0));
    const int rows = static_cast<int>(min(static_cast<int64_t>(32), p.M - m0));
    uint16_t* c = reinterpret_cast<uint16_t*>(p.C + (m0 + (lane >> 3)) * p.ldc + n0);
#pragma unroll 4
    for (int r = lane >> 3; r < 32; r += 4, c += 4 * p.ldc) {
        const int off = static_cast<int>(reinterpret_cast<uintptr_t>(c) >> 1) & 7, i0 = 8 * (lane & 7) + (-off & 7);
        uint32_t in[8], out[4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(in[4 * h]), "=r"(in[4 * h + 1]), "=r"(in[4 * h + 2]), "=r"(in[4 * h + 3])
                         : "r"(box + r * 128 + (((((i0 >> 3) + h) ^ r) & 7) << 4)) : "memory");
        funnel16(in, 2 * (i0 & 7), out);
        if (r >= rows) continue;
        if (i0 + 8 <= cols) {
            *reinterpret_cast<uint4*>(c + i0) = make_uint4(out[0], out[1], out[2], out[3]);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int i = (i0 + 2 * t) & 63, j = (i + 1) & 63;
                if (j > i && j < cols) {
                    *reinterpret_cast<uint32_t*>(c + i) = out[t];
                } else {
                    if (i < cols) c[i] = static_cast<uint16_t>(out[t]);
                    if (j < cols) c[j] = static_cast<uint16_t>(out[t] >> 16);
                }
            }
        }
    }
}

template <int kBN>
__global__ void __launch_bounds__(kPairThreads, 1) gemm_mxf4_pair(const __grid_constant__ PairParams p)
{
    using S = PairShape<kBN>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    __shared__ __align__(8) uint64_t bars[2 * 8 + 5];
    __shared__ __align__(16) float bias[8][kBN / 2];   // of an epilogue warp's columns
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int abort_flag;

    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 16u * s; };
    auto empty = [&](int s) { return bar0 + 16u * s + 8u; };
    const uint32_t tfull = bar0 + 128u, room = tfull + 16u, never = room + 8u, drain = never + 8u;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(tfull, 1);
        mbar_init(tfull + 8, 1);
        mbar_init(room, 16);   // every epilogue warp of both CTAs
        mbar_init(never, 1);
        mbar_init(drain, 1);
        abort_flag = 0;
        fence_mbarrier_init();
        tma_prefetch_desc(&p.tmA);
        tma_prefetch_desc(&p.tmB);
        tma_prefetch_desc(&p.tmSA);
        tma_prefetch_desc(&p.tmSB);
        if (p.c_tma) tma_prefetch_desc(&p.tmC);
    }
    if (warp == 9) {
        tmem_alloc_pair(smem_u32(&tmem_slot), 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    griddep_wait();
    griddep_launch_dependents();

    const volatile int* abort = &abort_flag;
    auto fail = [&]() {
        abort_flag = 1;
        atomicExch(p.status, GEMM_F16_ERR_TIMEOUT);
    };
    const int clusters = gridDim.x >> 1;
    const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    auto place = [&](int64_t t, int64_t* m0, int64_t* n0) {
        const int64_t band = static_cast<int64_t>(p.panel) * p.tiles_n, b = t / band, r = t - b * band;
        const int64_t rows = min(static_cast<int64_t>(p.panel), p.tiles_m - b * p.panel);
        *n0 = r / rows * kBN;
        *m0 = (b * p.panel + r % rows) * 256;
    };

    if (warp == 8) {
        const bool issue = elect_one();
        int st = 0;
        uint32_t par = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x >> 1; t < tiles && ok; t += clusters) {
            int64_t m0, n0;
            place(t, &m0, &n0);
            const int32_t am = static_cast<int32_t>(m0 + rank * 128), bm = static_cast<int32_t>(n0 + rank * (kBN / 2));
            const int32_t sa = static_cast<int32_t>(am >> 7) * p.kt, sb = static_cast<int32_t>(n0 >> 7) * p.kt;
            for (int s = 0; s < p.steps; ++s) {
                ok = mbar_wait_cluster(empty(st), par ^ 1u, abort, p.timeout_ns);
                if (!ok) break;
                const uint32_t a = base + st * S::kStage, b = a + kABytes, fa = b + S::kB, fb = fa + kSfBytes;
                const uint32_t bar = mapa_shared(full(st), 0);
                if (issue) {
                    if (rank == 0) mbar_arrive_expect_tx(full(st), 2 * S::kStage);
                    tma_load_2d_pair(a, &p.tmA, s * 128, am, bar);
                    tma_load_2d_pair(b, &p.tmB, s * 128, bm, bar);
                    // (past a row tile's last scale tile: another's, or zeros; not used)
                    tma_load_2d_pair(fa, &p.tmSA, 0, sa + 2 * s, bar);
#pragma unroll
                    for (int h = 0; h < kBN / 128; ++h) tma_load_2d_pair(fb + h * kSfBytes, &p.tmSB, 0, sb + h * p.kt + 2 * s, bar);
                }
                if (++st == S::kStages) st = 0, par ^= 1u;
            }
        }
        if (!ok && issue) {   // copies in flight land before the pair leaves: far longer than any takes
            fail();
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 5000000ull) __nanosleep(100000);
        }
    } else if (warp == 9) {
        if (rank == 0) {
            const bool issue = elect_one();
            int st = 0, acc = 0;
            uint32_t par = 0, rpar = 0;
            bool ok = !p.test_stall || mbar_wait(never, 0, abort, p.timeout_ns);
            bool first = true;
            const uint32_t tsa = tmem + S::kSfCol, tsb = tsa + 8;
            const uint32_t id0 = idesc_mxf4(256, kBN, 0), id1 = idesc_mxf4(256, kBN, 1);
            for (int64_t t = blockIdx.x >> 1; t < tiles && ok; t += clusters) {
                if (!first) {   // the tile before last is stored, the last one's shared columns are read
                    ok = mbar_wait_cluster(room, rpar, abort, p.timeout_ns);
                    if (!ok) break;
                    rpar ^= 1u;
                }
                first = false;
                const uint32_t d = tmem + (acc ? S::kAcc1 : 0u);
                ok = mbar_wait_cluster(full(st), par, abort, p.timeout_ns);
                for (int s = 0; s < p.steps && ok; ++s) {
                    tc_fence_after();
                    const uint32_t a = base + st * S::kStage, b = a + kABytes, fa = b + S::kB, fb = fa + kSfBytes;
                    const uint64_t da = umma_desc_sw128(a, 16, 1024), db = umma_desc_sw128(b, 16, 1024);
                    const uint64_t dfa = scale_desc(fa), dfb = scale_desc(fb);   // (16-byte units: 32 a tile)
                    const uint32_t done = empty(st);
                    const int n64 = min(4, p.k64 - 4 * s);
                    auto mma = [&](int q) {
                        umma_mxf4_pair(d, da + 2 * q, db + 2 * q, q & 1 ? id1 : id0, tsa + 4 * (q >> 1),
                                       tsb + (kBN / 32) * (q >> 1), s > 0 || q > 0);
                    };
                    if (issue) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (2 * h >= n64) break;
                            tmem_copy_scales_pair(tsa + 4 * h, dfa + 32 * h);
#pragma unroll
                            for (int j = 0; j < kBN / 128; ++j)
                                tmem_copy_scales_pair(tsb + (kBN / 32) * h + 4 * j, dfb + 64 * j + 32 * h);
                        }
#pragma unroll
                        for (int q = 0; q < 3; ++q)
                            if (q < n64) mma(q);
                    }
                    // the next step's wait, some 100 cycles, while these run (the stage that it
                    // waits for was emptied by an earlier step than this one)
                    if (++st == S::kStages) st = 0, par ^= 1u;
                    if (s + 1 < p.steps) ok = mbar_wait_cluster(full(st), par, abort, p.timeout_ns);
                    if (issue) {
                        if (n64 == 4) mma(3);
                        umma_commit_pair_mc(done, 0x3);
                    }
                }
                if (!ok) break;
                if (issue) umma_commit_pair_mc(tfull + 8 * acc, 0x3);
                acc ^= 1;
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
        // epilogue: warps 0-3 the first half of the columns, 4-7 the second; a
        // warp's lanes are the rows 32 (warp % 4) .. of its CTA's 128
        constexpr int kHalf = kBN / 2, kBoxes = kHalf / 64;
        const int half = warp >> 2;
        const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * kHalf;
        const uint32_t box_at = base + S::kStages * S::kStage + warp * kEpiBox, leader_room = mapa_shared(room, 0);
        int acc = 0;
        uint32_t tpar = 0;
        for (int64_t t = blockIdx.x >> 1; t < tiles; t += clusters) {
            int64_t m0, n0;
            place(t, &m0, &n0);
            if (p.bias) {   // (the warp has met since it read the last tile's)
                for (int c = lane; c < kHalf; c += 32) {
                    const int64_t n = n0 + half * kHalf + c;
                    bias[warp][c] = n < p.N ? __half2float(p.bias[n]) : 0.f;
                }
                __syncwarp();
            }
            const bool ok = __all_sync(~0u, mbar_wait_cluster(tfull + 8 * acc, tpar, abort, p.timeout_ns));
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            const uint32_t d = trow + (acc ? S::kAcc1 : 0u);
            const int64_t row0 = m0 + rank * 128 + (warp & 3) * 32;
            // the columns that the other accumulator shares come first: the last
            // box of the first accumulator, the first of the second
            const bool shares = kBN == 256 && half == (acc ? 0 : 1);
            if (!shares && lane == 0) mbar_arrive_cluster_relaxed(leader_room);
#pragma unroll 1
            for (int i = 0; i < 2 * kBoxes; ++i) {   // 32 columns, half a box, at a time
                const int b = acc ? i : 2 * kBoxes - 1 - i;
                uint32_t r[32];
                tmem_ld_x16(d + b * 32, r);
                tmem_ld_x16(d + b * 32 + 16, r + 16);
                tmem_wait_ld();
                if (shares && i == 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(leader_room);
                }
                float v[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(r[c]);
                if (p.bias) {
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        const float4 f = *reinterpret_cast<const float4*>(&bias[warp][b * 32 + c]);
                        v[c] += f.x, v[c + 1] += f.y, v[c + 2] += f.z, v[c + 3] += f.w;
                    }
                }
                act_all(p.act, v);
                if (p.c_tma && (i & 1) == 0) {
                    if (lane == 0) bulk_wait_group_read<0>();   // the box's last store has read it
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st_smem_v4(box_at + lane * 128 + (((4 * (b & 1) + c) ^ (lane & 7)) << 4),
                               make_uint4(pack_half2(v[8 * c], v[8 * c + 1]), pack_half2(v[8 * c + 2], v[8 * c + 3]),
                                          pack_half2(v[8 * c + 4], v[8 * c + 5]), pack_half2(v[8 * c + 6], v[8 * c + 7])));
                if ((i & 1) == 0) continue;
                const int64_t nb = n0 + half * kHalf + (b & ~1) * 32;
                if (p.c_tma) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && nb < p.N && row0 < p.M) {
                        tma_store_2d(&p.tmC, box_at, static_cast<int32_t>(nb), static_cast<int32_t>(row0));
                        bulk_commit_group();
                    }
                } else {
                    __syncwarp();
                    store_rows(p, box_at, row0, nb, lane);
                    __syncwarp();
                }
            }
            tc_fence_before();
            if (acc) tpar ^= 1u;
            acc ^= 1;
        }
        if (p.c_tma && lane == 0) bulk_wait_group_all();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    if (warp == 9) tmem_dealloc_pair(tmem, 512);
}

}  // namespace mxf4_dev
