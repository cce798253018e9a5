// A mixture-of-experts layer for a few tokens: the routing kernel and the
// experts' kernel.
//
// With a handful of rows an expert every weight is used a few times at most,
// so the layer is bound by reading the chosen experts' weights once.  The
// tensor cores are fed by warps (mma.sync, m16n8k16): a tcgen05 tile would
// leave 120 of 128 rows empty and stage every byte for it.  The weights take
// the 16-row side and up to 8 tokens the narrow side; gate and up rows of the
// same 8 hidden values share one instruction, so that their sums meet in one
// thread.  Every warp streams its own share of K through a private ring of
// asynchronous copies: no barrier stands between a warp and its next bytes.
//
// K is reordered within 32 values, the same on both sides: thread c of a quad
// holds values 8c .. 8c + 7 of the block, one 16-byte word (or, in MXFP4, one
// 32-bit word of codes) a row, split over two instructions.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "gemm_f16.h"
#include "mxf4_convert.cuh"
#include "ptx.cuh"

namespace moe_dev {

using namespace gemm_f16_dev;

constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTop = 8, kMaxSlots = kMaxTokens * kMaxTop;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kRouteCluster = 8;   // CTAs that share a router product, and tokens of a group

__device__ __forceinline__ float act_f32(int act, float x)
{
    switch (act) {
    case 1: return x < 0.f ? 0.f : x;
    case 2: return x / (1.f + expf(-x));
    case 3: return x * (0.5f * erfcf(-x * 0.70710678118654752f));
    default: return x;
    }
}

// D (+)= A * B, m16n8k16, fp16 in, fp32 sums.
__device__ __forceinline__ void mma16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8x8 transpose of 16-bit elements held two a thread, a row a quad.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint4 ld_smem_v4(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

struct Weight {
    const uint8_t* data;
    const uint8_t* scales;
    int64_t se, si, so;   // fp16: element strides; MXFP4: se, so bytes of codes an expert and a row
    int64_t scale_se;     // MXFP4: scale bytes an expert
    int32_t kt;           // MXFP4: scale tiles along the contracted axis
};

// Counters of one call, zeroed by the routing kernel.
struct Control {
    int ticket_up, done_up, ticket_down;
};

struct Params {
    const __half* x;
    int64_t sxt, sxi;
    const __half* router;
    int64_t sri, sre;
    Weight gate, up, down;
    int32_t T, D, F, E, top, renorm, act;
    int32_t dp, fp;        // D and F rounded up to 64
    __half* y;
    int64_t ldy;
    float* weights;
    int32_t* ids;
    Control* ctl;
    __half* xp;            // [T][dp]: the tokens, packed, zeros past D
    __half* hp;            // [T * top][2][fp]: the hidden values as high and low halves, by expert
    int32_t test_stall;
    uint64_t timeout_ns;
    int* status;
};

// ---------------------------------------------------------------- routing
// Order-preserving key of a logit; a NaN above everything.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (v != v) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ __half ld_nc_half(const __half* p) { return __ushort_as_half(ld_nc_u16(p)); }

// How the router's elements lie: 0 any strides, 1 contracted axis contiguous,
// 2 experts contiguous (16-byte words in both).
enum { kAnyStrides = 0, kInContiguous = 1, kOutContiguous = 2 };

// Expert row of accumulator half `h` (rows g or g + 8) of instruction `mt` in a
// 32-expert tile: with the experts contiguous, a thread's 16-byte word holds
// experts 8c .. 8c + 7, whose pairs become the rows of four 8x8 transposes.
template <int kLayout>
__device__ __forceinline__ int expert_row(int mt, int h, int g)
{
    return kLayout == kOutContiguous ? 8 * (g >> 1) + 2 * (2 * mt + h) + (g & 1) : 16 * mt + 8 * h + g;
}

// A cluster of 8 CTAs routes 8 tokens: CTA r sums the r-th part of D for all
// experts and tokens, then takes token r: adds the 8 parts over distributed
// shared memory and picks its experts.  Bound by latency: the router is read
// once a cluster, a few 16-byte loads deep a thread.
template <int kLayout>
__global__ void __launch_bounds__(kThreads) moe_route(const __grid_constant__ Params p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int rank = static_cast<int>(cluster_ctarank());
    const int t0 = (blockIdx.x / kRouteCluster) * kRouteCluster;
    const int nt = min(kRouteCluster, p.T - t0);
    const int chunks = p.dp >> 5;
    const int c_lo = chunks * rank / kRouteCluster, c_hi = chunks * (rank + 1) / kRouteCluster;
    const int k_lo = c_lo * 32, width = (c_hi - c_lo) * 32;
    const int tiles = (p.E + 31) >> 5;
    // shared: this part's tokens [8][width + 8] fp16, warp sums [16][32][8], logits [8][E rounded up]
    const int xpitch = width + 8;
    __half* xs = reinterpret_cast<__half*>(smem);
    float* red = reinterpret_cast<float*>(smem + ((chunks / kRouteCluster + 1) * 32 + 8) * 8 * 2);
    float* part = red + kWarps * 32 * 8;
    const int ep = tiles * 32;

    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.ctl = Control{0, 0, 0};

    for (int i = threadIdx.x; i < 8 * width; i += kThreads) {
        const int t = i / width, k = i - t * width;
        __half v = __ushort_as_half(0);
        if (t < nt) {
            if (k_lo + k < p.D) v = ld_nc_half(p.x + (t0 + t) * p.sxt + (k_lo + k) * p.sxi);
            p.xp[static_cast<int64_t>(t0 + t) * p.dp + k_lo + k] = v;
        }
        xs[t * xpitch + k] = v;
    }
    __syncthreads();

    const int wt = min(tiles, kWarps), share = kWarps / wt;   // tiles a pass, warps a tile
    for (int pass = 0; pass * wt < tiles; ++pass) {
        const int tl = warp % wt, mine = warp / wt;
        const int tile = pass * wt + tl;
        float acc[2][4] = {};
        if (mine < share && tile < tiles) {
            const int e0 = tile * 32;
#pragma unroll 4
            for (int ch = mine; ch < c_hi - c_lo; ch += share) {
                const int k0 = k_lo + ch * 32;
                uint4 w[4];
                if (kLayout == kInContiguous) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int e = e0 + 8 * q + g, k = k0 + 8 * c;
                        w[q] = make_uint4(0, 0, 0, 0);
                        if (e < p.E) {
                            const __half* src = p.router + e * p.sre + k;
                            if (k + 8 <= p.D)
                                w[q] = ld_nc_v4(src);
                            else {
                                uint32_t u[4] = {};
                                for (int i = 0; i < 8; ++i)
                                    if (k + i < p.D) u[i >> 1] |= static_cast<uint32_t>(ld_nc_u16(src + i)) << (16 * (i & 1));
                                w[q] = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        }
                    }
                } else if (kLayout == kOutContiguous) {
                    // rows k of the reordered block: quad g's row is value 8 (g / 2) + g % 2 + 2q
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int k = k0 + 8 * (g >> 1) + (g & 1) + 2 * q, e = e0 + 8 * c;
                        w[q] = make_uint4(0, 0, 0, 0);
                        if (k < p.D) {
                            const __half* src = p.router + k * p.sri + e;
                            if (e + 8 <= p.E)
                                w[q] = ld_nc_v4(src);
                            else {
                                uint32_t u[4] = {};
                                for (int i = 0; i < 8; ++i)
                                    if (e + i < p.E) u[i >> 1] |= static_cast<uint32_t>(ld_nc_u16(src + i)) << (16 * (i & 1));
                                w[q] = make_uint4(u[0], u[1], u[2], u[3]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int e = e0 + 8 * q + g;
                        uint32_t u[4] = {};
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int k = k0 + 8 * c + i;
                            if (e < p.E && k < p.D)
                                u[i >> 1] |= static_cast<uint32_t>(ld_nc_u16(p.router + k * p.sri + e * p.sre)) << (16 * (i & 1));
                        }
                        w[q] = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
                const uint4 b = ld_smem_v4(smem_u32(xs + g * xpitch + ch * 32 + 8 * c));
                if (kLayout == kOutContiguous) {
                    // w[q] word j: 8x8 of value rows (q) and expert pairs j; its transpose is
                    // the operand piece of expert rows j, K piece q
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        uint32_t a[2][4];
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const int j = 2 * mt + h;
                                a[h][q] = transpose8x8(j == 0 ? w[q].x : j == 1 ? w[q].y : j == 2 ? w[q].z : w[q].w);
                            }
                        mma16816(acc[mt], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
                        mma16816(acc[mt], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
                    }
                } else {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        mma16816(acc[mt], w[2 * mt].x, w[2 * mt + 1].x, w[2 * mt].y, w[2 * mt + 1].y, b.x, b.y);
                        mma16816(acc[mt], w[2 * mt].z, w[2 * mt + 1].z, w[2 * mt].w, w[2 * mt + 1].w, b.z, b.w);
                    }
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[(warp * 32 + expert_row<kLayout>(mt, i >> 1, g)) * 8 + 2 * c + (i & 1)] = acc[mt][i];
        __syncthreads();
        for (int i = threadIdx.x; i < wt * 32 * 8; i += kThreads) {
            const int t = i & 7, e = i >> 3;
            float v = 0.f;
            for (int m = 0; m < share; ++m) v += red[((m * wt + (e >> 5)) * 32 + (e & 31)) * 8 + t];
            if (pass * wt * 32 + e < ep) part[t * ep + pass * wt * 32 + e] = v;
        }
        __syncthreads();
    }
    cluster_sync_all();
    if (rank < nt && warp == 0) {
        float l[kMaxExperts / 32];
        uint32_t key[kMaxExperts / 32];
#pragma unroll
        for (int i = 0; i < kMaxExperts / 32; ++i) {
            const int e = i * 32 + lane;
            l[i] = 0.f;
            key[i] = 0u;
            if (i * 32 < ep) {
                float v = 0.f;
                const uint32_t at = smem_u32(part + rank * ep + e);
#pragma unroll
                for (uint32_t r = 0; r < kRouteCluster; ++r) v += ld_cluster_f32(mapa_shared(at, r));
                if (e < p.E) l[i] = v, key[i] = order_key(v);
            }
        }
        float best = 0.f, total = 0.f, chosen = 0.f;
        int id = 0;   // lane j keeps the j-th choice
        for (int j = 0; j < p.top; ++j) {
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i) top = max(top, key[i]);
            top = __reduce_max_sync(~0u, top);
            uint32_t at = 0xFFFFFFFFu;
#pragma unroll
            for (int i = kMaxExperts / 32 - 1; i >= 0; --i)
                if (key[i] == top && i * 32 + lane < p.E) at = i * 32 + lane;
            at = __reduce_min_sync(~0u, at);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i)
                if (i == static_cast<int>(at >> 5)) {
                    v = l[i];
                    if (lane == static_cast<int>(at & 31)) key[i] = 0u;   // (keys of numbers are above 0)
                }
            v = __shfl_sync(~0u, v, at & 31);
            if (j == 0) best = v;
            if (lane == j) chosen = v, id = static_cast<int>(at);
        }
        const float mine = lane < p.top ? expf(chosen - best) : 0.f;
        if (p.renorm) {
            total = mine;
        } else {
#pragma unroll
            for (int i = 0; i < kMaxExperts / 32; ++i)
                if (i * 32 + lane < p.E) total += expf(l[i] - best);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(~0u, total, s);
        if (lane < p.top) {
            p.weights[(t0 + rank) * p.top + lane] = mine / total;
            p.ids[(t0 + rank) * p.top + lane] = id;
        }
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while its sums are being read
}

// ---------------------------------------------------------------- experts
// Weight formats of the experts' kernel.
enum { kF16Rows = 0, kF16Strided = 1, kMxf4 = 2 };

template <int kFmt>
struct Stage {
    static constexpr int kVals = kFmt == kMxf4 ? 128 : 64;             // values of K a step
    static constexpr int kRowBytes = kFmt == kMxf4 ? 64 : 128;
    static constexpr int kBytes = 16 * kRowBytes + (kFmt == kMxf4 ? 64 : 0);   // 16 rows, and their scales
    static constexpr int kRing = kFmt == kMxf4 ? 8 : 4;                        // stages of a warp's ring
};

// 16 weight rows x kVals of K into a stage: row r of the stage is row o0 + r of
// one projection, or with `pair` rows o0 + r (r < 8) of w0 and o0 + r - 8 of w1.
// Rows from `rows` on and values from K on are zeros.
template <int kFmt>
__device__ __forceinline__ void load_stage(uint32_t dst, const Weight& w0, const Weight& w1, bool pair, int e, int o0,
                                           int rows, int k0, int K, int lane)
{
    if (kFmt == kF16Rows) {
        const int c = lane & 7, k = k0 + 8 * c;
        const uint32_t bytes = 2 * max(0, min(8, K - k));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = (lane >> 3) + 4 * j;
            const Weight& w = pair && j >= 2 ? w1 : w0;
            const int o = o0 + (pair ? r & 7 : r);
            const bool in = o < rows && bytes;
            const __half* src = reinterpret_cast<const __half*>(w.data) + (in ? e * w.se + o * w.so + k : 0);
            cp_async16(dst + r * 128 + ((c ^ ((r & 1) << 2)) << 4), src, in ? bytes : 0u);
        }
    } else if (kFmt == kF16Strided) {
        const int c = lane & 7, k = k0 + 8 * c;
#pragma unroll 1
        for (int j = 0; j < 4; ++j) {
            const int r = (lane >> 3) + 4 * j;
            const Weight& w = pair && j >= 2 ? w1 : w0;
            const int o = o0 + (pair ? r & 7 : r);
            uint32_t u[4] = {};
            if (o < rows) {
                const __half* src = reinterpret_cast<const __half*>(w.data) + e * w.se + o * w.so;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < K) u[i >> 1] |= static_cast<uint32_t>(ld_nc_u16(src + (k + i) * w.si)) << (16 * (i & 1));
            }
            st_smem_v4(dst + r * 128 + ((c ^ ((r & 1) << 2)) << 4), make_uint4(u[0], u[1], u[2], u[3]));
        }
    } else {
        const int c = lane & 3, k = k0 + 32 * c;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = (lane >> 2) + 8 * j;
            const Weight& w = pair && j ? w1 : w0;
            const int o = o0 + (pair ? r & 7 : r);
            const bool in = o < rows && k < K;
            const uint8_t* src = w.data + (in ? e * w.se + o * w.so + (k >> 1) : 0);
            cp_async16(dst + r * 64 + ((c ^ ((r >> 1) & 3)) << 4), src, in ? 16u : 0u);
        }
        if (lane < 16) {
            const Weight& w = pair && lane >= 8 ? w1 : w0;
            const int o = o0 + (pair ? lane & 7 : lane);
            const bool in = o < rows && k0 < K;
            const uint8_t* src = w.scales + (in ? e * w.scale_se + mxf4_dev::scale_at(o, k0 >> 5, w.kt) : 0);
            cp_async4(dst + 1024 + lane * 4, src, in ? 4u : 0u);
        }
    }
}

// acc += the stage's rows times the step's values of the columns' vectors b
// (one 16-byte word for each 32 values and group of 8 columns).
template <int kFmt, int kGroups>
__device__ __forceinline__ void mma_stage(float (*acc)[4], uint32_t src, const uint4 (*b)[kGroups], int groups, int g,
                                          int c)
{
    if (kFmt != kMxf4) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = src + g * 128 + (((4 * h + c) ^ ((g & 1) << 2)) << 4);
            const uint4 lo = ld_smem_v4(at), hi = ld_smem_v4(at + 8 * 128);
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                if (q < groups) {
                    mma16816(acc[q], lo.x, hi.x, lo.y, hi.y, b[h][q].x, b[h][q].y);
                    mma16816(acc[q], lo.z, hi.z, lo.w, hi.w, b[h][q].z, b[h][q].w);
                }
            }
        }
    } else {
        const uint32_t slo = ld_smem_u32(src + 1024 + g * 4), shi = ld_smem_u32(src + 1024 + (g + 8) * 4);
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t at = src + g * 64 + ((h ^ ((g >> 1) & 3)) << 4) + c * 4;
            uint32_t lo[4], hi[4];
            mxf4_dev::halves_of(ld_smem_u32(at), lo);
            mxf4_dev::halves_of(ld_smem_u32(at + 8 * 64), hi);
            const float s0 = mxf4_dev::scale_value(slo >> (8 * h) & 255u), s1 = mxf4_dev::scale_value(shi >> (8 * h) & 255u);
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                if (q < groups) {
                    // the block's sum, exact products of fp16 values, then its scale
                    float d[4] = {};
                    mma16816(d, lo[0], hi[0], lo[1], hi[1], b[h][q].x, b[h][q].y);
                    mma16816(d, lo[2], hi[2], lo[3], hi[3], b[h][q].z, b[h][q].w);
                    acc[q][0] = fmaf(d[0], s0, acc[q][0]);
                    acc[q][1] = fmaf(d[1], s0, acc[q][1]);
                    acc[q][2] = fmaf(d[2], s1, acc[q][2]);
                    acc[q][3] = fmaf(d[3], s1, acc[q][3]);
                }
            }
        }
    }
}

__device__ __forceinline__ uint4 ld_v4(const void* p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// What a piece of an expert's work is: up to 8 * kGroups tokens of one expert
// (an expert with more is read once for each such piece).
struct Item {
    uint16_t expert, first, count;   // first: place in the list of choices ordered by expert
};

struct Shared {
    uint16_t slot[kMaxSlots];        // choices (token * top + j) ordered by expert, then by token
    float weight[kMaxSlots];         // their routing weights
    Item item[kMaxSlots];
    uint16_t first_of[kMaxExperts];
    uint32_t scan[kWarps];
    int items, ticket, ok;
};

// All experts of the layer.  Two phases, gate/up and down, each cut into
// gridDim parts of equal bytes; a CTA takes a part by ticket and, before it
// starts on a down part, waits until every gate/up part is done.  Tickets of
// gate/up parts are taken by running CTAs only and are all gone before any CTA
// waits, so the wait ends whichever CTAs the device holds at once.  A down
// part's first weights are on their way before the wait.
template <int kFmt, int kGroups>
__global__ void __launch_bounds__(kThreads, 1) moe_experts(const __grid_constant__ Params p)
{
    using St = Stage<kFmt>;
    constexpr int kB = St::kVals / 32, kRing = St::kRing;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Shared sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (kRing * St::kBytes);
    uint8_t* tail = smem + kWarps * kRing * St::kBytes;   // sums: gate/up [2][16][kGroups][32] float4, down [16][T][16]
    const int parts = gridDim.x;

    griddep_wait();
    griddep_launch_dependents();

    // ---- the choices ordered by expert
    const int slots = p.T * p.top;
    {
        uint16_t* wcount = reinterpret_cast<uint16_t*>(smem);   // [16 warps][E], in the ring before its first use
        const int nw = (slots + 31) >> 5;
        for (int i = threadIdx.x; i < nw * p.E; i += kThreads) wcount[i] = 0;
        if (threadIdx.x == 0) sh.ticket = atomicAdd(&p.ctl->ticket_up, 1);
        __syncthreads();
        const bool mine = static_cast<int>(threadIdx.x) < slots;
        const int e = mine ? p.ids[threadIdx.x] : -1;
        const uint32_t same = __match_any_sync(~0u, e);
        const int before = __popc(same & ((1u << lane) - 1u));
        if (mine && before == 0) wcount[warp * p.E + e] = static_cast<uint16_t>(__popc(same));
        __syncthreads();
        // thread e: this expert's count, its place, its pieces
        const int ex = threadIdx.x;
        int count = 0;
        if (ex < p.E)
            for (int w = 0; w < nw; ++w) {
                const int n = wcount[w * p.E + ex];
                wcount[w * p.E + ex] = static_cast<uint16_t>(count);
                count += n;
            }
        const int pieces = (count + 8 * kGroups - 1) / (8 * kGroups);
        uint32_t sum = static_cast<uint32_t>(count) << 16 | pieces;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const uint32_t o = __shfl_up_sync(~0u, sum, s);
            if (lane >= s) sum += o;
        }
        if (lane == 31) sh.scan[warp] = sum;
        __syncthreads();
        uint32_t base = 0;
        for (int w = 0; w < warp; ++w) base += sh.scan[w];
        sum += base;
        const int first = static_cast<int>(sum >> 16) - count, piece0 = static_cast<int>(sum & 0xFFFFu) - pieces;
        if (ex < p.E) {
            sh.first_of[ex] = static_cast<uint16_t>(first);
            for (int i = 0; i < pieces; ++i)
                sh.item[piece0 + i] = Item{static_cast<uint16_t>(ex), static_cast<uint16_t>(first + i * 8 * kGroups),
                                           static_cast<uint16_t>(min(8 * kGroups, count - i * 8 * kGroups))};
        }
        if (threadIdx.x == kThreads - 1) sh.items = static_cast<int>(sum & 0xFFFFu);
        __syncthreads();
        if (mine) {
            const int at = sh.first_of[e] + wcount[warp * p.E + e] + before;
            sh.slot[at] = static_cast<uint16_t>(threadIdx.x);
            sh.weight[at] = p.weights[threadIdx.x];
        }
        __syncthreads();
    }
    const int items = sh.items;
    int ticket = sh.ticket;

    // ---- gate and up: a unit is one piece's 8 hidden values, K dealt to the warps
    const int units_each = p.fp >> 3, steps = (p.D + St::kVals - 1) / St::kVals;
    const int wsteps = (steps - warp + kWarps - 1) / kWarps;   // this warp's steps of a unit
    while (ticket < parts) {
        const int64_t all = static_cast<int64_t>(items) * units_each;
        const int u_lo = static_cast<int>(all * ticket / parts), u_hi = static_cast<int>(all * (ticket + 1) / parts);
        const int mine = (u_hi - u_lo) * wsteps;   // steps of this warp in all
        int pu = u_lo, ps = 0;                     // the next one to load
        auto issue = [&](int n) {
            if (n < mine) {
                const int it = pu / units_each, f0 = (pu - it * units_each) * 8;
                load_stage<kFmt>(ring + (n % kRing) * St::kBytes, p.gate, p.up, true, sh.item[it].expert, f0, p.F,
                                 (warp + ps * kWarps) * St::kVals, p.D, lane);
                if (++ps == wsteps) ps = 0, ++pu;
            }
            cp_async_commit();
        };
        for (int n = 0; n < kRing - 1; ++n) issue(n);
        int n = 0;
        for (int u = u_lo; u < u_hi; ++u) {
            const int it = u / units_each, f0 = (u - it * units_each) * 8;
            const Item im = sh.item[it];
            const int groups = (im.count + 7) >> 3;
            const __half* col[kGroups];
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                col[q] = p.xp + static_cast<int64_t>(sh.slot[im.first + min(8 * q + g, im.count - 1)] / p.top) * p.dp + 8 * c;
            float acc[kGroups][4] = {};
            for (int s = 0; s < wsteps; ++s, ++n) {
                uint4 b[kB][kGroups];
                const int k0 = (warp + s * kWarps) * St::kVals;
#pragma unroll
                for (int h = 0; h < kB; ++h)
#pragma unroll
                    for (int q = 0; q < kGroups; ++q)
                        b[h][q] = q < groups && k0 + 32 * h < p.dp ? ld_v4(col[q] + k0 + 32 * h) : make_uint4(0, 0, 0, 0);
                cp_async_wait<kRing - 2>();
                __syncwarp();   // (every lane is done with the stage that is filled next)
                issue(n + kRing - 1);
                mma_stage<kFmt, kGroups>(acc, ring + (n % kRing) * St::kBytes, b, groups, g, c);
            }
            float4* sums = reinterpret_cast<float4*>(tail) + (u & 1) * (kWarps * kGroups * 32);
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                if (q < groups) sums[(warp * kGroups + q) * 32 + lane] = make_float4(acc[q][0], acc[q][1], acc[q][2], acc[q][3]);
            __syncthreads();
            // one warp a group adds the 16 parts; the warps take turns
            const int q = (warp + kWarps - u * kGroups % kWarps) % kWarps;
            if (q < groups) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 a = sums[(w * kGroups + q) * 32 + lane];
                    v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = 8 * q + 2 * c + i;
                    if (j < im.count) {
                        // (past F: zeros, whatever the tokens hold)
                        const float hv = f0 + g < p.F ? act_f32(p.act, i ? v.y : v.x) * (i ? v.w : v.z) : 0.f;
                        const __half hi = __float2half_rn(hv);
                        const float back = __half2float(hi);
                        const __half lo = isfinite(back) ? __float2half_rn(hv - back) : __ushort_as_half(0);
                        __half* dst = p.hp + static_cast<int64_t>(im.first + j) * 2 * p.fp + f0 + g;
                        dst[0] = hi;
                        dst[p.fp] = lo;
                    }
                }
            }
        }
        cp_async_wait<0>();
        __syncthreads();
        if (threadIdx.x == 0) {
            if (!p.test_stall) atom_add_acq_rel_gpu(&p.ctl->done_up, 1);
            sh.ticket = atomicAdd(&p.ctl->ticket_up, 1);
        }
        __syncthreads();
        ticket = sh.ticket;
    }

    // ---- down: a part is a range of 16-column tiles; a warp takes a range of a
    // tile's (piece, step) pairs and keeps its own weighted sums of the tokens
    if (threadIdx.x == 0) sh.ticket = atomicAdd(&p.ctl->ticket_down, 1);
    __syncthreads();
    ticket = sh.ticket;
    constexpr int kCols = 2 * kGroups;   // groups of 8 columns: a choice takes two (high and low half)
    const int tiles = (p.D + 15) >> 4, fsteps = (p.F + St::kVals - 1) / St::kVals;
    const int total = items * fsteps;
    const int w_lo = total * warp / kWarps, w_hi = total * (warp + 1) / kWarps, per = w_hi - w_lo;
    float* ysum = reinterpret_cast<float*>(tail);
    float* mysum = ysum + warp * p.T * 16;
    bool waited = false;
    while (ticket < parts) {
        const int t_lo = static_cast<int>(static_cast<int64_t>(tiles) * ticket / parts),
                  t_hi = static_cast<int>(static_cast<int64_t>(tiles) * (ticket + 1) / parts);
        const int mine = (t_hi - t_lo) * per;
        int pt = t_lo, pi = w_lo;
        auto issue = [&](int n) {
            if (n < mine) {
                const int it = pi / fsteps;
                load_stage<kFmt>(ring + (n % kRing) * St::kBytes, p.down, p.down, false, sh.item[it].expert, pt * 16, p.D,
                                 (pi - it * fsteps) * St::kVals, p.F, lane);
                if (++pi == w_hi) pi = w_lo, ++pt;
            }
            cp_async_commit();
        };
        for (int n = 0; n < kRing - 1; ++n) issue(n);
        for (int i = threadIdx.x; i < kWarps * p.T * 16; i += kThreads) ysum[i] = 0.f;
        if (!waited) {
            if (threadIdx.x == 0) {
                const uint64_t t0 = globaltimer_ns();
                sh.ok = 1;
                while (ld_acquire_gpu(&p.ctl->done_up) < parts) {
                    if (globaltimer_ns() - t0 > p.timeout_ns) {
                        sh.ok = 0;
                        atomicExch(p.status, GEMM_F16_ERR_TIMEOUT);
                        break;
                    }
                }
            }
            waited = true;
        }
        __syncthreads();
        if (!sh.ok) break;
        int n = 0;
        for (int tile = t_lo; tile < t_hi; ++tile) {
            int it = -1;
            Item im = {};
            int groups = 0;
            const __half* col[kCols];
            float acc[kCols][4];
            auto flush = [&]() {
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    const int j = 4 * q + c;   // this thread's columns are the halves of choice j
                    if (j < im.count) {
                        const float w = sh.weight[im.first + j];
                        float* to = mysum + sh.slot[im.first + j] / p.top * 16;
                        to[g] = fmaf(w, acc[q][0] + acc[q][1], to[g]);
                        to[g + 8] = fmaf(w, acc[q][2] + acc[q][3], to[g + 8]);
                    }
                }
                __syncwarp();
            };
            for (int i = w_lo; i < w_hi; ++i, ++n) {
                if (i / fsteps != it) {
                    if (it >= 0) flush();
                    it = i / fsteps;
                    im = sh.item[it];
                    groups = (2 * im.count + 7) >> 3;
#pragma unroll
                    for (int q = 0; q < kCols; ++q) {
                        const int j = im.first + min(4 * q + (g >> 1), im.count - 1);
                        col[q] = p.hp + (static_cast<int64_t>(j) * 2 + (g & 1)) * p.fp + 8 * c;
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[q][e] = 0.f;
                    }
                }
                const int k0 = (i - it * fsteps) * St::kVals;
                uint4 b[kB][kCols];
#pragma unroll
                for (int h = 0; h < kB; ++h)
#pragma unroll
                    for (int q = 0; q < kCols; ++q)
                        b[h][q] = q < groups && k0 + 32 * h < p.fp ? ld_v4(col[q] + k0 + 32 * h) : make_uint4(0, 0, 0, 0);
                cp_async_wait<kRing - 2>();
                __syncwarp();   // (every lane is done with the stage that is filled next)
                issue(n + kRing - 1);
                mma_stage<kFmt, kCols>(acc, ring + (n % kRing) * St::kBytes, b, groups, g, c);
            }
            if (it >= 0) flush();
            __syncthreads();
            for (int i = threadIdx.x; i < p.T * 16; i += kThreads) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    v += ysum[w * p.T * 16 + i];
                    ysum[w * p.T * 16 + i] = 0.f;
                }
                const int t = i >> 4, d = tile * 16 + (i & 15);
                if (d < p.D) p.y[t * p.ldy + d] = __float2half_rn(v);
            }
            __syncthreads();
        }
        cp_async_wait<0>();
        __syncthreads();
        if (threadIdx.x == 0) sh.ticket = atomicAdd(&p.ctl->ticket_down, 1);
        __syncthreads();
        ticket = sh.ticket;
    }
    cp_async_wait<0>();
}

}  // namespace moe_dev
