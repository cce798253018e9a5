// A mixture-of-experts layer for a few tokens: the routing kernel, and the
// experts' kernel for weights at any strides (moe_stream.cuh has the one for
// weights that TMA can address).
//
// That kernel is bound by the loads that turn unaligned rows into operands, so
// warps feed the tensor cores themselves (mma.sync, m16n8k16).  The weights take
// the 16-row side and up to 8 tokens the narrow side; gate and up rows of the
// same 8 hidden values share one instruction, so that their sums meet in one
// thread.  Every warp brings its own share of K through a private ring: no
// barrier stands between a warp and its next bytes.
//
// Measured on 16 tokens, 8 of 64 experts of 2047 x 1023, 0.7 GB: 274 to 282 us with
// rows contiguous along k (issue on 59 % of cycles: the shifts), 299 to 321 us the
// other way (64-byte runs that start anywhere: DRAM reads 2.6 times the bytes).  With
// loads through registers, waited for before the next step's, they were 360 and 433.
// Projections of different orders share no unit stride and are read value by
// value: 561 us where 2048 x 1024 in one order streams in 133.
//
// K is reordered within 32 values, the same on both sides: thread c of a quad
// holds values 8c .. 8c + 7 of the block, one 16-byte word a row, split over two
// instructions.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "gemm_f16.h"
#include "mxf4_format.cuh"
#include "ptx.cuh"

namespace moe_dev {

using namespace gemm_f16_dev;

constexpr int kMaxTokens = 64, kMaxExperts = 512, kMaxTop = 8, kMaxSlots = kMaxTokens * kMaxTop;
constexpr int kPieces = 8;   // MXFP4 columns that a value of the narrow side is held in (split_blocks)
constexpr int kThreads = 512, kWarps = kThreads / 32;
// Shares of the experts' K that a range of y's columns is cut into at most, where the
// ranges alone leave CTAs idle: more cost more in sums than they fill (8 of 64 experts of
// 2047 x 1023, rows contiguous along k and the other way: 1 token 51 and 58 us with up to
// 4 shares, 72 and 65 with 8, 51 and 67 with none; 16 tokens 274 and 321, 287 and 337, 274
// and 412).
constexpr int kMaxSplits = 4, kMaxRanges = 2048;   // ranges of 16 columns at least, 32768 in all
constexpr int kRouteCluster = 8;   // CTAs that share a router product, and tokens of a group

__device__ __forceinline__ float act_f32(int act, float x)
{
    switch (act) {
    case 1: return x < 0.f ? 0.f : x;
    case 2: return __fdividef(x, 1.f + __expf(-x));   // (no branch; x < -87: 0 for a value under 2^-119)
    case 3: return x * (0.5f * erfcf(-x * 0.70710678118654752f));
    default: return x;
    }
}

// A hidden value for fp16 weights: its rounding to fp16 and 2^11 times what that
// leaves, in fp16 too.  What is left is at most half the first one's last place,
// 2^-11 of the power of two below the value, so that the second neither
// overflows (16 * 2^11 at most) nor, down to values of 2^-14, falls under its own
// type: the pair is within 2^-23 of the value, or 2^-36 where that is less.
// (Without the factor the second half lost bits below 2^-3 and all of them
// below 2^-14: outputs of 2^-12 from hidden values of 2^-17 were 2.2e-3 off.)
constexpr float kLowScale = 2048.f;

__device__ __forceinline__ void split_hidden(float h, __half* hi, __half* lo)
{
    *hi = __float2half_rn(h);
    const float back = __half2float(*hi);
    *lo = isfinite(back) ? __float2half_rn((h - back) * kLowScale) : __ushort_as_half(0);
}

// The sum of the two halves' products.
__device__ __forceinline__ float join_hidden(float hi, float lo) { return fmaf(lo, 1.f / kLowScale, hi); }

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

// Counters of one call.
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
    int* zero;             // the experts' kernel's counters: the routing kernel sets `nzero` words to 0
    int32_t nzero;
    uint8_t* xq;           // MXFP4 weights: the tokens as [T][kPieces] rows of xq_pitch bytes of codes,
    uint8_t* xs;           // and their scales, xs_pitch bytes a row (otherwise null)
    int32_t xq_pitch, xs_pitch;
    Control* ctl;
    int32_t splits;        // shares of the experts' K a range of y's columns is cut into
    int32_t* counts;       // [column ranges]: finished shares
    float* parts;          // [splits][T][dp]: their sums
    __half* xp;            // [T][dp]: the tokens, packed, zeros past D
    __half* hp;            // [T * top][2][fp]: the hidden values as split_hidden's halves, by expert
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

// How the router's elements lie: 0 any strides, 1 contracted axis contiguous,
// 2 experts contiguous (16-byte words in both).
enum { kAnyStrides = 0, kInContiguous = 1, kOutContiguous = 2 };

// Four blocks of 32 values as kPieces MXFP4 columns; lane 8j + i holds values 4i
// .. 4i + 3 of block j in v.  `codes`: this lane's two bytes of column 0, `pitch`
// bytes to the next column; `scale`: its block's scale of column 0.  Blocks with
// `on` false are not written.
//
// Column 0's scale 2^s is the smallest under which the block's largest magnitude
// does not saturate, so that it is above 3 * 2^s (a quantised operand's is a step
// smaller for magnitudes of 6 to 8 times 2^s).  e2m1 steps by 2 up to 6, by 1 up
// to 4: column 0 leaves at most 2^s, 4 steps under 2^(s - 2), and from then on
// each column leaves at most half of its own unit, 4 steps of one 8 times
// smaller.  So the scales are known beforehand, s, s - 2, s - 5, s - 8, .., and 8
// columns leave at most 2^(s - 21), 2^-22.5 of the block's largest magnitude: what
// a sum in 32 bits loses beside a term of that size, so that values next to an
// outlier keep their bits.  (6 columns leave 2^-16.5: beside an outlier of 1000
// the other 31 values were 2.3e-3 of their norm off, ten times an fp16 value's
// own rounding, and 64 tokens over 64 experts took 280 us instead of 288.  A
// search for each remainder's own largest magnitude took 2.5 times as long.)
__device__ __forceinline__ void split_blocks(float* v, bool on, int lane, uint8_t* codes, int64_t pitch, uint8_t* scale,
                                             int64_t spitch)
{
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) top = max(top, __shfl_xor_sync(~0u, top, s));
    uint32_t code = mxf4_dev::scale_code<float>(top);
    const bool nan = code == 255u;
    if (!nan) code += (top & 0x7FFFFFu) > 0x400000u && code > 0u;   // above 6 * 2^s: mantissa above 1.5
#pragma unroll 1
    for (int q = 0; q < kPieces; ++q) {
        uint32_t e = 0;
        if (!nan) {
            const float f = mxf4_dev::pow2f(127 - static_cast<int>(code)), back = mxf4_dev::scale_value(code);
            uint32_t h0, h1;
            asm("{\n\t.reg .b8 b0, b1;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 b0, %4, %3;\n\t"
                "cvt.rn.satfinite.e2m1x2.f32 b1, %6, %5;\n\t"
                "cvt.rn.f16x2.e2m1x2 %1, b0;\n\t"
                "cvt.rn.f16x2.e2m1x2 %2, b1;\n\t"
                "mov.b32 %0, {b0, b1, b0, b1};\n\t}"
                : "=r"(e), "=r"(h0), "=r"(h1)
                : "f"(v[0] * f), "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f));
            v[0] -= back * __half2float(__ushort_as_half(static_cast<unsigned short>(h0)));
            v[1] -= back * __half2float(__ushort_as_half(static_cast<unsigned short>(h0 >> 16)));
            v[2] -= back * __half2float(__ushort_as_half(static_cast<unsigned short>(h1)));
            v[3] -= back * __half2float(__ushort_as_half(static_cast<unsigned short>(h1 >> 16)));
        }
        if (on) {
            *reinterpret_cast<uint16_t*>(codes + q * pitch) = static_cast<uint16_t>(e);
            if ((lane & 7) == 0) scale[q * spitch] = static_cast<uint8_t>(code);
        }
        if (!nan) code -= min(code, q == 0 ? 2u : 3u);
    }
}

// 16 bytes of fp16 at base + at to shared memory, `n` of the 8 values in range
// (less: zeros).
__device__ __forceinline__ void bring_eight(uint32_t dst, const __half* base, int64_t at, int64_t step, bool vector, int n)
{
    const __half* src = base + (n > 0 ? at : 0);
    if (vector) {
        cp_async16(dst, src, 2 * max(0, min(8, n)));
        return;
    }
    uint32_t u[4] = {};
    for (int i = 0; i < min(n, 8); ++i) {
        const uint32_t v = static_cast<uint32_t>(ld_nc_u16(src + i * step)) << (16 * (i & 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] |= j == i >> 1 ? v : 0u;
    }
    st_smem_v4(dst, make_uint4(u[0], u[1], u[2], u[3]));
}

template <bool kTrans>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t* a)
{
    if (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]) : "r"(addr) : "memory");
}

// How a cluster's CTA lays out its shared memory; the same on the host.
struct RouteShape {
    int width, kc, wpitch, xpitch;      // values of D a CTA takes at most, at a time; bytes a row of weights, tokens
    int x, w, red, part, bytes;         // offsets
    __host__ __device__ RouteShape(int dp, int experts, bool out_contiguous)
    {
        const int ep = (experts + 15) / 16 * 16;
        width = ((dp >> 5) / kRouteCluster + 1) * 32;
        const int most = (112 * 1024 / (2 * ep + 16)) / 32 * 32;
        kc = width < most ? width : most;
        wpitch = 2 * (out_contiguous ? ep : kc) + 16;
        xpitch = 2 * width + 16;
        x = 0;
        w = x + 8 * xpitch;
        red = w + (out_contiguous ? kc : ep) * wpitch;
        part = red + (kWarps * 16 * 8 > kRouteCluster * ep ? kWarps * 16 * 8 : kRouteCluster * ep) * 4;
        bytes = part + 8 * ep * 4;
    }
};

// A cluster of 8 CTAs routes 8 tokens: CTA r sums the r-th part of D for all
// experts and tokens, then takes token r: adds the 8 parts over distributed
// shared memory and picks its experts.  Bound by latency: the tokens' and the
// router's parts are brought to shared memory at once, and the loops are not
// unrolled (every instruction is fetched once, cold: with the loads and the
// MMAs unrolled in registers this part took 7 us instead of 4).  kPer: experts
// a lane of the choosing warp looks at.
template <int kLayout, int kPer>
__global__ void __launch_bounds__(kThreads) moe_route(const __grid_constant__ Params p)
{
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int t0 = (blockIdx.x / kRouteCluster) * kRouteCluster;
    const int nt = min(kRouteCluster, p.T - t0);
    const int chunks = p.dp >> 5;
    const int c_lo = chunks * rank / kRouteCluster, c_hi = chunks * (rank + 1) / kRouteCluster;
    const int k_lo = c_lo * 32, width = (c_hi - c_lo) * 32;
    const int tiles = (p.E + 15) >> 4, ep = tiles * 16;
    constexpr bool kOut = kLayout == kOutContiguous;
    const RouteShape sh(p.dp, p.E, kOut);
    const uint32_t base = smem_u32(smem);
    float* red = reinterpret_cast<float*>(smem + sh.red);     // [16 warps][16 experts][8 tokens], then [8 parts][ep]
    float* part = reinterpret_cast<float*>(smem + sh.part);   // [8 tokens][ep]

    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0)
        for (int i = threadIdx.x; i < p.nzero; i += kThreads) p.zero[i] = 0;
    const bool xvec = p.sxi == 1 && ((reinterpret_cast<uintptr_t>(p.x) | (2 * p.sxt)) & 15) == 0;
    {   // tokens: 64 threads each, 8 values a thread and turn
        const int t = threadIdx.x >> 6;
#pragma unroll 1
        for (int k = (threadIdx.x & 63) * 8; k < width; k += 512)
            bring_eight(base + sh.x + t * sh.xpitch + 2 * k, p.x, (t0 + t) * p.sxt + (k_lo + k) * p.sxi, p.sxi, xvec,
                        t < nt ? p.D - k_lo - k : 0);
    }
    for (int i = threadIdx.x; i < 8 * ep; i += kThreads) part[i] = 0.f;
    const int share = tiles < kWarps ? kWarps / tiles : 1;   // warps of a 16-expert tile
#pragma unroll 1
    for (int k0 = 0; k0 < width; k0 += sh.kc) {
        const int kn = min(sh.kc, width - k0);
        // the router's rows k (experts contiguous) or e (values contiguous)
        const int words = kOut ? ep / 8 : kn / 8, rows = kOut ? kn : ep;
#pragma unroll 1
        for (int i = threadIdx.x; i < rows * words; i += kThreads) {
            const int r = i / words, c = i - r * words;
            const int k = k_lo + k0 + (kOut ? r : 8 * c), e = kOut ? 8 * c : r;
            const bool in = kOut ? k < p.D : e < p.E;
            bring_eight(base + sh.w + r * sh.wpitch + 16 * c, p.router, k * p.sri + e * p.sre, kOut ? p.sre : p.sri,
                        kLayout != kAnyStrides, in ? (kOut ? p.E - e : p.D - k) : 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll 1
        for (int first = 0; first < tiles; first += kWarps) {
            const int tile = first + warp / share, mine = warp % share;
            const int here = min(tiles - first, kWarps / share);   // tiles of this turn
            float acc[4] = {};
            if (warp / share < here) {
                // operand pieces: rows 0-7 and 8-15 of the first 8 values, then of the next 8
                const int j = lane & 7, piece = lane >> 3;
                const uint32_t wa = base + sh.w + (kOut ? (j + 8 * (piece >> 1)) * sh.wpitch + (tile * 16 + 8 * (piece & 1)) * 2
                                                        : (tile * 16 + j + 8 * (piece & 1)) * sh.wpitch + 16 * (piece >> 1));
                const uint32_t xa = base + sh.x + (lane >> 2) * sh.xpitch + (lane & 3) * 4 + 2 * k0;
                const uint32_t wstep = kOut ? 16 * sh.wpitch : 32;
#pragma unroll 2
                for (int s = mine; s < kn / 16; s += share) {
                    uint32_t a[4];
                    ldmatrix4<kOut>(wa + s * wstep, a);
                    mma16816(acc, a[0], a[1], a[2], a[3], ld_smem_u32(xa + 32 * s), ld_smem_u32(xa + 32 * s + 16));
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) red[(warp * 16 + (lane >> 2) + 8 * (i >> 1)) * 8 + 2 * (lane & 3) + (i & 1)] = acc[i];
            __syncthreads();
            for (int i = threadIdx.x; i < here * 128; i += kThreads) {
                const int t = i & 7, e = i >> 3;
                float v = 0.f;
                for (int m = 0; m < share; ++m) v += red[(((e >> 4) * share + m) * 16 + (e & 15)) * 8 + t];
                part[t * ep + first * 16 + e] += v;
            }
            __syncthreads();
        }
    }
    cluster_sync_all();
    // this CTA's token: the 8 parts of its logits
    if (rank < nt)
        for (int i = threadIdx.x; i < kRouteCluster * ep; i += kThreads)
            red[i] = ld_cluster_f32(mapa_shared(smem_u32(part + rank * ep + i % ep), static_cast<uint32_t>(i / ep)));
    __syncthreads();
    if (rank < nt && warp == 0) {
        float l[kPer];
        uint32_t key[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = i * 32 + lane;
            l[i] = 0.f;
            key[i] = 0u;
            if (e < p.E) {
                for (int r = 0; r < kRouteCluster; ++r) l[i] += red[r * ep + e];
                key[i] = order_key(l[i]);
            }
        }
        float best = 0.f, chosen = 0.f;
        int id = 0;   // lane j keeps the j-th choice
#pragma unroll 1
        for (int j = 0; j < p.top; ++j) {
            uint32_t top = 0u;
#pragma unroll
            for (int i = 0; i < kPer; ++i) top = max(top, key[i]);
            top = __reduce_max_sync(~0u, top);
            uint32_t at = 0xFFFFFFFFu;
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i)
                if (key[i] == top && i * 32 + lane < p.E) at = i * 32 + lane;
            at = __reduce_min_sync(~0u, at);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i == static_cast<int>(at >> 5)) {
                    v = l[i];
                    if (lane == static_cast<int>(at & 31)) key[i] = 0u;   // (keys of numbers are above 0)
                }
            v = __shfl_sync(~0u, v, at & 31);
            if (j == 0) best = v;
            if (lane == j) chosen = v, id = static_cast<int>(at);
        }
        const float mine = lane < p.top ? expf(chosen - best) : 0.f;
        float total = mine;
        if (!p.renorm) {
            total = 0.f;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i * 32 + lane < p.E) total += expf(l[i] - best);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) total += __shfl_xor_sync(~0u, total, s);
        if (lane < p.top) {
            p.weights[(t0 + rank) * p.top + lane] = mine / total;
            p.ids[(t0 + rank) * p.top + lane] = id;
        }
    } else if (warp > 0) {
        const uint8_t* xs = smem + sh.x;
        if (p.xq) {   // the tokens' part as MXFP4 columns, four blocks a warp and turn
            const int blocks = width >> 5, all = nt * blocks;
#pragma unroll 1
            for (int i = (warp - 1) * 4; i < all; i += (kWarps - 1) * 4) {
                const int n = min(i + (lane >> 3), all - 1), t = n / blocks, blk = n - t * blocks;
                const uint2 u = *reinterpret_cast<const uint2*>(xs + t * sh.xpitch + blk * 64 + (lane & 7) * 8);
                float v[4];
                v[0] = __half2float(__ushort_as_half(static_cast<unsigned short>(u.x)));
                v[1] = __half2float(__ushort_as_half(static_cast<unsigned short>(u.x >> 16)));
                v[2] = __half2float(__ushort_as_half(static_cast<unsigned short>(u.y)));
                v[3] = __half2float(__ushort_as_half(static_cast<unsigned short>(u.y >> 16)));
                const int64_t row = static_cast<int64_t>(t0 + t) * kPieces, at = (k_lo >> 5) + blk;
                split_blocks(v, i + (lane >> 3) < all, lane, p.xq + row * p.xq_pitch + at * 16 + (lane & 7) * 2, p.xq_pitch,
                             p.xs + row * p.xs_pitch + at, p.xs_pitch);
            }
        } else {
            for (int i = threadIdx.x - 32; i < nt * (width >> 3); i += kThreads - 32) {
                const int t = i / (width >> 3), k = (i - t * (width >> 3)) * 8;
                *reinterpret_cast<uint4*>(p.xp + static_cast<int64_t>(t0 + t) * p.dp + k_lo + k) =
                    *reinterpret_cast<const uint4*>(xs + t * sh.xpitch + 2 * k);
            }
        }
    }
    __syncwarp();
    cluster_sync_all();   // no CTA leaves while its sums are being read
}

// ---------------------------------------------------------------- experts
// How the fp16 weights of the any-stride kernel lie: contracted axis contiguous,
// the other one contiguous (rows that start at any element in both), or neither.
enum { kF16Rows = 0, kF16Cols = 1, kF16Strided = 2 };

// What a warp does at once.  A step is kVals of K for kTiles 16-row tiles, 2 KB
// of fp16 (64-byte pieces of global rows at least).
template <int kFmt, bool kUp>
struct Step {
    static constexpr int kTiles = kFmt == kF16Cols ? (kUp ? 4 : 2) : 1;
    static constexpr int kVals = kFmt == kF16Cols ? (kUp ? 16 : 32) : 64;
    static constexpr int kOut = (kUp ? 8 : 16) * kTiles;   // hidden values, or columns of y, of a unit
    static constexpr int kWords = kVals / 8;               // 32-bit words of a column a thread holds
};
constexpr int kStepBytes = 2560;   // a stage: 2 KB in place, and the words that hold them before

// A step of one projection (down) or of two (up: w0 the gate, w1 the up rows);
// outputs o0 .., values k0 ..; outputs from `rows` and values from K on are zeros.
//   kF16Rows/kF16Strided: 16 rows of 64 values, word c of row r at c ^ 4 (r & 1);
//     a pair's rows 0-7 are the gate's, 8-15 the up projection's.
//   kF16Cols: rows of K; up: 16 of 32 gate and 32 up outputs, down: 32 of 32
//     outputs.  Two down rows k, k + 16 share 128 bytes.
// Rows that start anywhere come in two moves: the aligned 16-byte words that
// hold a run of neighbouring values, one more than they fill, go to the stage
// asynchronously (fetch_stage); once there, a shift puts them in place (align_stage).
// Where a unit's weights begin: what changes with the expert and the outputs alone.
struct Origin {
    uintptr_t a0, a1;         // output o0, value 0 of w0 and of w1
    int64_t pitch0, pitch1;   // bytes from one row to the next
    int left;                 // outputs from o0 on
};

template <int kFmt>
__device__ __forceinline__ Origin origin(const Weight& w0, const Weight& w1, int e, int o0, int rows)
{
    auto at = [&](const Weight& w) {
        return reinterpret_cast<uintptr_t>(w.data) + 2 * (e * w.se + o0 * (kFmt == kF16Cols ? int64_t(1) : w.so));
    };
    return {at(w0), at(w1), 2 * (kFmt == kF16Cols ? w0.si : w0.so), 2 * (kFmt == kF16Cols ? w1.si : w1.so), rows - o0};
}

template <int kFmt, bool kUp>
struct Run {
    static constexpr int kWords = kFmt == kF16Cols ? 4 : 8;   // words of a run
    uintptr_t at;   // of the run's first value
    int n;          // its values in range, possibly more than it has
    __device__ Run(const Origin& b, int k0, int K, int run)
    {
        if (kFmt == kF16Cols) {
            const int half = run & 1, k = k0 + (run >> 1) + (!kUp && half ? 16 : 0);
            at = kUp && half ? b.a1 + k * b.pitch1 : b.a0 + k * b.pitch0;
            n = k < K ? b.left : 0;
        } else {
            const int o = kUp ? run & 7 : run;
            at = (kUp && run >= 8 ? b.a1 + o * b.pitch1 : b.a0 + o * b.pitch0) + 2 * k0;
            n = o < b.left ? K - k0 : 0;
        }
    }
};

// Where word c of stage row r lies.
template <int kFmt>
__device__ __forceinline__ uint32_t stage_word(int r, int c)
{
    return r * 128 + ((kFmt == kF16Cols ? c ^ (((r >> 2) << 1) | (r & 1)) : c ^ ((r & 1) << 2)) << 4);
}

template <int kFmt, bool kUp>
__device__ __forceinline__ void fetch_stage(uint32_t dst, const Origin& b, const Weight& w0, const Weight& w1, int k0, int K,
                                            int lane)
{
    if constexpr (kFmt == kF16Strided) {   // no neighbouring values: element by element, to their places
        const int c = lane & 7, k = k0 + 8 * c;
#pragma unroll 2
        for (int j = 0; j < 4; ++j) {
            const int r = (lane >> 3) + 4 * j, o = kUp ? r & 7 : r;
            const bool second = kUp && j >= 2;
            const __half* row = reinterpret_cast<const __half*>(second ? b.a1 + o * b.pitch1 : b.a0 + o * b.pitch0);
            const int64_t step = (second ? w1 : w0).si;
            uint32_t u[4] = {};
            if (o < b.left) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (k + i < K) u[i >> 1] |= static_cast<uint32_t>(ld_nc_u16(row + (k + i) * step)) << (16 * (i & 1));
            }
            st_smem_v4(dst + stage_word<kFmt>(r, c), make_uint4(u[0], u[1], u[2], u[3]));
        }
    } else {
        constexpr int kWords = Run<kFmt, kUp>::kWords + 1, kAll = 128 / (kWords - 1) * kWords;
#pragma unroll
        for (int j = 0; j < (kAll + 31) / 32; ++j) {
            const int i = lane + 32 * j;
            if (kAll % 32 && i >= kAll) break;
            const int run = i / kWords, word = i - run * kWords;
            const Run<kFmt, kUp> v(b, k0, K, run);
            const int bytes = 2 * min(v.n, 8 * (kWords - 1));
            const bool holds = bytes > 0 && 16 * word < static_cast<int>(v.at & 15u) + bytes;
            const uintptr_t src = (holds ? v.at + 16 * word : b.a0) & ~uintptr_t(15);
            cp_async16(dst + i * 16, reinterpret_cast<const void*>(src), holds ? 16u : 0u);
        }
        cp_async_commit();
    }
}

template <int kFmt, bool kUp>
__device__ __forceinline__ void align_stage(uint32_t stage, const Origin& b, int k0, int K, int lane)
{
    if constexpr (kFmt != kF16Strided) {
        constexpr int kWords = Run<kFmt, kUp>::kWords;
        const int c = lane & 7;
        uint32_t u[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = (lane >> 3) + 4 * j, run = kWords == 8 ? r : 2 * r + (c >> 2), word = c & (kWords - 1);
            const Run<kFmt, kUp> v(b, k0, K, run);
            const uint32_t from = stage + (run * (kWords + 1) + word) * 16;
            const uint4 lo = ld_smem_v4(from), hi = ld_smem_v4(from + 16);
            const uint32_t in[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            mxf4_dev::funnel16(in, static_cast<uint32_t>(v.at) & 15u, u[j]);
            if (v.n < 8 * (word + 1)) mxf4_dev::mask_tail<__half>(u[j], v.n - 8 * word);
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
            st_smem_v4(stage + stage_word<kFmt>((lane >> 3) + 4 * j, c), make_uint4(u[j][0], u[j][1], u[j][2], u[j][3]));
    }
    __syncwarp();
}

// Four 8x8 pieces, each transposed: operand registers of a 16-row tile from
// stage rows of K.
__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t* a)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(addr)
                 : "memory");
}

// A thread's words of one column: the values 8c .. 8c + 7 of each 32, or with
// 16 values a step 4c .. 4c + 3.
template <int kVals>
__device__ __forceinline__ void load_column(const __half* col, int k0, int end, bool on, uint32_t* b)
{
    if constexpr (kVals == 16) {
        uint2 v = make_uint2(0, 0);
        if (on && k0 < end)
            asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(col + k0));
        b[0] = v.x, b[1] = v.y;
    } else {
#pragma unroll
        for (int h = 0; h < kVals / 32; ++h) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (on && k0 + 32 * h < end)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                             : "l"(col + k0 + 32 * h));
            b[4 * h] = v.x, b[4 * h + 1] = v.y, b[4 * h + 2] = v.z, b[4 * h + 3] = v.w;
        }
    }
}

// acc[tile][group] += the stage's rows times the step's values of the columns.
template <int kFmt, bool kUp, int kGroups>
__device__ __forceinline__ void mma_stage(float (*acc)[kGroups][4], uint32_t src, const uint32_t (*b)[Step<kFmt, kUp>::kWords],
                                          int groups, int lane)
{
    const int g = lane >> 2, c = lane & 3;
    if (kFmt == kF16Rows || kFmt == kF16Strided) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = src + g * 128 + (((4 * h + c) ^ ((g & 1) << 2)) << 4);
            const uint4 lo = ld_smem_v4(at), hi = ld_smem_v4(at + 8 * 128);
#pragma unroll
            for (int q = 0; q < kGroups; ++q) {
                if (q < groups) {
                    mma16816(acc[0][q], lo.x, hi.x, lo.y, hi.y, b[q][4 * h], b[q][4 * h + 1]);
                    mma16816(acc[0][q], lo.z, hi.z, lo.w, hi.w, b[q][4 * h + 2], b[q][4 * h + 3]);
                }
            }
        }
    } else if (kFmt == kF16Cols && kUp) {
        // row 4 (j / 2) + j % 2 of K is row j of a piece, 2 rows on the same of
        // the second half of K; pieces in operand order: gate, up, gate, up
        const int j = lane & 7, piece = lane >> 3;
        const int r = 4 * (j >> 1) + (j & 1) + 2 * (piece >> 1);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            uint32_t a[4];
            ldmatrix_trans(src + r * 128 + (((t + 4 * (piece & 1)) ^ j) << 4), a);
#pragma unroll
            for (int q = 0; q < kGroups; ++q)
                if (q < groups) mma16816(acc[t][q], a[0], a[1], a[2], a[3], b[q][0], b[q][1]);
        }
    } else {
        // row 8 (j / 2) + j % 2 + 2m of 32 is row j of the m-th quarter of K; K
        // rows from 16 on are the upper words of the stage's rows
        const int j = lane & 7, piece = lane >> 3;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int k = 8 * (j >> 1) + (j & 1) + 4 * m + 2 * (piece >> 1), r = k & 15;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t a[4];
                const int word = 2 * t + (piece & 1) + (k >= 16 ? 4 : 0);
                ldmatrix_trans(src + r * 128 + ((word ^ (((r >> 2) << 1) | (r & 1))) << 4), a);
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    if (q < groups) mma16816(acc[t][q], a[0], a[1], a[2], a[3], b[q][2 * m], b[q][2 * m + 1]);
            }
        }
    }
}

// What a piece of an expert's work is: up to 8 * kGroups tokens of one expert
// (an expert with more is read once for each such piece).
struct Item {
    uint16_t expert, first, count;   // first: place in the list of choices ordered by expert
};

// The choices ordered by expert, in shared memory.
struct Choices {
    uint16_t slot[kMaxSlots];        // choices (token * top + j) ordered by expert, then by token
    float weight[kMaxSlots];         // their routing weights
    Item item[kMaxSlots];
    uint16_t first_of[kMaxExperts];
    uint32_t scan[kWarps];
    int items;
};

// Fills `ch` with pieces of `cap` tokens at most; `wcount`: room for 16 x E
// counts.  A counting sort by all kThreads threads of a CTA: each slot's rank
// within its warp by matching, then the warps' counts of each expert in turn,
// so that the order is that of the slots.  Ends with a barrier.
__device__ __forceinline__ void order_choices(const Params& p, Choices& ch, uint16_t* wcount, int cap)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int slots = p.T * p.top, nw = (slots + 31) >> 5;
    for (int i = threadIdx.x; i < nw * p.E; i += kThreads) wcount[i] = 0;
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
    const int pieces = (count + cap - 1) / cap;
    uint32_t sum = static_cast<uint32_t>(count) << 16 | pieces;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const uint32_t o = __shfl_up_sync(~0u, sum, s);
        if (lane >= s) sum += o;
    }
    if (lane == 31) ch.scan[warp] = sum;
    __syncthreads();
    uint32_t base = 0;
    for (int w = 0; w < warp; ++w) base += ch.scan[w];
    sum += base;
    const int first = static_cast<int>(sum >> 16) - count, piece0 = static_cast<int>(sum & 0xFFFFu) - pieces;
    if (ex < p.E) {
        ch.first_of[ex] = static_cast<uint16_t>(first);
        for (int i = 0; i < pieces; ++i)
            ch.item[piece0 + i] = Item{static_cast<uint16_t>(ex), static_cast<uint16_t>(first + i * cap),
                                       static_cast<uint16_t>(min(cap, count - i * cap))};
    }
    if (threadIdx.x == kThreads - 1) ch.items = static_cast<int>(sum & 0xFFFFu);
    __syncthreads();
    if (mine) {
        const int at = ch.first_of[e] + wcount[warp * p.E + e] + before;
        ch.slot[at] = static_cast<uint16_t>(threadIdx.x);
        ch.weight[at] = p.weights[threadIdx.x];
    }
    __syncthreads();
}

// All experts of the layer for fp16 weights at strides that TMA cannot address:
// the chosen experts are read by vector loads that a shift puts in place (or by
// elements, with no unit stride) into the same products.  Two phases, gate/up and down, each cut into
// gridDim parts of equal bytes; a CTA takes a part by ticket and, before it
// starts on a down part, waits until every gate/up part is done.  Tickets of
// gate/up parts are taken by running CTAs only and are all gone before any CTA
// waits, so the wait ends whichever CTAs the device holds at once.  A down
// part's first weights are on their way before the wait.
//
// A down unit is a range of columns and one of `splits` shares of the experts'
// K; with more than one share the sums go to the workspace, and the CTA that
// finishes a column range last adds the shares in order.
template <int kFmt, int kGroups, int kRing>
__global__ void __launch_bounds__(kThreads, 1) moe_experts(const __grid_constant__ Params p)
{
    using Up = Step<kFmt, true>;
    using Down = Step<kFmt, false>;
    constexpr int kBytes = kStepBytes;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Choices sh;
    __shared__ int ticket_slot, last_flag, wait_ok;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * (kRing * kBytes);
    uint8_t* tail = smem + kWarps * kRing * kBytes;   // sums: gate/up [2][16][groups][32] float4, down [16][T][kOut]
    const int parts = gridDim.x;

    griddep_wait();
    griddep_launch_dependents();

    if (threadIdx.x == 0) ticket_slot = atomicAdd(&p.ctl->ticket_up, 1);
    order_choices(p, sh, reinterpret_cast<uint16_t*>(smem), 8 * kGroups);
    const int items = sh.items;
    int ticket = ticket_slot;

    // ---- gate and up: a unit is one piece's next kOut hidden values, K dealt to the warps
    {
        constexpr int kVals = Up::kVals, kTiles = Up::kTiles, kWords = Up::kWords;
        const int units_each = p.fp / Up::kOut, steps = (p.D + kVals - 1) / kVals;
        const int wsteps = (steps - warp + kWarps - 1) / kWarps;   // this warp's steps of a unit
        uint32_t turn = 0;
        while (ticket < parts) {
            const int64_t all = static_cast<int64_t>(items) * units_each;
            const int u_lo = static_cast<int>(all * ticket / parts), u_hi = static_cast<int>(all * (ticket + 1) / parts);
            const int mine = (u_hi - u_lo) * wsteps;   // steps of this warp in all
            int pu = u_lo, ps = 0;                     // the next one to load
            auto begin = [&](int u) {
                const int it = u / units_each;
                return origin<kFmt>(p.gate, p.up, sh.item[it].expert, (u - it * units_each) * Up::kOut, p.F);
            };
            Origin ahead = {};
            auto issue = [&](int n) {
                if (n < mine) {
                    if (ps == 0) ahead = begin(pu);
                    fetch_stage<kFmt, true>(ring + (n % kRing) * kBytes, ahead, p.gate, p.up, (warp + ps * kWarps) * kVals, p.D,
                                            lane);
                    if (++ps == wsteps) ps = 0, ++pu;
                } else {
                    cp_async_commit();
                }
            };
            for (int n = 0; n < kRing - 1; ++n) issue(n);
            int n = 0;
            for (int u = u_lo; u < u_hi; ++u) {
                const int it = u / units_each, f0 = (u - it * units_each) * Up::kOut;
                const Item im = sh.item[it];
                const Origin here = begin(u);
                const int groups = (im.count + 7) >> 3;
                const __half* col[kGroups];
#pragma unroll
                for (int q = 0; q < kGroups; ++q)
                    col[q] = p.xp + static_cast<int64_t>(sh.slot[im.first + min(8 * q + g, im.count - 1)] / p.top) * p.dp +
                             (kVals == 16 ? 4 : 8) * c;
                float acc[kTiles][kGroups][4] = {};
                for (int s = 0; s < wsteps; ++s, ++n) {
                    uint32_t b[kGroups][kWords];
#pragma unroll
                    for (int q = 0; q < kGroups; ++q)
                        load_column<kVals>(col[q], (warp + s * kWarps) * kVals, p.dp, q < groups, b[q]);
                    cp_async_wait<kRing - 2>();
                    __syncwarp();   // (and every lane is done with the stage that is filled next)
                    align_stage<kFmt, true>(ring + (n % kRing) * kBytes, here, (warp + s * kWarps) * kVals, p.D, lane);
                    issue(n + kRing - 1);
                    mma_stage<kFmt, true, kGroups>(acc, ring + (n % kRing) * kBytes, b, groups, lane);
                }
#pragma unroll
                for (int t = 0; t < kTiles; ++t) {
                    float4* sums = reinterpret_cast<float4*>(tail) + (turn & 1) * (kWarps * kGroups * 32);
#pragma unroll
                    for (int q = 0; q < kGroups; ++q)
                        if (q < groups)
                            sums[(warp * kGroups + q) * 32 + lane] =
                                make_float4(acc[t][q][0], acc[t][q][1], acc[t][q][2], acc[t][q][3]);
                    __syncthreads();
                    // one warp a group adds the 16 parts; the warps take turns
                    const int q = static_cast<int>((warp - turn * kGroups) % kWarps);
                    ++turn;
                    if (q < groups) {
                        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                        for (int w = 0; w < kWarps; ++w) {
                            const float4 a = sums[(w * kGroups + q) * 32 + lane];
                            v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
                        }
                        const int f = f0 + 8 * t + g;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = 8 * q + 2 * c + i;
                            if (j < im.count) {
                                // (past F: zeros, whatever the tokens hold)
                                const float hv = f < p.F ? act_f32(p.act, i ? v.y : v.x) * (i ? v.w : v.z) : 0.f;
                                __half* dst = p.hp + static_cast<int64_t>(im.first + j) * 2 * p.fp + f;
                                split_hidden(hv, dst, dst + p.fp);
                            }
                        }
                    }
                }
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                if (!p.test_stall) atom_add_acq_rel_gpu(&p.ctl->done_up, 1);
                ticket_slot = atomicAdd(&p.ctl->ticket_up, 1);
            }
            __syncthreads();
            ticket = ticket_slot;
        }
    }

    // ---- down: a warp takes a range of a unit's (piece, step) pairs and keeps
    // its own weighted sums of the tokens
    if (threadIdx.x == 0) ticket_slot = atomicAdd(&p.ctl->ticket_down, 1);
    __syncthreads();
    ticket = ticket_slot;
    constexpr int kVals = Down::kVals, kTiles = Down::kTiles, kWords = Down::kWords, kOut = Down::kOut;
    constexpr int kCols = 2 * kGroups;   // groups of 8 columns: a choice takes two (high and low half)
    const int tiles = (p.D + kOut - 1) / kOut, fsteps = (p.F + kVals - 1) / kVals;
    const int total = items * fsteps, units = tiles * p.splits;
    float* ysum = reinterpret_cast<float*>(tail);
    float* mysum = ysum + warp * p.T * kOut;
    auto share = [&](int unit, int* lo, int* hi) {   // this warp's pairs
        const int w = (unit % p.splits) * kWarps + warp, n = p.splits * kWarps;
        *lo = static_cast<int>(static_cast<int64_t>(total) * w / n);
        *hi = static_cast<int>(static_cast<int64_t>(total) * (w + 1) / n);
    };
    bool waited = false;
    while (ticket < parts) {
        const int u_lo = static_cast<int>(static_cast<int64_t>(units) * ticket / parts),
                  u_hi = static_cast<int>(static_cast<int64_t>(units) * (ticket + 1) / parts);
        int pu = u_lo, pi = 0, pend = 0, pk = -1;   // pk: step of the item, -1 before the unit's first
        if (u_lo < u_hi) share(u_lo, &pi, &pend);
        auto begin = [&](int it, int unit) {
            return origin<kFmt>(p.down, p.down, sh.item[it].expert, unit / p.splits * kOut, p.D);
        };
        Origin ahead = {};
        auto issue = [&](int n) {
            while (pu < u_hi && pi == pend) {
                pk = -1;
                if (++pu < u_hi) share(pu, &pi, &pend);
            }
            if (pu < u_hi) {
                if (pk < 0 || pk == fsteps) {
                    const int it = pi / fsteps;
                    pk = pi - it * fsteps;
                    ahead = begin(it, pu);
                }
                fetch_stage<kFmt, false>(ring + (n % kRing) * kBytes, ahead, p.down, p.down, pk * kVals, p.F, lane);
                ++pi, ++pk;
            } else {
                cp_async_commit();
            }
        };
        for (int n = 0; n < kRing - 1; ++n) issue(n);
        for (int i = threadIdx.x; i < kWarps * p.T * kOut; i += kThreads) ysum[i] = 0.f;
        if (!waited) {
            if (threadIdx.x == 0) {
                const uint64_t t0 = globaltimer_ns();
                wait_ok = 1;
                while (ld_acquire_gpu(&p.ctl->done_up) < parts) {
                    if (globaltimer_ns() - t0 > p.timeout_ns) {
                        wait_ok = 0;
                        atomicExch(p.status, GEMM_F16_ERR_TIMEOUT);
                        break;
                    }
                }
            }
            waited = true;
        }
        __syncthreads();
        if (!wait_ok) break;
        int n = 0;
        for (int unit = u_lo; unit < u_hi; ++unit) {
            int lo, hi;
            share(unit, &lo, &hi);
            int it = -1, k = fsteps;   // item, the step within it
            Item im = {};
            Origin here = {};
            int groups = 0;
            const __half* col[kCols];
            float acc[kTiles][kCols][4];
            auto flush = [&]() {
#pragma unroll
                for (int q = 0; q < kCols; ++q) {
                    const int j = 4 * q + c;   // this thread's columns are the halves of choice j
                    if (j < im.count) {
                        const float w = sh.weight[im.first + j];
                        float* to = mysum + sh.slot[im.first + j] / p.top * kOut;
#pragma unroll
                        for (int t = 0; t < kTiles; ++t) {
                            to[16 * t + g] = fmaf(w, join_hidden(acc[t][q][0], acc[t][q][1]), to[16 * t + g]);
                            to[16 * t + g + 8] = fmaf(w, join_hidden(acc[t][q][2], acc[t][q][3]), to[16 * t + g + 8]);
                        }
                    }
                }
                __syncwarp();
            };
            for (int i = lo; i < hi; ++i, ++n, ++k) {
                if (k == fsteps) {
                    if (it >= 0) flush();
                    it = i / fsteps;
                    k = i - it * fsteps;
                    im = sh.item[it];
                    here = begin(it, unit);
                    groups = (2 * im.count + 7) >> 3;
#pragma unroll
                    for (int q = 0; q < kCols; ++q) {
                        const int j = im.first + min(4 * q + (g >> 1), im.count - 1);
                        col[q] = p.hp + (static_cast<int64_t>(j) * 2 + (g & 1)) * p.fp + 8 * c;
#pragma unroll
                        for (int t = 0; t < kTiles; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[t][q][e] = 0.f;
                    }
                }
                uint32_t b[kCols][kWords];
#pragma unroll
                for (int q = 0; q < kCols; ++q)
                    load_column<kVals>(col[q], k * kVals, p.fp, q < groups, b[q]);
                cp_async_wait<kRing - 2>();
                __syncwarp();   // (and every lane is done with the stage that is filled next)
                align_stage<kFmt, false>(ring + (n % kRing) * kBytes, here, k * kVals, p.F, lane);
                issue(n + kRing - 1);
                mma_stage<kFmt, false, kCols>(acc, ring + (n % kRing) * kBytes, b, groups, lane);
            }
            if (it >= 0) flush();
            __syncthreads();
            const int tile = unit / p.splits;
            for (int i = threadIdx.x; i < p.T * kOut; i += kThreads) {
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    v += ysum[w * p.T * kOut + i];
                    ysum[w * p.T * kOut + i] = 0.f;
                }
                const int t = i / kOut, d = tile * kOut + i % kOut;
                if (d < p.D) {
                    if (p.splits == 1)
                        p.y[t * p.ldy + d] = __float2half_rn(v);
                    else
                        p.parts[(static_cast<int64_t>(unit % p.splits) * p.T + t) * p.dp + d] = v;
                }
            }
            __syncthreads();
            if (p.splits > 1) {
                if (threadIdx.x == 0) last_flag = atom_add_acq_rel_gpu(&p.counts[tile], 1) == p.splits - 1;
                __syncthreads();
                if (last_flag) {
                    for (int i = threadIdx.x; i < p.T * kOut; i += kThreads) {
                        const int t = i / kOut, d = tile * kOut + i % kOut;
                        if (d >= p.D) continue;
                        float v = 0.f;
                        for (int s = 0; s < p.splits; ++s) v += ld_cg_f32(p.parts + (static_cast<int64_t>(s) * p.T + t) * p.dp + d);
                        p.y[t * p.ldy + d] = __float2half_rn(v);
                    }
                }
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) ticket_slot = atomicAdd(&p.ctl->ticket_down, 1);
        __syncthreads();
        ticket = ticket_slot;
    }
}

}  // namespace moe_dev
