// Root-mean-square norm of rows, with a residual added before and an output in 8 bits.
//
//   h = x + residual (rounded to their type: what the next layer adds to)
//   y = h / sqrt(mean(h^2) + eps) * weight, rounded once, to their type or to 8 bits
//
// Bound by HBM: a row is read once, kept in registers over the sum of its squares
// (fp32), and written once.  Sixteen lanes
// hold a block of 128 values, so the 8-bit form's scales are four shuffles away.
//
// 131072 x 7168 in fp16 with a residual: 1055 us (7.1 TB/s), to 8 bits 917 us (7.2); without
// one 546 us (6.9).  Rows that start anywhere: 32768 x 4097 in bf16 with a residual 234 us
// (4.6), by issue (the shifts of 16 bytes).
#pragma once

#include "activation.cuh"
#include "fp8_format.cuh"
#include "rows.cuh"

namespace norm_dev {

using namespace gemm_f16_dev;
using fp8_dev::Bool;
using mxf4_dev::Elem;

using mxf4_dev::fma2;
using mxf4_dev::mul2;
using mxf4_dev::pack2;
using mxf4_dev::unpack2;

// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

struct Params {
    const uint16_t* x;
    const uint16_t* residual;   // null: none
    const uint16_t* weight;
    uint16_t* sum;              // h; null without a residual
    uint16_t* y;                // null: codes and scales
    uint8_t* codes;
    uint8_t* scales;
    int64_t sx, sr, ss, sy;     // row strides in elements
    int64_t rows, d, pitch, kt, row_tiles;
    float eps;
};

// bf16 reaches further than its squares do in fp32: they are infinite from 2^64 on, and
// below 2^-63 lose bits.  A row whose squares' sum is infinite, or whose mean square with eps
// is below 2^-90 (more than 2^45 as a factor), is done here once more, `f` times as large,
// 2^80 or 2^-80: bound by latency, out of the way of the others' registers.  By whole warps,
// each of which sums up all of the row, so that the sum has one order here, too (at most 69
// roundings of it); then every warp takes blocks of 128 values and writes over what the
// kernel gave them.  That and h have been written, and the writes are visible to the warp.
template <typename T, int kMost>
__device__ __forceinline__ void far_row(const Params& p, float f)
{
    constexpr bool kWarpRow = kMost == 256;
    const int lane = threadIdx.x & 31, d = static_cast<int>(p.d);
    const int warp = kWarpRow ? 0 : threadIdx.x >> 5, warps = kWarpRow ? 1 : blockDim.x >> 5;
    const int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kMost / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.rows) return;
    const uint16_t* h = p.residual ? p.sum + row * p.ss : p.x + row * p.sx;
    auto value = [](const uint16_t* at) { return Elem<T>::to_f32(*at); };
    float s = 0.f;
#pragma unroll 1
    for (int i0 = 0; i0 < d; i0 += 1024) {
        float some = 0.f;
#pragma unroll 1
        for (int i = i0 + lane; i < min(d, i0 + 1024); i += 32) some = fmaf(value(h + i) * f, value(h + i) * f, some);
        s += some;
    }
#pragma unroll
    for (int k = 16; k; k /= 2) s += __shfl_xor_sync(~0u, s, k);
    const float r = 1.f / sqrtf(s / static_cast<float>(d) + p.eps * f * f);
    // f h is exact where f is large, and r f may be past fp32 there; where f is small h
    // keeps its small values, and r f has 21 bits at least
    const float fh = f > 1.f ? f : 1.f, fr = f > 1.f ? r : r * f;
    const int end = static_cast<int>(p.y ? p.d : p.pitch);
#pragma unroll 1
    for (int i = warp * 128 + lane * 4; i - lane * 4 < end; i += warps * 128) {
        float y[4], top = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            y[c] = i + c < d ? value(h + i + c) * fh * fr * value(p.weight + i + c) : 0.f;
            top = max_nan(top, fabsf(y[c]));
        }
        if (p.y) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (i + c < d) p.y[row * p.sy + i + c] = static_cast<uint16_t>(row_dev::narrow2<T>(y[c], 0.f));
            continue;
        }
#pragma unroll
        for (int k = 16; k; k /= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, k));
        const uint32_t code = fp8_dev::scale_code_f32(top);
        const float g = code == 255u ? 0.f : fp8_dev::inverse_scale(code);
        *reinterpret_cast<uint32_t*>(p.codes + row * p.pitch + i) =
            code == 255u ? 0u : fp8_dev::e4m3_of(y[0] * g, y[1] * g, y[2] * g, y[3] * g);
        if (lane == 0) p.scales[fp8_dev::scale_at(row, i >> 7, p.kt)] = static_cast<uint8_t>(code);
    }
}

// As a call, for two forms that are slower with it inside: of rows past 9216 values (68
// registers a thread instead of 64 are a block less of three an SM: 4882 x 12288 44 us, 54 so)
// and of 257 to 512 (117187 x 512 to 8 bits 44.8 us, 48.4 so).  In the others a call costs more:
// it takes 40 registers, and rows of up to 256 values, whose form has 32, a fifth longer.
// Over the kernel without far rows it is 1 to 4 %: 3001 x 4097 as it was, 16 x 4096 1.59 us, now 1.64.
template <typename T, int kMost>
__device__ __noinline__ void far_row_apart(const Params& p, float f)
{
    far_row<T, kMost>(p, f);
}

// kMost 256: a warp a row, eight rows a block.  Otherwise a block of at most kMost threads
// a row.  A thread takes kVecs times 8 values.
// (At least three blocks of the largest an SM for rows that start anywhere, three times
// eight values a thread: 32768 x 4097 in bf16 with a residual 233 us, 276 without.  The other
// forms were not measured with such a bound.)
template <typename T, int kMost, int kVecs, bool kVec>
__global__ void __launch_bounds__(kMost, kVecs == 3 && !kVec ? 3 : 0) rms_norm(const Params p)
{
    constexpr bool kWarpRow = kMost == 256;
    __shared__ float part[kVecs * kMost / 32];
    __shared__ uint4 edge[kVec ? 1 : kVecs * kMost / 32];
    const int threads = kWarpRow ? 32 : blockDim.x, warps = kWarpRow ? 1 : threads >> 5;
    const int t = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = kWarpRow ? static_cast<int64_t>(blockIdx.x) * (kMost / 32) + (threadIdx.x >> 5) : blockIdx.x;
    const bool in = row < p.rows;   // (of whole warps; a block's row always is)
    const int64_t d = in ? p.d : 0;
    griddep_wait();
    griddep_launch_dependents();

    // Where rows start anywhere a thread takes the values of 16 aligned bytes of x's row,
    // `lead` before a multiple of eight, where residual and sum mostly have theirs, too.
    // Then the values move to their multiples of eight, so that the sum of squares has
    // one order wherever the rows lie, and y's go back on their way out.
    const int lead = kVec ? 0 : row_dev::lead_of(p.x + row * p.sx);
    auto at = [&](int v, int before) { return (v * threads + t) * 8 - before; };

    // The values' neighbours: of the thread before (kNext: after), of a warp's end through
    // shared memory.  By all threads of a row.
    auto neighbours = [&](auto next, uint32_t (&w)[kVecs][4], uint32_t (&n)[kVecs][4]) {
        constexpr bool kNext = decltype(next)::value;
        const int lane = threadIdx.x & 31, first = kWarpRow ? (threadIdx.x >> 5) * kVecs : 0;   // of this row's edges
        if (!kWarpRow) __syncthreads();   // (the last edges have been read)
        if (lane == (kNext ? 0 : 31))
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                edge[first + v * warps + (t >> 5)] = make_uint4(w[v][0], w[v][1], w[v][2], w[v][3]);
        if (kWarpRow) __syncwarp();
        else __syncthreads();
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
#pragma unroll
            for (int c = 0; c < 4; ++c) n[v][c] = kNext ? __shfl_down_sync(~0u, w[v][c], 1) : __shfl_up_sync(~0u, w[v][c], 1);
            if (lane == (kNext ? 31 : 0)) {
                const int e = v * warps + (t >> 5) + (kNext ? 1 : -1);
                const uint4 x = e >= 0 && e < kVecs * warps ? edge[first + e] : make_uint4(0u, 0u, 0u, 0u);
                n[v][0] = x.x, n[v][1] = x.y, n[v][2] = x.z, n[v][3] = x.w;
            }
        }
        __syncwarp();
    };

    // Values that begin `from` before multiples of eight.
    auto store_row = [&](uint16_t* out, uint32_t (&w)[kVecs][4], int from) {
        const int o = kVec ? 0 : (row_dev::lead_of(out) - from) & 7;   // (the same in all of a row's threads, and a row of several warps is a block)
        if (o == 0) {
#pragma unroll
            for (int v = 0; v < kVecs; ++v) row_dev::store8<kVec>(out, at(v, from), d, w[v]);
        } else if constexpr (!kVec) {
            // 16 aligned bytes that end in the thread's own values
            uint32_t before[kVecs][4];
            neighbours(Bool<false>(), w, before);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                uint32_t mine[4];
                row_dev::take8(before[v], w[v], 8 - o, mine);
                const int i = at(v, from);
                row_dev::store8<false>(out, i - o, d, mine);
                // the last o of the last thread, where the row goes on to there
                if (v == kVecs - 1 && t == threads - 1 && i + 8 - o < d)
                    row_dev::store_some(out + i, w[v], 8 - o, static_cast<int>(min(static_cast<int64_t>(8), d - i)));
            }
        }
    };

    uint32_t h[kVecs][4];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) row_dev::load8<kVec>(p.x + row * p.sx, at(v, lead), d, h[v]);
    if (p.residual) {
        uint32_t r[kVecs][4];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) row_dev::load8<kVec>(p.residual + row * p.sr, at(v, lead), d, r[v]);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
#pragma unroll
            for (int c = 0; c < 4; ++c) h[v][c] = row_dev::add2<T>(h[v][c], r[v][c]);
        }
        store_row(p.sum + row * p.ss, h, lead);
    }
    if constexpr (!kVec) {
        uint32_t after[kVecs][4];
        neighbours(Bool<true>(), h, after);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            uint32_t mine[4];
            row_dev::take8(h[v], after[v], lead, mine);
#pragma unroll
            for (int c = 0; c < 4; ++c) h[v][c] = mine[c];
        }
    }
    // One order for every form and place: 256 values, eight a lane (even and odd ones apart),
    // by a warp's tree, then the sums of all such chunks by a tree over 32 lanes.
    float s = 0.f, chunk[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        uint64_t two = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 a = row_dev::widen2<T>(h[v][c]);
            const uint64_t both = pack2(a.x, a.y);
            two = fma2(both, both, two);
        }
        float even, odd;
        unpack2(two, &even, &odd);
        chunk[v] = even + odd;
#pragma unroll
        for (int k = 16; k; k /= 2) chunk[v] += __shfl_xor_sync(~0u, chunk[v], k);
    }
    if constexpr (kWarpRow) {
        s = kVecs == 4 ? (chunk[0] + chunk[kVecs / 2]) + (chunk[1 % kVecs] + chunk[3 % kVecs])
                       : kVecs == 2 ? chunk[0] + chunk[1 % kVecs] : chunk[0];
    } else {
        if ((t & 31) == 0)
#pragma unroll
            for (int v = 0; v < kVecs; ++v) part[v * warps + (t >> 5)] = chunk[v];
        __syncthreads();
        for (int k = t & 31; k < kVecs * warps; k += 32) s += part[k];
#pragma unroll
        for (int k = 16; k; k /= 2) s += __shfl_xor_sync(~0u, s, k);
    }
    const float r = 1.f / sqrtf(s / static_cast<float>(p.d) + p.eps);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int i = at(v, 0);
        uint32_t w[4];
        row_dev::load8<kVec>(p.weight, i, p.d, w);
        float y[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 a = row_dev::widen2<T>(h[v][c]), b = row_dev::widen2<T>(w[c]);
            unpack2(mul2(mul2(pack2(a.x, a.y), pack2(r, r)), pack2(b.x, b.y)), &y[2 * c], &y[2 * c + 1]);
        }
        if (p.y) {
#pragma unroll
            for (int c = 0; c < 4; ++c) h[v][c] = row_dev::narrow2<T>(y[2 * c], y[2 * c + 1]);
            if (kVec) row_dev::store8<true>(p.y + row * p.sy, i, d, h[v]);
        } else {
            if (i + 8 > p.d) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (i + c >= p.d) y[c] = 0.f;   // (an infinite r times nothing)
            }
            float top = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) top = max_nan(top, fabsf(y[c]));
#pragma unroll
            for (int k = 1; k < 16; k *= 2) top = max_nan(top, __shfl_xor_sync(~0u, top, k));
            const uint32_t code = fp8_dev::scale_code_f32(top);
            uint2 q = make_uint2(0u, 0u);
            if (code != 255u) {
                const float f = fp8_dev::inverse_scale(code);
#pragma unroll
                for (int c = 0; c < 8; c += 2) unpack2(mul2(pack2(y[c], y[c + 1]), pack2(f, f)), &y[c], &y[c + 1]);
                q = make_uint2(fp8_dev::e4m3_of(y[0], y[1], y[2], y[3]), fp8_dev::e4m3_of(y[4], y[5], y[6], y[7]));
            }
            if (in && i + 8 <= p.pitch) *reinterpret_cast<uint2*>(p.codes + row * p.pitch + i) = q;
            if (in && (t & 15) == 0 && i < p.d)
                p.scales[fp8_dev::scale_at(row, i >> 7, p.kt)] = static_cast<uint8_t>(code);
        }
    }
    if (p.y) {
        if (!kVec) store_row(p.y + row * p.sy, h, 0);
    } else {   // the scale tiles' padding: blocks past the row's, rows past the last
        const int64_t blocks = (p.d + 127) >> 7;
        if (in && t < 4 * p.kt - blocks) p.scales[fp8_dev::scale_at(row, blocks + t, p.kt)] = 0;
        if (row == p.rows - 1) {
            const int kt = static_cast<int>(p.kt), words = static_cast<int>(p.row_tiles * 128 - p.rows) * kt;
            for (int q = t; q < words; q += threads)
                *reinterpret_cast<uint32_t*>(p.scales + fp8_dev::scale_at(p.rows + q / kt, 4 * (q % kt), p.kt)) = 0u;
        }
    }
    if constexpr (Elem<T>::kInf == 0x7F80u) {
        // (here, so that nothing of the others' is held over it or waits behind it)
        if (!(r > 0.f && r <= 0x1p45f)) {   // (the same in all of a row's threads)
            if (kWarpRow) __syncwarp();
            else __syncthreads();
            const float f = r > 1.f ? 0x1p80f : 0x1p-80f;
            if constexpr (kMost == 832 || (kMost == 256 && kVecs == 2)) far_row_apart<T, kMost>(p, f);
            else far_row<T, kMost>(p, f);
        }
    }
}

}  // namespace norm_dev
