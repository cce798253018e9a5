// Root-mean-square norm of rows, with a residual added before and an output in 8 bits.
//
//   h = x + residual (rounded to their type: what the next layer adds to)
//   y = h / sqrt(mean(h^2) + eps) * weight, rounded once, to their type or to 8 bits
//
// Bound by HBM: a row is read once, kept in registers over the sum of its squares
// (fp32: eight values a lane in order, then a tree), and written once.  Sixteen lanes
// hold a block of 128 values, so the 8-bit form's scales are four shuffles away.
#pragma once

#include "fp8_format.cuh"
#include "rows.cuh"

namespace norm_dev {

using namespace gemm_f16_dev;

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

// A row takes kThreads threads of kVecs x 8 values each; a block of 256 threads (or
// more, where a row takes more) has 256 / kThreads rows.
template <typename T, int kThreads, int kVecs, bool kVec>
__global__ void __launch_bounds__(kThreads < 256 ? 256 : kThreads) rms_norm(const Params p)
{
    constexpr int kBlock = kThreads < 256 ? 256 : kThreads, kWarps = kThreads / 32;
    __shared__ float part[kBlock / 32];
    const int t = threadIdx.x % kThreads;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kBlock / kThreads) + threadIdx.x / kThreads;
    const bool in = row < p.rows;   // (of whole warps, and of whole blocks where a row takes more than one)
    const int64_t d = in ? p.d : 0;
    griddep_wait();
    griddep_launch_dependents();

    uint32_t h[kVecs][4];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) row_dev::load8<kVec>(p.x + row * p.sx, (v * kThreads + t) * 8, d, h[v]);
    if (p.residual) {
        uint32_t r[kVecs][4];
#pragma unroll
        for (int v = 0; v < kVecs; ++v) row_dev::load8<kVec>(p.residual + row * p.sr, (v * kThreads + t) * 8, d, r[v]);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float2 a = row_dev::widen2<T>(h[v][c]), b = row_dev::widen2<T>(r[v][c]);
                h[v][c] = row_dev::narrow2<T>(a.x + b.x, a.y + b.y);
            }
            row_dev::store8<kVec>(p.sum + row * p.ss, (v * kThreads + t) * 8, d, h[v]);
        }
    }
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 a = row_dev::widen2<T>(h[v][c]);
            s = fmaf(a.x, a.x, s);
            s = fmaf(a.y, a.y, s);
        }
#pragma unroll
    for (int k = 16; k; k /= 2) s += __shfl_xor_sync(~0u, s, k);
    if (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
        __syncthreads();
        s = part[(threadIdx.x & 31) % kWarps];
#pragma unroll
        for (int k = kWarps / 2; k; k /= 2) s += __shfl_xor_sync(~0u, s, k);
    }
    const float r = 1.f / sqrtf(s / static_cast<float>(p.d) + p.eps);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int i = (v * kThreads + t) * 8;
        uint32_t w[4];
        row_dev::load8<kVec>(p.weight, i, p.d, w);
        float y[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float2 a = row_dev::widen2<T>(h[v][c]), b = row_dev::widen2<T>(w[c]);
            y[2 * c] = a.x * r * b.x, y[2 * c + 1] = a.y * r * b.y;
        }
        if (p.y) {
            uint32_t o[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) o[c] = row_dev::narrow2<T>(y[2 * c], y[2 * c + 1]);
            row_dev::store8<kVec>(p.y + row * p.sy, i, d, o);
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                if (i + c >= p.d) y[c] = 0.f;   // (an infinite r times nothing)
                top = max(top, __float_as_uint(y[c]) & 0x7FFFFFFFu);
            }
#pragma unroll
            for (int k = 1; k < 16; k *= 2) top = max(top, __shfl_xor_sync(~0u, top, k));
            const uint32_t code = fp8_dev::scale_code<float>(top);
            const uint2 q = fp8_dev::codes8<float>(reinterpret_cast<const uint32_t*>(y), code);
            if (in && i + 8 <= p.pitch) *reinterpret_cast<uint2*>(p.codes + row * p.pitch + i) = q;
            if (in && (t & 15) == 0 && i < p.d)
                p.scales[fp8_dev::scale_at(row, i >> 7, p.kt)] = static_cast<uint8_t>(code);
        }
    }
    if (!p.y) {   // the scale tiles' padding: blocks past the row's, rows past the last
        const int64_t blocks = (p.d + 127) >> 7;
        if (in && t < 4 * p.kt - blocks) p.scales[fp8_dev::scale_at(row, blocks + t, p.kt)] = 0;
        if (row == p.rows - 1)
            for (int64_t q = p.rows; q < p.row_tiles * 128; ++q)
                for (int64_t b = t; b < 4 * p.kt; b += kThreads) p.scales[fp8_dev::scale_at(q, b, p.kt)] = 0;
    }
}

}  // namespace norm_dev
