// MXFP4 quantisation and its inverse: pure streaming kernels, bound by HBM.
//
// Quantising reads 2 (fp16, bf16) or 4 bytes a value once and writes 17/32 of
// a byte; the arithmetic (a maximum, one multiply, one conversion a value)
// hides under the loads.  A block of threads takes a tile of 128 rows x 256
// values: the 128 rows fill whole 512-byte scale tiles, which are put together
// in shared memory and leave in one piece, and 256 values of a row are 128
// bytes of codes, one full line.
#pragma once

#include "mxf4_format.cuh"

namespace mxf4_dev {

constexpr int kTileRows = 128, kTileVals = 256, kConvThreads = 256;

struct QuantParams {
    const void* x;
    int64_t sb, sr, sk;   // element strides
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows, k, pitch;   // pitch: code bytes a row
    int64_t kt;               // scale tiles along k
    int64_t row_tiles;        // ceil(rows / 128)
    int64_t col_tiles;        // ceil(k / 256): blocks are numbered columns first
};

// 8 values of one row from `i` on as words of T (2 or 4 bytes a value), values
// from `k` on zero.  The row has unit stride; `vec` says its start and so every
// 8th value is 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t i, int64_t k, bool vec, uint32_t* w)
{
    constexpr int kWords = 8 * sizeof(T) / 4;
    if (vec && i + 8 <= k) {
#pragma unroll
        for (int c = 0; c < kWords / 4; ++c) {
            const uint4 v = ld_nc_v4(row + i + c * (16 / sizeof(T)));
            w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < kWords; ++c) w[c] = 0u;
    if (sizeof(T) == 4) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (i + c < k) w[c] = ld_nc_u32(row + i + c);
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (i + c < k) w[c >> 1] |= static_cast<uint32_t>(ld_nc_u16(row + i + c)) << (16 * (c & 1));
    }
}

// Unit stride along k: a warp takes the 256 values of one row, 8 a lane, so its
// loads and its 128 bytes of codes are contiguous; four lanes share a block.
template <typename T>
__global__ void __launch_bounds__(kConvThreads) quantize_rows(const QuantParams p)
{
    __shared__ __align__(16) uint8_t sc[2 * kScaleTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rt = blockIdx.x / p.col_tiles;
    const int64_t r0 = rt * kTileRows, i0 = (blockIdx.x - rt * p.col_tiles) * kTileVals;
    const int64_t b = blockIdx.z;
    const T* x = static_cast<const T*>(p.x) + b * p.sb;
    uint8_t* codes = p.codes + b * p.rows * p.pitch;
    uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    const bool vec = (reinterpret_cast<uintptr_t>(x) | (static_cast<uint64_t>(p.sr) * sizeof(T))) % 16 == 0;
    const int64_t i = i0 + lane * 8;
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kUnroll = sizeof(T) == 4 ? 2 : 4;
    constexpr int kWarps = kConvThreads / 32;
#pragma unroll 1
    for (int rr = warp; rr < kTileRows; rr += kWarps * kUnroll) {
        uint32_t w[kUnroll][8 * sizeof(T) / 4];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t r = r0 + rr + u * kWarps;
            load8<T>(x + r * p.sr, r < p.rows ? i : p.k, p.k, vec, w[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int lr = rr + u * kWarps;
            const int64_t r = r0 + lr;
            uint32_t top = top_bits<T>(w[u]);
            top = max(top, __shfl_xor_sync(~0u, top, 1));
            top = max(top, __shfl_xor_sync(~0u, top, 2));
            const bool in = r < p.rows && (i >> 5) < (p.k + 31) / 32;
            const uint32_t code = in ? scale_code<T>(top) : 0u;
            if (in) *reinterpret_cast<uint32_t*>(codes + r * p.pitch + (i >> 1)) = codes_of<T>(w[u], code);
            // lane / 4 is the block in the tile: four scale bytes of one row are one word
            uint32_t four = code << (8 * ((lane >> 2) & 3));
            four |= __shfl_xor_sync(~0u, four, 4);
            four |= __shfl_xor_sync(~0u, four, 8);
            if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(sc + (lane >> 4) * kScaleTile + (lr & 31) * 16 + (lr >> 5) * 4) = four;
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int t = threadIdx.x >> 5;   // of the two scale tiles
        const int64_t kt = (i0 >> 7) + t;
        if (kt < p.kt)
            reinterpret_cast<uint4*>(scales + (rt * p.kt + kt) * kScaleTile)[lane] =
                reinterpret_cast<const uint4*>(sc + t * kScaleTile)[lane];
    }
}

// Any strides (a transposed view has unit stride along the rows): a lane takes
// a row and a warp 32 neighbouring rows, so that a unit row stride gives
// contiguous loads; the codes of the tile are turned in shared memory.
template <typename T>
__global__ void __launch_bounds__(kConvThreads) quantize_strided(const QuantParams p)
{
    constexpr int kPitch = 128 + 16;   // bytes a row of the staged codes: 16-byte stores spread over the banks
    __shared__ __align__(16) uint8_t cs[kTileRows * kPitch];
    __shared__ __align__(16) uint8_t sc[2 * kScaleTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rt = blockIdx.x / p.col_tiles;
    const int64_t r0 = rt * kTileRows, i0 = (blockIdx.x - rt * p.col_tiles) * kTileVals;
    const int64_t b = blockIdx.z;
    const T* x = static_cast<const T*>(p.x) + b * p.sb;
    uint8_t* codes = p.codes + b * p.rows * p.pitch;
    uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    griddep_wait();
    griddep_launch_dependents();
    const int lr = (warp & 3) * 32 + lane;
    const int64_t r = r0 + lr;
#pragma unroll 1
    for (int blk = warp >> 2; blk < kTileVals / 32; blk += 2) {
        const int64_t i = i0 + blk * 32;
        uint32_t w[4][8 * sizeof(T) / 4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (unsigned c = 0; c < 8 * sizeof(T) / 4; ++c) w[q][c] = 0u;
            if (r >= p.rows) continue;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int64_t j = i + q * 8 + c;
                if (j >= p.k) continue;
                const T* src = x + r * p.sr + j * p.sk;
                if (sizeof(T) == 4)
                    w[q][c] = ld_nc_u32(src);
                else
                    w[q][c >> 1] |= static_cast<uint32_t>(ld_nc_u16(src)) << (16 * (c & 1));
            }
        }
        const uint32_t top = max(max(top_bits<T>(w[0]), top_bits<T>(w[1])), max(top_bits<T>(w[2]), top_bits<T>(w[3])));
        const uint32_t code = r < p.rows && i < p.k ? scale_code<T>(top) : 0u;
        uint4 c4;
        c4.x = codes_of<T>(w[0], code), c4.y = codes_of<T>(w[1], code);
        c4.z = codes_of<T>(w[2], code), c4.w = codes_of<T>(w[3], code);
        *reinterpret_cast<uint4*>(cs + lr * kPitch + blk * 16) = c4;
        sc[(blk >> 2) * kScaleTile + lane * 16 + (warp & 3) * 4 + (blk & 3)] = static_cast<uint8_t>(code);
    }
    __syncthreads();
    const int64_t bytes = min(p.pitch - (i0 >> 1), static_cast<int64_t>(128));
    for (int t = threadIdx.x; t < kTileRows * 8; t += kConvThreads) {
        const int row = t >> 3, c = t & 7;
        if (r0 + row < p.rows && c * 16 < bytes)
            *reinterpret_cast<uint4*>(codes + (r0 + row) * p.pitch + (i0 >> 1) + c * 16) =
                *reinterpret_cast<const uint4*>(cs + row * kPitch + c * 16);
    }
    if (threadIdx.x < 64) {
        const int t = threadIdx.x >> 5;
        const int64_t kt = (i0 >> 7) + t;
        if (kt < p.kt)
            reinterpret_cast<uint4*>(scales + (rt * p.kt + kt) * kScaleTile)[lane] =
                reinterpret_cast<const uint4*>(sc + t * kScaleTile)[lane];
    }
}

struct DequantParams {
    const uint8_t* codes;
    const uint8_t* scales;
    void* y;
    int64_t rows, k, pitch, kt, row_tiles;
};

// Eight values of a row, 16 (fp32: 32) contiguous bytes a thread.  With k a
// multiple of 8 the eight share a code word and a scale; otherwise the output's
// rows start at odd places, and a thread takes 8 values of the flat output,
// each with its own row, code and scale.
template <typename T, bool kWhole>
__global__ void __launch_bounds__(kConvThreads) dequantize(const DequantParams p)
{
    const int64_t b = blockIdx.z;
    const uint8_t* codes = p.codes + b * p.rows * p.pitch;
    const uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    T* y = static_cast<T*>(p.y) + b * p.rows * p.k;
    const int64_t n = p.rows * p.k;
    griddep_wait();
    griddep_launch_dependents();
    const int64_t f = (static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x) * 8;
    if (f >= n) return;
    int64_t r = f / p.k, i = f - r * p.k;
    T v[8];
    if (kWhole) {
        uint32_t h[4];
        halves_of(*reinterpret_cast<const uint32_t*>(codes + r * p.pitch + (i >> 1)), h);
        const float s = scale_value(scales[scale_at(r, i >> 5, p.kt)]);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            v[c] = Elem<T>::from_f32(s * Elem<__half>::to_f32(c & 1 ? h[c >> 1] >> 16 : h[c >> 1] & 0xFFFFu));
    } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            v[c] = Elem<T>::from_f32(0.f);
            if (f + c < n) {
                const uint32_t byte = codes[r * p.pitch + (i >> 1)];
                uint32_t h[4];
                halves_of(byte >> (4 * (i & 1)) & 15u, h);
                v[c] = Elem<T>::from_f32(scale_value(scales[scale_at(r, i >> 5, p.kt)]) *
                                         Elem<__half>::to_f32(h[0] & 0xFFFFu));
            }
            if (++i == p.k) i = 0, ++r;
        }
    }
    // (the batch's matrices start wherever the previous one ends)
    if (f + 8 <= n && reinterpret_cast<uintptr_t>(y + f) % 16 == 0) {
        uint4 o[sizeof(T) / 2];
        memcpy(o, v, sizeof(v));
#pragma unroll
        for (unsigned c = 0; c < sizeof(T) / 2; ++c) reinterpret_cast<uint4*>(y + f)[c] = o[c];
    } else {
        for (int c = 0; c < 8; ++c)
            if (f + c < n) y[f + c] = v[c];
    }
}

}  // namespace mxf4_dev
