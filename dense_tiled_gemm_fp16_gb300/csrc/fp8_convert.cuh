// Quantisation to 8 bits and its inverse: streaming kernels, bound by HBM (2 or 4
// bytes a value in, 1 + 1/128 out, and back; the inverse of 131072 x 7168 to fp16 takes 409
// us, 6.9 TB/s).
//
// A block of threads takes a tile of 128 rows x 512 values: whole 512-byte scale
// tiles, put together in shared memory, and whole 128-byte lines of codes.
#pragma once

#include "fp8_format.cuh"

namespace fp8_dev {

constexpr int kTileRows = 128, kTileVals = 512, kConvThreads = 256;
constexpr int kDequantRows = 32;   // rows a block writes

struct QuantParams {
    const void* x;
    int64_t sb, sr, sk;   // element strides
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows, k, pitch;   // pitch: code bytes a row
    int64_t kt, row_tiles;
    int64_t tile_rows;        // rows of a tile that a block takes: 8, 16 or 32 (strided: 128)
};

// Unit stride along k: a warp takes the 512 values of a row of the tile, 8 a lane twice,
// so that its loads and stores are contiguous, 16 lanes share a block and the row's four
// scales make one word.  Rows of a scale tile that another block of threads takes
// (tile_rows < 128) are left to it; the one with the matrix's last row also writes the
// padding rows' scales.
//
// One row at a time and full occupancy keep more loads under way than several rows and
// less of it: 131072 x 7168 in fp16 565 us with four rows a warp, 445 with two, 409 so
// (6.9 TB/s); fp32 has the bytes under way with half the occupancy (32768 x 7168: 175 us,
// 6.7 TB/s).  (At 32 registers the aligned 16-bit form keeps 12 to 16 bytes a thread in local
// memory.)  Rows that start anywhere, 32768 x 4097 in bf16: 89 us (4.5 TB/s), by the second
// load and the shift of every 16 bytes, most of which the lane beside has loaded, too.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kConvThreads, sizeof(T) == 4 ? 4 : 8) quantize_rows(const QuantParams p)
{
    constexpr int kWarps = kConvThreads / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t parts = (p.rows + p.tile_rows - 1) / p.tile_rows;
    const int64_t ct = blockIdx.x / parts, part = blockIdx.x - ct * parts;
    const int64_t r0 = part * p.tile_rows, b = blockIdx.z;
    const T* x = static_cast<const T*>(p.x) + b * p.sb;
    uint8_t* codes = p.codes + b * p.rows * p.pitch;
    uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    const int n = static_cast<int>(p.k), i = static_cast<int>(ct) * kTileVals + lane * 8;   // (k is below 2^31)
    griddep_wait();
    griddep_launch_dependents();
    const int64_t end = min(p.rows, r0 + p.tile_rows);
    auto rows = [&](auto whole) {   // whole: no value of the tile is past the row's end
        constexpr bool kWhole = decltype(whole)::value;
#pragma unroll 1
        for (int64_t r = r0 + warp; r < end; r += kWarps) {
            uint32_t w[2][8 * sizeof(T) / 4], word = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mxf4_dev::load8<T, kVec>(x + r * p.sr, i + 256 * h, n, w[h]);
                if (!kWhole && i + 256 * h + 8 > n) mxf4_dev::mask_tail<T>(w[h], n - i - 256 * h);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t top = mxf4_dev::top_bits<T>(w[h]);
#pragma unroll
                for (int d = 1; d < 16; d *= 2) top = max(top, __shfl_xor_sync(~0u, top, d));
                const bool some = kWhole || ((i + 256 * h) & ~(kBlock - 1)) < n;
                const uint32_t code = some ? scale_code<T>(top) : 0u;
                const uint2 c = codes8<T>(w[h], code);
                if (kWhole || i + 256 * h + 8 <= p.pitch) *reinterpret_cast<uint2*>(codes + r * p.pitch + i + 256 * h) = c;
                word |= (code | __shfl_xor_sync(~0u, code, 16) << 8) << (16 * h);
            }
            if (lane == 0) *reinterpret_cast<uint32_t*>(scales + scale_at(r, 4 * ct, p.kt)) = word;
        }
    };
    if ((ct + 1) * kTileVals <= p.k)
        rows(Bool<true>());
    else
        rows(Bool<false>());
    if (end == p.rows)   // padding rows of the last scale tile
        for (int64_t r = p.rows + threadIdx.x; r < p.row_tiles * 128; r += kConvThreads)
            *reinterpret_cast<uint32_t*>(scales + scale_at(r, 4 * ct, p.kt)) = 0u;
}

// Any strides (a transposed view has unit stride along the rows): a lane takes a
// block of a row and a warp 32 neighbouring rows, so that a unit row stride gives
// contiguous loads; the codes, 128 bytes a row, are turned in shared memory.  A lane's 128
// values stay in its registers from the largest magnitude on, 254 registers in fp16 and 182 in
// bf16: one block of threads an SM, with too few loads of 64 bytes a warp under way.  A weight
// [7168, 2048] takes 51 us in fp16 and 73 in bf16, 64 of them 2560 and 3570 (1.1 and 0.8 TB/s;
// one that is contiguous along k 8.5 us, its bytes need 6.5).
template <typename T>
__global__ void __launch_bounds__(kConvThreads) quantize_strided(const QuantParams p)
{
    constexpr int kPitch = kBlock + 16;   // bytes a row of the staged codes: 16-byte stores spread over the banks
    constexpr int kWords = kBlock * sizeof(T) / 4;
    __shared__ __align__(16) uint8_t cs[2][kTileRows * kPitch];
    __shared__ __align__(16) uint8_t sc[kScaleTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2;
    const int64_t ct = blockIdx.x / p.row_tiles, rt = blockIdx.x - ct * p.row_tiles;   // (neighbours along the rows)
    const int64_t r0 = rt * kTileRows, b = blockIdx.z;
    const T* x = static_cast<const T*>(p.x) + b * p.sb;
    uint8_t* codes = p.codes + b * p.rows * p.pitch;
    uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    griddep_wait();
    griddep_launch_dependents();
    const int lr = (warp & 3) * 32 + lane;
    const int64_t r = r0 + lr;
#pragma unroll 1
    for (int it = 0; it < 2; ++it) {
        const int blk = 2 * it + half;   // of the tile's four
        const int64_t i = ct * kTileVals + blk * kBlock;
        const int left = r < p.rows ? static_cast<int>(max(int64_t(0), min(int64_t(kBlock), p.k - i))) : 0;
        const T* src = x + r * p.sr + i * p.sk;
        uint32_t w[kWords];
#pragma unroll
        for (int c = 0; c < kBlock; ++c) {
            const uint32_t v = c < left ? (sizeof(T) == 4 ? ld_nc_u32(src + c * p.sk) : ld_nc_u16(src + c * p.sk)) : 0u;
            if (sizeof(T) == 4)
                w[c] = v;
            else
                w[c >> 1] = c & 1 ? w[c >> 1] | v << 16 : v;
        }
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < 16; ++c) top = max(top, mxf4_dev::top_bits<T>(w + c * kWords / 16));
        const uint32_t code = left > 0 ? scale_code<T>(top) : 0u;
#pragma unroll
        for (int c = 0; c < 16; c += 2) {
            const uint2 a = codes8<T>(w + c * kWords / 16, code), d = codes8<T>(w + (c + 1) * kWords / 16, code);
            *reinterpret_cast<uint4*>(cs[half] + lr * kPitch + c * 8) = make_uint4(a.x, a.y, d.x, d.y);
        }
        sc[lane * 16 + (warp & 3) * 4 + blk] = static_cast<uint8_t>(code);
        __syncthreads();
        for (int t = threadIdx.x & 127; t < kTileRows * 8; t += 128) {
            const int row = t >> 3, c = t & 7;
            if (r0 + row < p.rows && i + c * 16 < p.pitch)
                *reinterpret_cast<uint4*>(codes + (r0 + row) * p.pitch + i + c * 16) =
                    *reinterpret_cast<const uint4*>(cs[half] + row * kPitch + c * 16);
        }
        __syncthreads();
    }
    if (warp == 0)
        reinterpret_cast<uint4*>(scales + (rt * p.kt + ct) * kScaleTile)[lane] = reinterpret_cast<const uint4*>(sc)[lane];
}

struct DequantParams {
    const uint8_t* codes;
    const uint8_t* scales;
    void* y;
    int64_t rows, k, pitch, kt, row_tiles;
    int64_t col_tiles;   // of 256 values and the 7 that a row may begin before one
};

// A warp writes 256 neighbouring values of a row, 8 a lane, from the first multiple
// of 8 values of the output's memory on, so that every full store is aligned
// whatever the row's length; the codes are then taken from any byte on (three words
// and a shift), and 8 values may lie in two blocks.
// kVec: every row starts aligned, so that 8 values are 8 aligned bytes of codes.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kConvThreads) dequantize(const DequantParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rt = blockIdx.x / p.col_tiles, b = blockIdx.z;
    const int64_t c0 = (blockIdx.x - rt * p.col_tiles) * 32 + lane;   // this lane's group of 8
    const uint8_t* codes = p.codes + b * p.rows * p.pitch;
    const uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    T* y = static_cast<T*>(p.y) + b * p.rows * p.k;
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kUnroll = 4, kWarps = kConvThreads / 32;
    const int64_t k = p.k, words = p.pitch >> 2, r0 = rt * kDequantRows + warp;
    uint32_t w[kUnroll][3], sc[kUnroll][2];
    int64_t at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t r = r0 + u * kWarps;
        const int shift = kVec ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(y + r * k) / sizeof(T) & 7);
        const int64_t i = c0 * 8 - shift;
        at[u] = r < p.rows && i < k ? i : k;
        w[u][0] = w[u][1] = w[u][2] = sc[u][0] = sc[u][1] = 0u;
        if (at[u] >= k) continue;
        const uint32_t* src = reinterpret_cast<const uint32_t*>(codes + r * p.pitch);
        if (kVec) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src) + c0);
            w[u][0] = v.x, w[u][1] = v.y;
            sc[u][0] = __ldg(scales + scale_at(r, i >> 7, p.kt));
            continue;
        }
        const int64_t word = i >> 2;   // (words -1 and -2 hold nothing of the row)
#pragma unroll
        for (int c = 0; c < 3; ++c)
            if (word + c >= 0 && word + c < words) w[u][c] = __ldg(src + word + c);
        const int64_t first = max(i, int64_t(0)) >> 7, last = min(i + 7, k - 1) >> 7;
        sc[u][0] = __ldg(scales + scale_at(r, first, p.kt));
        sc[u][1] = last != first ? __ldg(scales + scale_at(r, last, p.kt)) : sc[u][0];
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = at[u];
        if (i >= k) continue;
        T* row = y + (r0 + u * kWarps) * k;
        uint32_t h[4];
        const uint32_t o = 8 * static_cast<uint32_t>(i & 3);
        halves_of(kVec ? w[u][0] : __funnelshift_r(w[u][0], w[u][1], o), h);
        halves_of(kVec ? w[u][1] : __funnelshift_r(w[u][1], w[u][2], o), h + 2);
        T v[8];
        uint4 out[sizeof(T) / 2];
        const int turn = kVec ? 8 : static_cast<int>(kBlock - (i & (kBlock - 1)));   // values of the first block
        if (Elem<T>::kInf == 0x7C00u && sc[u][0] - 103u <= 39u && (kVec || sc[u][1] - 103u <= 39u)) {
            // fp16 holds the factors (2^-24 to 2^15): one rounding, two values an instruction
            auto half_scale = [](uint32_t c) { return c >= 113u ? (c - 112u) << 10 : 1u << (c - 103u); };
            const uint32_t f0 = half_scale(sc[u][0]), f1 = kVec ? f0 : half_scale(sc[u][1]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t f = (2 * c < turn ? f0 : f1) | (2 * c + 1 < turn ? f0 : f1) << 16;
                asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[c]) : "r"(h[c]), "r"(f));
            }
            out[0] = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            const float s0 = scale_value(sc[u][0]), s1 = kVec ? s0 : scale_value(sc[u][1]);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                v[c] = Elem<T>::from_f32((c < turn ? s0 : s1) * Elem<__half>::to_f32(c & 1 ? h[c >> 1] >> 16 : h[c >> 1] & 0xFFFFu));
            memcpy(out, v, sizeof(v));
        }
        if (kVec || (i >= 0 && i + 8 <= k)) {
#pragma unroll
            for (unsigned c = 0; c < sizeof(T) / 2; ++c) __stcs(reinterpret_cast<uint4*>(row + i) + c, out[c]);
        } else {
            memcpy(v, out, sizeof(v));
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (i + c >= 0 && i + c < k) row[i + c] = v[c];
        }
    }
}

}  // namespace fp8_dev
