// MXFP4 quantisation and its inverse: pure streaming kernels, bound by HBM.
//
// Quantising reads 2 (fp16, bf16) or 4 bytes a value once and writes 17/32 of
// a byte; the arithmetic (a maximum, one multiply, one conversion a value)
// hides under the loads.  A block of threads takes a tile of 128 rows x 256
// values: the 128 rows fill whole 512-byte scale tiles, which are put together
// in shared memory and leave in one piece, and 256 values of a row are 128
// bytes of codes, one full line.
//
// Measured on 131072 x 7168 fp16: 336 us (7.1 TB/s), the inverse 349 us (6.8), fp32
// 577 us (7.4); 65536 x 7168 transposed 241 us (4.9), fp32 312 us (6.8); rows that
// start anywhere, 65536 x 7001: 244 us (4.8) and 286 us (4.1), bound by the second
// load and the shift of every 16 bytes (issue 57 and 73 % of cycles).
#pragma once

#include "mxf4_format.cuh"

namespace mxf4_dev {

constexpr int kTileRows = 128, kTileVals = 256, kConvThreads = 256;
constexpr int kStridedVals = 256;  // values of a row in a tile of the strided form
constexpr int kDequantRows = 64;   // rows a block writes

template <bool kValue>
struct Bool {
    static constexpr bool value = kValue;
};

struct QuantParams {
    const void* x;
    int64_t sb, sr, sk;   // element strides
    uint8_t* codes;
    uint8_t* scales;
    int64_t rows, k, pitch;   // pitch: code bytes a row
    int64_t kt;               // scale tiles along k
    int64_t row_tiles;        // ceil(rows / 128)
    int64_t col_tiles;        // tiles along k
};

// Unit stride along k: a warp takes the 256 values of one row, 8 a lane, so its
// loads and its 128 bytes of codes are contiguous; four lanes share a block.
template <typename T, bool kVec>
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
    const int i = static_cast<int>(i0) + lane * 8, n = static_cast<int>(p.k);   // (k is below 2^31)
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kUnroll = sizeof(T) == 4 ? 2 : 4;
    constexpr int kWarps = kConvThreads / 32;
    const T* src = x + (r0 + warp) * p.sr;
    uint8_t* dst = codes + (r0 + warp) * p.pitch + (i >> 1);
    // this lane's scale byte: block lane / 4 of the row, tile lane / 16
    uint8_t* mine = sc + (lane >> 4) * kScaleTile + ((lane >> 2) & 3);
    const bool some = i >> 5 < (n + 31) >> 5;
    const int64_t step = kWarps * p.sr, cstep = kWarps * p.pitch;
    auto rows = [&](auto whole) {   // whole: the tile lies inside the matrix
        constexpr bool kWhole = decltype(whole)::value;
#pragma unroll 1
        for (int rr = warp; rr < kTileRows; rr += kWarps * kUnroll) {
            if (!kWhole && r0 + rr >= p.rows) {   // (few rows: the rest of the scale tile is padding)
                if ((lane & 3) == 0)
                    for (int lr = rr; lr < kTileRows; lr += kWarps) mine[(lr & 31) * 16 + (lr >> 5) * 4] = 0;
                break;
            }
            uint32_t w[kUnroll][8 * sizeof(T) / 4];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int k = kWhole || r0 + rr + u * kWarps < p.rows ? n : 0;
                if (kWhole && kVec) {
#pragma unroll
                    for (unsigned c = 0; c < sizeof(T) / 2; ++c) {
                        const uint4 v = ld_nc_v4(src + u * step + i + c * (16 / sizeof(T)));
                        w[u][4 * c] = v.x, w[u][4 * c + 1] = v.y, w[u][4 * c + 2] = v.z, w[u][4 * c + 3] = v.w;
                    }
                } else {
                    load8<T, kVec>(src + u * step, i, k, w[u]);
                    if (!kWhole && i + 8 > k) mask_tail<T>(w[u], k - i);
                }
            }
            src += kUnroll * step;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int lr = rr + u * kWarps;
                uint32_t top = top_bits<T>(w[u]);
                top = max(top, __shfl_xor_sync(~0u, top, 1));
                top = max(top, __shfl_xor_sync(~0u, top, 2));
                const bool in = kWhole || (some && r0 + lr < p.rows);
                const uint32_t code = in ? scale_code<T>(top) : 0u;
                if (in) *reinterpret_cast<uint32_t*>(dst + u * cstep) = codes_of<T>(w[u], code);
                if ((lane & 3) == 0) mine[(lr & 31) * 16 + (lr >> 5) * 4] = static_cast<uint8_t>(code);
            }
            dst += kUnroll * cstep;
        }
    };
    if (r0 + kTileRows <= p.rows && i0 + kTileVals <= p.k)
        rows(Bool<true>());
    else
        rows(Bool<false>());
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
// contiguous loads; the codes of the tile are turned in shared memory.  A tile
// is wide enough for whole 128-byte lines of codes: with half lines, 64 bytes a
// row, a 65536 x 7168 fp16 matrix took 1.04 ms instead of 0.24 (5.0 TB/s).
template <typename T>
__global__ void __launch_bounds__(kConvThreads, 4) quantize_strided(const QuantParams p)
{
    constexpr int kPitch = kStridedVals / 2 + 16, kScTiles = kStridedVals / 128;   // bytes a row of the staged codes: 16-byte stores spread over the banks
    __shared__ __align__(16) uint8_t cs[kTileRows * kPitch];
    __shared__ __align__(16) uint8_t sc[kScTiles * kScaleTile];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ct = blockIdx.x / p.row_tiles, rt = blockIdx.x - ct * p.row_tiles;   // (neighbours along the rows)
    const int64_t r0 = rt * kTileRows, i0 = ct * kStridedVals;
    const int64_t b = blockIdx.z;
    const T* x = static_cast<const T*>(p.x) + b * p.sb;
    uint8_t* codes = p.codes + b * p.rows * p.pitch;
    uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    griddep_wait();
    griddep_launch_dependents();
    const int lr = (warp & 3) * 32 + lane;
    const int64_t r = r0 + lr;
    auto blocks = [&](auto whole) {   // whole: the tile lies inside the matrix, its strides in 32 bits
        constexpr bool kWhole = decltype(whole)::value;
#pragma unroll 1
        for (int blk = warp >> 2; blk < kStridedVals / 32; blk += kConvThreads / 128) {
            const int64_t i = i0 + blk * 32;
            uint32_t w[4][8 * sizeof(T) / 4];
            const T* src = x + r * p.sr + i * p.sk;
            const int left = kWhole ? 32 : static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(32), p.k - i)));
            const bool row = kWhole || r < p.rows;
            auto at = [&](int c) { return kWhole ? src + static_cast<uint32_t>(c) * static_cast<uint32_t>(p.sk) : src + c * p.sk; };
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] = c < left && row ? (sizeof(T) == 4 ? ld_nc_u32(at(c)) : ld_nc_u16(at(c))) : 0u;
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
                if (sizeof(T) == 4)
                    w[c >> 3][c & 7] = v[c], w[c >> 3][(c & 7) + 1] = v[c + 1];
                else
                    w[c >> 3][(c & 7) >> 1] = __byte_perm(v[c], v[c + 1], 0x5410);
            }
            const uint32_t top = max(max(top_bits<T>(w[0]), top_bits<T>(w[1])), max(top_bits<T>(w[2]), top_bits<T>(w[3])));
            const uint32_t code = kWhole || (row && left > 0) ? scale_code<T>(top) : 0u;
            uint4 c4;
            c4.x = codes_of<T>(w[0], code), c4.y = codes_of<T>(w[1], code);
            c4.z = codes_of<T>(w[2], code), c4.w = codes_of<T>(w[3], code);
            *reinterpret_cast<uint4*>(cs + lr * kPitch + blk * 16) = c4;
            sc[(blk >> 2) * kScaleTile + lane * 16 + (warp & 3) * 4 + (blk & 3)] = static_cast<uint8_t>(code);
        }
    };
    if (r0 + kTileRows <= p.rows && i0 + kStridedVals <= p.k && p.sk < (int64_t(1) << 26))
        blocks(Bool<true>());
    else
        blocks(Bool<false>());
    __syncthreads();
    const int64_t bytes = min(p.pitch - (i0 >> 1), static_cast<int64_t>(kStridedVals / 2));
    constexpr int kWords = kStridedVals / 32;   // 16-byte words of a row's codes
    for (int t = threadIdx.x; t < kTileRows * kWords; t += kConvThreads) {
        const int row = t / kWords, c = t % kWords;
        if (r0 + row < p.rows && c * 16 < bytes)
            *reinterpret_cast<uint4*>(codes + (r0 + row) * p.pitch + (i0 >> 1) + c * 16) =
                *reinterpret_cast<const uint4*>(cs + row * kPitch + c * 16);
    }
    const int t = threadIdx.x >> 5;
    if (t < kScTiles && (i0 >> 7) + t < p.kt)
        reinterpret_cast<uint4*>(scales + (rt * p.kt + (i0 >> 7) + t) * kScaleTile)[lane] =
            reinterpret_cast<const uint4*>(sc + t * kScaleTile)[lane];
}

struct DequantParams {
    const uint8_t* codes;
    const uint8_t* scales;
    void* y;
    int64_t rows, k, pitch, kt, row_tiles;
    int64_t col_tiles;   // of 256 values and the 7 that a row may begin before one
};

// A warp writes 256 neighbouring values of a row, 8 a lane, from the first
// multiple of 8 values of the output's memory on, so that every full store is
// aligned whatever the row's length; the codes are then taken from any nibble on
// (two words and a shift), and 8 values may lie in two blocks.
// kVec: every row starts aligned, so that 8 values are one word of codes.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kConvThreads) dequantize(const DequantParams p)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t rt = blockIdx.x / p.col_tiles, b = blockIdx.z;
    const int c0 = static_cast<int>(blockIdx.x - rt * p.col_tiles) * 32 + lane;   // this lane's group of 8
    const int k = static_cast<int>(p.k), words = static_cast<int>(p.pitch >> 2);   // (k is below 2^31)
    const uint8_t* codes = p.codes + b * p.rows * p.pitch;
    const uint8_t* scales = p.scales + b * p.row_tiles * p.kt * kScaleTile;
    T* y = static_cast<T*>(p.y) + b * p.rows * p.k;
    griddep_wait();
    griddep_launch_dependents();
    constexpr int kUnroll = 4, kWarps = kConvThreads / 32;
    const int64_t r0 = rt * kDequantRows;
    T* to = y + (r0 + warp) * p.k;
    const uint8_t* from = codes + (r0 + warp) * p.pitch;
    // a tile's 64 rows are half of a scale tile's: place of (row 0, block 0)
    const uint8_t* srow = scales + (r0 >> 7) * p.kt * kScaleTile + ((r0 >> 5) & 3) * 4;
    auto place = [&](int lr, int blk) { return srow + static_cast<int64_t>(blk >> 2) * kScaleTile + (blk & 3) + (lr & 31) * 16 + (lr >> 5) * 4; };
#pragma unroll 1
    for (int rr = warp; rr < kDequantRows; rr += kUnroll * kWarps, to += kUnroll * kWarps * p.k, from += kUnroll * kWarps * p.pitch) {
        uint32_t w[kUnroll][2], sc[kUnroll][2];
        int i0[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int lr = rr + u * kWarps;
            const int shift = kVec ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(to + u * kWarps * p.k) / sizeof(T) & 7);
            const int i = c0 * 8 - shift;
            i0[u] = r0 + lr < p.rows && i < k ? i : k;
            w[u][0] = w[u][1] = sc[u][0] = sc[u][1] = 0u;
            if (i0[u] >= k) continue;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(from + u * kWarps * p.pitch);
            if (kVec) {
                w[u][0] = __ldg(src + c0);
                sc[u][0] = __ldg(place(lr, i >> 5));
                continue;
            }
            const int word = i >> 3;   // (word -1 holds nothing of the row)
            if (word >= 0) w[u][0] = __ldg(src + word);
            if (shift != 0 && word + 1 < words) w[u][1] = __ldg(src + word + 1);
            const int blk = max(i, 0) >> 5, last = min(i + 7, k - 1) >> 5;
            sc[u][0] = __ldg(place(lr, blk));
            sc[u][1] = last != blk ? __ldg(place(lr, last)) : sc[u][0];
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = i0[u];
            if (i >= k) continue;
            T* row = to + u * kWarps * p.k;
            uint32_t h[4];
            halves_of(kVec ? w[u][0] : __funnelshift_r(w[u][0], w[u][1], 4 * (i & 7)), h);
            T v[8];
            uint4 o[sizeof(T) / 2];
            const int turn = kVec ? 8 : 32 - (i & 31);   // values of the first block
            if (Elem<T>::kInf == 0x7C00u && sc[u][0] - 103u <= 39u && (kVec || sc[u][1] - 103u <= 39u)) {
                // fp16 holds the factors (2^-24 to 2^15): one rounding, two values an instruction
                auto half_scale = [](uint32_t c) { return c >= 113u ? (c - 112u) << 10 : 1u << (c - 103u); };
                const uint32_t f0 = half_scale(sc[u][0]), f1 = kVec ? f0 : half_scale(sc[u][1]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t f = (2 * c < turn ? f0 : f1) | (2 * c + 1 < turn ? f0 : f1) << 16;
                    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[c]) : "r"(h[c]), "r"(f));
                }
                o[0] = make_uint4(h[0], h[1], h[2], h[3]);
            } else {
                const float s0 = scale_value(sc[u][0]), s1 = kVec ? s0 : scale_value(sc[u][1]);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    v[c] = Elem<T>::from_f32((c < turn ? s0 : s1) * Elem<__half>::to_f32(c & 1 ? h[c >> 1] >> 16 : h[c >> 1] & 0xFFFFu));
                memcpy(o, v, sizeof(v));
            }
            if (kVec || (i >= 0 && i + 8 <= k)) {
#pragma unroll
                for (unsigned c = 0; c < sizeof(T) / 2; ++c) __stcs(reinterpret_cast<uint4*>(row + i) + c, o[c]);
            } else {
                memcpy(v, o, sizeof(v));
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    if (i + c >= 0 && i + c < k) row[i + c] = v[c];
            }
        }
    }
}

}  // namespace mxf4_dev
