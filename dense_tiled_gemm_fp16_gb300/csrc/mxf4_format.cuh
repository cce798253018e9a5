// The MXFP4 format on the device: scales, values to codes and back;
// and vector loads of rows that start at any element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace mxf4_dev {

using namespace gemm_f16_dev;

constexpr int kScaleTile = 512;   // bytes: 128 rows x 4 blocks

// 2^e exactly, -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// The scale's value: 2^(code - 127), 2^-127 is subnormal, 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t code)
{
    return code == 255u ? __uint_as_float(0x7FFFFFFFu) : code == 0u ? __uint_as_float(1u << 22) : pow2f(int(code) - 127);
}

template <typename T>
struct Elem;
template <>
struct Elem<__half> {
    static constexpr uint32_t kAbs = 0x7FFFu, kInf = 0x7C00u;
    static __device__ float to_f32(uint32_t b) { return __half2float(__ushort_as_half(static_cast<unsigned short>(b))); }
    static __device__ __half from_f32(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr uint32_t kAbs = 0x7FFFu, kInf = 0x7F80u;
    static __device__ float to_f32(uint32_t b) { return __uint_as_float(b << 16); }
    static __device__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<float> {
    static constexpr uint32_t kAbs = 0x7FFFFFFFu, kInf = 0x7F800000u;
    static __device__ float to_f32(uint32_t b) { return __uint_as_float(b); }
    static __device__ float from_f32(float v) { return v; }
};

// Largest magnitude of 8 values as the bits of |x|: for IEEE types the order
// of the bits is the order of the magnitudes, infinity and NaN above them all.
template <typename T>
__device__ __forceinline__ uint32_t top_bits(const uint32_t* w)
{
    if (sizeof(T) == 4) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, w[i] & Elem<T>::kAbs);
        return m;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
}

template <typename T>
__device__ __forceinline__ float value_of(const uint32_t* w, int i)
{
    if (sizeof(T) == 4) return Elem<T>::to_f32(w[i]);
    return Elem<T>::to_f32(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu);
}

// Scale code of a block whose largest magnitude has the bits `top`.
template <typename T>
__device__ __forceinline__ uint32_t scale_code(uint32_t top)
{
    if (top >= Elem<T>::kInf) return 255u;
    const float a = Elem<T>::to_f32(top);
    // floor(log2 a) from the bits; a subnormal a (fp32, bf16) is at most 2^-127
    // below the clamp anyway, since s = floor(log2 a) - 2 is at least -127.
    const int e = static_cast<int>(__float_as_uint(a) >> 23) - 127;   // zero and subnormals: -127
    return static_cast<uint32_t>(max(e - 2, -127) + 127);
}

// Eight values times 2^-s as e2m1 codes, the first in the low nibble: round to
// nearest even, magnitudes above 6 saturate.  The products are exact but where
// they are subnormal, far under the rounding point 0.25.
__device__ __forceinline__ uint32_t codes_of_f32(const float* v)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

template <typename T>
__device__ __forceinline__ uint32_t codes_of(const uint32_t* w, uint32_t code)
{
    if (code == 255u) return 0u;
    uint32_t r;
    if (Elem<T>::kInf == 0x7C00u && code >= 112u) {
        // fp16 holds 2^-s up to 2^15 (largest magnitudes from 2^-13 on): two values an instruction
        const uint32_t f = (142u - code) << 10, ff = f | f << 16;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 p0, p1, p2, p3;\n\t"
            "mul.rn.f16x2 p0, %1, %5;\n\tmul.rn.f16x2 p1, %2, %5;\n\t"
            "mul.rn.f16x2 p2, %3, %5;\n\tmul.rn.f16x2 p3, %4, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f16x2 b0, p0;\n\tcvt.rn.satfinite.e2m1x2.f16x2 b1, p1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f16x2 b2, p2;\n\tcvt.rn.satfinite.e2m1x2.f16x2 b3, p3;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(r)
            : "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(ff));
        return r;
    }
    const float f = pow2f(127 - static_cast<int>(code));
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value_of<T>(w, i) * f;
    return codes_of_f32(v);
}

// Eight e2m1 codes (a 32-bit word) as four half2, exactly.
__device__ __forceinline__ void halves_of(uint32_t codes, uint32_t* h)
{
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// ------------------------------------------------------- rows at any place
// Sixteen bytes from byte `o` (0, 2, .. 14) of 32.
__device__ __forceinline__ void funnel16(const uint32_t* in, uint32_t o, uint32_t* out)
{
    uint32_t w[6], v[5];
#pragma unroll
    for (int c = 0; c < 6; ++c) w[c] = o & 8u ? in[c + 2] : in[c];
#pragma unroll
    for (int c = 0; c < 5; ++c) v[c] = o & 4u ? w[c + 1] : w[c];
#pragma unroll
    for (int c = 0; c < 4; ++c) out[c] = __funnelshift_r(v[c], v[c + 1], (o & 2u) * 8u);
}

// The words of 8 values of a row of unit stride, value `i` first, values from
// `k` on undefined (mask_tail): aligned 16-byte loads, one more than the values
// fill where the row starts at another place, each holding at least one of them.
// kVec: every row starts aligned.
template <typename T, bool kVec>
__device__ __forceinline__ void load8(const T* row, int i, int k, uint32_t* w)
{
    constexpr int kLoads = sizeof(T) / 2;   // of a row that starts aligned
    if constexpr (kVec) {
#pragma unroll
        for (int c = 0; c < kLoads; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (i + c * (16 / static_cast<int>(sizeof(T))) < k) v = ld_nc_v4(row + i + c * (16 / sizeof(T)));
            w[4 * c] = v.x, w[4 * c + 1] = v.y, w[4 * c + 2] = v.z, w[4 * c + 3] = v.w;
        }
    } else {
        uint32_t t[4 * (kLoads + 1)];
#pragma unroll
        for (int c = 0; c < 4 * (kLoads + 1); ++c) t[c] = 0u;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + i);
        const uint32_t o = at & 15u;
        const uint4* p = reinterpret_cast<const uint4*>(at - o);
        const int bytes = i < k ? min(8, k - i) * static_cast<int>(sizeof(T)) + static_cast<int>(o) : 0;
#pragma unroll
        for (int c = 0; c <= kLoads; ++c)
            if (16 * c < bytes) {
                const uint4 v = ld_nc_v4(p + c);
                t[4 * c] = v.x, t[4 * c + 1] = v.y, t[4 * c + 2] = v.z, t[4 * c + 3] = v.w;
            }
#pragma unroll
        for (int c = 0; c < kLoads; ++c) funnel16(t + 4 * c, o, w + 4 * c);
    }
}

// Values from `n` on of 8 set to zero.
template <typename T>
__device__ __forceinline__ void mask_tail(uint32_t* w, int n)
{
#pragma unroll
    for (int c = 0; c < 8 * static_cast<int>(sizeof(T)) / 4; ++c) {
        if (sizeof(T) == 4)
            w[c] = c < n ? w[c] : 0u;
        else
            w[c] = 2 * c + 1 < n ? w[c] : 2 * c < n ? w[c] & 0xFFFFu : 0u;
    }
}

}  // namespace mxf4_dev
