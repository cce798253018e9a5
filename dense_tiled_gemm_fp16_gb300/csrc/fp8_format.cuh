// The 8-bit format on the device: e4m3 values, a power-of-two scale for 128 of
// them along the contracted axis, and its conversions.
#pragma once

#include "mxf4_format.cuh"

namespace fp8_dev {

using namespace gemm_f16_dev;
using mxf4_dev::Elem;
using mxf4_dev::kScaleTile;   // 512 bytes: 128 rows x 4 blocks
using mxf4_dev::pow2f;
using mxf4_dev::scale_value;

constexpr int kBlock = 128;   // values that share a scale

template <bool kValue>
struct Bool {
    static constexpr bool value = kValue;
};

// Scale code of a block whose largest magnitude has the bits `top`: s + 127 for the
// smallest s with |x| <= 448 * 2^s (448 = 1.75 * 2^8 is e4m3's largest), 255 (NaN)
// with an infinity or a NaN among them.  Being no smaller than the largest value
// needs, no value saturates; a scale that is a power of two rounds nothing itself,
// and the tensor cores apply it to the products.
__device__ __forceinline__ uint32_t scale_code_f32(float top)
{
    const uint32_t u = __float_as_uint(top);
    if (u >= 0x7F800000u) return 255u;
    const int s = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u);
    return static_cast<uint32_t>(max(s, -127) + 127);
}

template <typename T>
__device__ __forceinline__ uint32_t scale_code(uint32_t top)
{
    return top >= Elem<T>::kInf ? 255u : scale_code_f32(Elem<T>::to_f32(top));
}

// 2^-s of a scale code (not 255).
__device__ __forceinline__ float inverse_scale(uint32_t code) { return pow2f(127 - static_cast<int>(code)); }

// Four values as e4m3, the first in the low byte: round to nearest even.
__device__ __forceinline__ uint32_t e4m3_of(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Eight values (words w of type T) times 2^-s as e4m3.  The products are exact but
// where they are subnormal in fp32 or fp16, at most 2^-14, where the least step of
// e4m3 is 2^-9: a value on the wrong side of a rounding point does not come of it.
template <typename T>
__device__ __forceinline__ uint2 codes8(const uint32_t* w, uint32_t code)
{
    if (code == 255u) return make_uint2(0u, 0u);
    if constexpr (Elem<T>::kInf == 0x7C00u) {
        if (code >= 112u) {   // fp16 holds 2^-s up to 2^15: two values an instruction
            const uint32_t f = (142u - code) << 10, ff = f | f << 16;
            uint2 r;
            asm("{\n\t.reg .b16 b0, b1, b2, b3;\n\t.reg .b32 p0, p1, p2, p3;\n\t"
                "mul.rn.f16x2 p0, %2, %6;\n\tmul.rn.f16x2 p1, %3, %6;\n\t"
                "mul.rn.f16x2 p2, %4, %6;\n\tmul.rn.f16x2 p3, %5, %6;\n\t"
                "cvt.rn.satfinite.e4m3x2.f16x2 b0, p0;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b1, p1;\n\t"
                "cvt.rn.satfinite.e4m3x2.f16x2 b2, p2;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b3, p3;\n\t"
                "mov.b32 %0, {b0, b1};\n\tmov.b32 %1, {b2, b3};\n\t}"
                : "=r"(r.x), "=r"(r.y)
                : "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(ff));
            return r;
        }
    }
    const float f = inverse_scale(code);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mxf4_dev::value_of<T>(w, i) * f;
    return make_uint2(e4m3_of(v[0], v[1], v[2], v[3]), e4m3_of(v[4], v[5], v[6], v[7]));
}

// Four e4m3 values (a word) as two half2, exactly.
__device__ __forceinline__ void halves_of(uint32_t codes, uint32_t* h)
{
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "r"(codes));
}

// Byte of row r's scale of block b inside a matrix's scale tiles.
__host__ __device__ __forceinline__ int64_t scale_at(int64_t r, int64_t b, int64_t kt)
{
    return ((r >> 7) * kt + (b >> 2)) * kScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

}  // namespace fp8_dev
